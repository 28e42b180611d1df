// attn_common.hpp -- what the attention kernels share: how a call's work is cut
// into equal shares, and where partial results go.
//
// A UNIT is a run of rows that read the same keys: up to `ROWS` of a sequence's
// rows times its query heads of one kv head, flattened (row r of a unit is token
// r / group, head r % group of the sequence's rows).  Its work is the TILES of
// keys that any of its rows sees.  All units' tiles in one line are dealt to the
// workgroups in equal, contiguous shares, so that sequences of different lengths
// need no balancing and a single long one fills the chip.  A unit that lies
// within one share is finished there; of one that does not, each share leaves its
// running maximum, sum and unnormalised output in the workspace, and a second
// launch joins them in the order of the keys (no atomics: the result does not
// depend on timing).  A share continues at most one unit that began before it
// (slot 2w) and begins at most one that ends after it (slot 2w + 1).
#pragma once

#include "qp_device.hpp"
#include "decoder.hpp"

namespace qp {
namespace attn {

constexpr float LOG2E = 1.4426950408889634f;

// One entry per share: the unit that goes on in the next share.
struct Begun {
    int32_t first, last; // the shares that hold its first and its last tile; last = -1: no such unit
    int32_t token;       // the row of q of the sequence's first row
    int32_t row;         // the unit's first flattened row
    int32_t rows;        // its rows
    int32_t head;        // its kv head
    int32_t pad[2];
};

// The workspace of `shares` shares of units of up to `rows` rows.
struct Parts {
    Begun *begun;        // [shares]
    f32x2 *ml;           // [2 shares][rows]: maximum (of base-2 scores) and sum
    float *o;            // [2 shares][rows][d]
};

inline uint64_t parts_bytes(uint64_t shares, uint64_t rows, uint64_t d)
{
    return shares * sizeof(Begun) + 2 * shares * rows * (8 + 4 * d);
}

inline Parts parts_at(void *work, uint64_t shares, uint64_t rows)
{
    uint8_t *p = (uint8_t *)work;
    Parts r;
    r.begun = (Begun *)p;
    r.ml = (f32x2 *)(p + shares * sizeof(Begun));
    r.o = (float *)(p + shares * sizeof(Begun) + 2 * shares * rows * 8);
    return r;
}

// A value that is the same in the whole wave, in scalars.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t uniform(uint64_t v)
{
    return (uint64_t)uniform((uint32_t)(v >> 32)) << 32 | uniform((uint32_t)v);
}

// The same value, computed where it is used: what follows from it is not kept in
// registers through the loop, nor computed outside the branch it is in.
__device__ __forceinline__ uint32_t here(uint32_t v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// `bytes` of device memory from an address that is the same in the whole wave:
// what a lane reads behind them is 0, and not fetched.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t window_at(const void *base, uint64_t offset, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc((void *)uniform((uint64_t)base + offset), (short)0, (int)uniform(bytes), 0x00020000);
}

// Bytes behind the end of any such window: a lane that has no element of K there
// reads zeros (an element of its own, even times a zero of Q, would be NaN if infinite).
constexpr uint32_t BEYOND = 1u << 30;

// A sequence as the host's arrays give it; n = 0 where its numbers do not fit.
struct Seq {
    int token, n, len;       // first row, rows, positions
    int first;               // the first position that any row sees
};

__device__ __forceinline__ Seq read_seq(const AttnArgs &a, uint32_t s)
{
    Seq q;
    const int lo = a.q_start[s], hi = a.q_start[s + 1], len = a.kv_len[s];
    const bool ok = lo >= 0 && hi > lo && (uint32_t)hi <= a.t && (uint32_t)(hi - lo) <= a.max_q && len >= 0 &&
                    (uint32_t)len <= a.width << a.cache.page_log2;
    q.token = lo;
    q.n = ok ? hi - lo : 0;
    q.len = ok ? len : 0;
    const int64_t back = (int64_t)q.len - q.n - (int64_t)a.window + 1;
    q.first = a.window && back > 0 ? (int)back : 0;
    return q;
}

// The same for a sequence number that is the same in the whole wave, in scalars.
__device__ __forceinline__ Seq read_seq_uniform(const AttnArgs &a, uint32_t s)
{
    Seq q = read_seq(a, s);
    q.token = __builtin_amdgcn_readfirstlane(q.token);
    q.n = __builtin_amdgcn_readfirstlane(q.n);
    q.len = __builtin_amdgcn_readfirstlane(q.len);
    q.first = __builtin_amdgcn_readfirstlane(q.first);
    return q;
}

// The top bits of those of two BF16 values that are NaN or infinite (one more in
// the exponent's last place carries into the sign's).
__device__ __forceinline__ uint32_t odd_tops(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }
// The same as masks of 0xFFFF.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return (odd_tops(w) >> 15) * 0xFFFFu; }

// Scores (of base 2) from which on s * scale - m in one step, whose product is not
// rounded as m is, could be past 1 at the maximum itself, and past F32's exponents
// where they are 2^31: the row's scores are scaled first, and rounded.
__device__ __forceinline__ bool far(float m) { return __builtin_fabsf(m) >= 0x1p24f; }

// A scale of V, finite: 0 times it is 0 in the rows that do not see its key.
__device__ __forceinline__ float finite_scale(float s) { return __builtin_amdgcn_fmed3f(s, 0.0f, 3.4e38f); }

// Eight E4M3 codes as BF16 (exact: three bits of significand, exponents that fit).
__device__ __forceinline__ u32x4 bf16_of_e4m3(u32x2 c)
{
    auto two = [](uint32_t w, bool hi) {
        return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))
                  : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
    };
    return (u32x4){two(c[0], false), two(c[0], true), two(c[1], false), two(c[1], true)};
}

// The share that holds tile x of n tiles dealt to `shares` shares, share w
// taking tiles w * n / shares .. (w + 1) * n / shares - 1.
__device__ __forceinline__ uint32_t share_of(uint64_t x, uint64_t n, uint64_t shares)
{
    return (uint32_t)(((x + 1) * shares - 1) / n);
}

// Joins the parts of the units that several shares have (attn_decode.hip); `rows` of a part, of which `live` at most are used.
hipError_t launch_attn_join(const AttnArgs &a, const Parts &p, uint32_t shares, uint32_t rows, uint32_t live,
                            hipStream_t st);

// Rows of a sequence (times heads of a kv head) up to which attn_decode.hip serves
// it.  Measured with 4 kv heads, few rows' kernel / tiles', us, over 16 sequences of
// 4500 to 9001 positions, one of 32000, 64 of 500 to 1000:
//   rows                 16                    32                    64                   128
//   BF16 d =  64   31/33 16/18 21/24     34/33 18/20 24/25     41/37 22/22 30/28     65/45 30/25 45/33
//   BF16 d = 128   47/49 23/24 29/36     56/50 29/25 39/38     63/52 32/26 46/38    101/60 44/29 72/45
//   BF16 d = 192   77/85 29/31 40/41     95/87 33/32 54/43    139/94 49/35 85/49
//   BF16 d = 256  102/105 35/35 47/45   116/109 37/35 61/48  163/118 55/38 95/54
//   E4M3 d =  64   25/35 15/19 18/25     28/35 18/20 23/26     38/41 23/23 29/30     58/48 29/28 41/36
//   E4M3 d = 128   33/64 20/28 24/43     39/65 24/29 32/45     50/68 29/30 40/45     80/72 39/33 61/50
//   E4M3 d = 192   42/91 23/38 34/51     55/92 28/39 45/54     91/97 40/41 68/58
//   E4M3 d = 256   51/92 26/38 36/52     58/94 29/40 46/55     95/100 41/43 70/62
// The last rows of a range are near the crossing, which moves with the lengths: 16
// sequences of 9001 each, BF16, d = 128, 32 rows 61/65.
constexpr uint32_t decode_rows(uint32_t d, bool fp8) { return fp8 || d <= 64 ? 64 : d <= 128 ? 32 : 16; }
uint64_t decode_work(uint32_t rows, uint32_t d);
hipError_t launch_attn_decode(const AttnArgs &a, hipStream_t st);
uint64_t tiles_work(uint32_t d);
hipError_t launch_attn_tiles(const AttnArgs &a, hipStream_t st);

} // namespace attn
} // namespace qp
