// moe_fp8.hip -- a whole mixture-of-experts layer for a few tokens, in two
// launches.  x [T,H] BF16, router logits [T,E] F32, experts' weights E4M3 with
// one F32 scale per 128 x 128 block: w13 [E,2I,H] (gate rows, then up rows),
// w2 [E,H,I].
//
//   p      = softmax over the experts of a token's logits, its topk largest
//            kept (ties to the lowest expert), renormalised if asked
//   h_e    = silu(W1_e x) * (W3_e x)                       (F32)
//   out    = bf16( sum_e p_e W2_e h_e )
//
// Bytes bound it: the chosen experts' weights are read once for all their
// tokens, and nothing else is large.
//
//  * Routing is repeated by every workgroup of the first launch (a few logits
//    from L2, topk maxima over lanes): cheaper than a launch of its own.  It leaves
//    the active experts, their tokens and the weights in LDS, and workgroup 0
//    leaves the lists in the workspace for the second launch.
//  * The contraction runs on v_mfma_f32_4x4x4_16b_bf16: 16 blocks that are 16
//    K slices of the same 4 tokens and 4 weight rows.  Lane l loads 16 codes
//    of weight row l % 4 at byte 16 (l / 4) of a 256-byte window, so a load
//    instruction covers 4 rows x 256 contiguous bytes and feeds four MFMAs
//    with no exchange between lanes.  E4M3 converts to BF16 exactly.  A lane
//    receives its own weight row for the four tokens; its 16 codes lie in one
//    128-block, so a window's sums start from zero and join the running F32
//    sums with one FMA by the lane's block scale.
//  * h_e is kept between the launches as two BF16 rows, hi = bf16(h) and
//    lo = bf16(h - hi) (error 2^-17 of h, where one row would leave 2^-9).  They
//    are two of the four rows an MFMA takes, so one token costs the second
//    product no more than one rounded row would.
//  * The second launch's workgroups own output columns for all experts, so a
//    token's sum over its experts needs no atomics and has a fixed order.
//
// Measured (both launches, replayed from a graph): 16 tokens, 6 of 64 experts,
// 5120 x 1408: 192 to 201 us by the experts chosen, 5.7 TB/s of weights (in a
// kernel trace, which slows them, 122 and 78 us; one read of the weights at 6.2
// TB/s: 177 us); 5 tokens, 2 of 8, 4096 x 8192: 109 us, 5.6 TB/s; 1 token, 8 of
// 128, 2048 x 768: 14.1 us (traced 8.7 and 6.4), where each launch is
// mostly its start, the choice of the first expert and one trip to HBM.
#include "qp_device.hpp"
#include "qp_launch.hpp"

namespace qp {
namespace {

typedef __attribute__((ext_vector_type(4))) short s16x4;

constexpr int MAX_T = 16, MAX_TOPK = 16, MAX_E = 512, MAX_PAIRS = MAX_T * MAX_TOPK;
constexpr int WIN = 256;                        // K elements per window
// Past every buffer (each is below 2^31 bytes): such a load returns zero.
constexpr uint32_t OOB = 0x80000000u;
// Offset of a weight row that does not exist and size of the weights' buffers
// (an expert's matrix is a multiple of 2^14 bytes below 2^31).
constexpr uint32_t NOROW = 0x7FFFFF00u;

// A part is an expert and at most S of its tokens: an expert with more has
// several parts, which each read its weights.  An MFMA takes four operand rows:
// four tokens of x, or two of h (hi and lo).  A part has one such group (S = 4
// and 2) or two (S = 8 and 4), see launch_moe_fp8.

struct Parts {
    uint32_t n;
    uint32_t expert[MAX_PAIRS];                 // of each part, ascending
    uint32_t first[MAX_PAIRS + 1];              // its first pair (its last is before the next part's first)
};
// What the first launch leaves for the second (behind the rows of h).
struct Plan {
    Parts down;
    uint32_t token[MAX_PAIRS];                  // of each pair
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v)
{
    return __uint_as_float(dpp_u<CTRL>(__float_as_uint(v)));
}

// Both halves of a lane swap of v with itself: rows of 16 lanes 0 0 2 2 and
// 1 1 3 3 (swap16), lanes 0 .. 31 twice and 32 .. 63 twice (swap32).
__device__ __forceinline__ u32x2 swap16(uint32_t v)
{
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (u32x2){r[0], r[1]};
}
__device__ __forceinline__ u32x2 swap32(uint32_t v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (u32x2){r[0], r[1]};
}
__device__ __forceinline__ float add_halves(u32x2 h)
{
    return __uint_as_float(h[0]) + __uint_as_float(h[1]);
}

__device__ __forceinline__ uint32_t row_max_u(uint32_t v)
{
    v = max(v, dpp_u<0xB1>(v));                 // pairs, quads, eights, sixteens
    v = max(v, dpp_u<0x4E>(v));
    v = max(v, dpp_u<0x141>(v));
    return max(v, dpp_u<0x140>(v));
}
__device__ __forceinline__ uint32_t wave_max_u(uint32_t v)
{
    u32x2 h = swap16(row_max_u(v));
    h = swap32(max(h[0], h[1]));
    return max(h[0], h[1]);
}
__device__ __forceinline__ float row_sum_f(float v)
{
    v += dpp_f<0xB1>(v);
    v += dpp_f<0x4E>(v);
    v += dpp_f<0x141>(v);
    return v + dpp_f<0x140>(v);
}
__device__ __forceinline__ float wave_sum_f(float v)
{
    return add_halves(swap32(__float_as_uint(add_halves(swap16(__float_as_uint(row_sum_f(v)))))));
}
// Sum of v over the lanes up to and including this one.
__device__ __forceinline__ uint32_t wave_scan_u(uint32_t v)
{
    v += dpp_u<0x111>(v);                       // shifts by 1, 2, 4, 8 in a row of 16
    v += dpp_u<0x112>(v);
    v += dpp_u<0x114>(v);
    v += dpp_u<0x118>(v);
    // the last lane of rows 0 and 2 to rows 1 and 3, then lane 31 to the upper half
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);
    return v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, 0x00020000);
}
// (weights: nontemporal, they are read once)
__device__ __forceinline__ u32x4 load16_nt(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 2));
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
__device__ __forceinline__ float load4(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
}

// Monotone integer key of a logit; 0 only for -inf and for what is no expert.
__device__ __forceinline__ uint32_t key_of(float f)
{
    const uint32_t u = __float_as_uint(f);
    return f == -__builtin_inff() ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

struct Routing {
    Plan plan;
    Parts up;
    float weight[MAX_PAIRS];                    // p of each pair
    // scratch
    uint32_t sel_e[MAX_T][MAX_TOPK], nsel[MAX_T];
    float sel_w[MAX_T][MAX_TOPK];
    uint32_t mask[MAX_E], base[MAX_E];          // tokens of an expert; its first pair
};

// Logits past the table's end (bytes) read as zeros and take key 0: a load
// under a condition of its own would be waited for before the next is issued.
__device__ __forceinline__ uint32_t load_key(__amdgpu_buffer_rsrc_t logits, uint32_t at, bool live)
{
    const uint32_t k = key_of(load4(logits, 4 * at) + 0.0f);    // (-0 ties with +0)
    return live ? k : 0u;
}

// The topk of a single token by a wave: lane l holds experts l*EPL .. , so
// among equal keys the lowest lane, and in it the lowest slot, is the lowest
// expert.  Lane i < n holds the i-th chosen expert.
template <int EPL>
struct ChooseOne {
    uint32_t key[EPL], had[EPL], n, e, k, top_k;
    bool done;                                  // nothing left to choose

    __device__ __forceinline__ ChooseOne(__amdgpu_buffer_rsrc_t logits, uint32_t E)
        : n(0), e(0), k(0), top_k(0), done(false)
    {
        const uint32_t lane = threadIdx.x & 63;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            key[j] = had[j] = load_key(logits, lane * EPL + j, lane * EPL + j < E);
    }
    // choose until there are `want`
    __device__ __forceinline__ void until(uint32_t want)
    {
        const uint32_t lane = threadIdx.x & 63;
        while (n < want && !done) {
            uint32_t b = key[0], bj = 0;
#pragma unroll
            for (int j = 1; j < EPL; ++j) {
                bj = key[j] > b ? j : bj;
                b = max(b, key[j]);
            }
            const uint32_t m = __builtin_amdgcn_readfirstlane(wave_max_u(b));
            if (m == 0) {
                done = true;
                break;
            }
            const uint32_t who = (uint32_t)__builtin_ctzll(__ballot(b == m));
            const uint32_t j = (uint32_t)__builtin_amdgcn_readlane((int)bj, (int)who);
            top_k = n == 0 ? m : top_k;
            e = lane == n ? who * EPL + j : e;
            k = lane == n ? m : k;
#pragma unroll
            for (int q = 0; q < EPL; ++q)
                key[q] = lane * EPL + q == who * EPL + j ? 0u : key[q];
            ++n;
        }
    }
    // this lane's weight, when all are chosen
    __device__ __forceinline__ float weight(bool renorm) const
    {
        const uint32_t lane = threadIdx.x & 63;
        const float top = value_of(top_k), w = lane < n ? expf(value_of(k) - top) : 0.0f;
        float total = w;
        if (!renorm) {
            total = 0.0f;
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                total += had[j] ? expf(value_of(had[j]) - top) : 0.0f;
        }
        return w / wave_sum_f(total);
    }
};

// The topk of four tokens by a wave, one to each row of 16 lanes: lane l of
// the row holds experts l, l + 16, ..., and of equal keys the lowest expert is
// found by a second reduction.  Lane i < n (of the row) gets the row's i-th.
template <int EPL>
__device__ __forceinline__ uint32_t choose_four(__amdgpu_buffer_rsrc_t logits, uint32_t t, uint32_t T,
                                                uint32_t E, uint32_t topk, bool renorm, uint32_t &my_e,
                                                float &my_w)
{
    const uint32_t l = threadIdx.x & 15;
    uint32_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j)
        key[j] = load_key(logits, t * E + l + 16 * j, t < T && l + 16 * j < E);
    uint32_t n = 0, e = 0, k = 0, top_k = 0;
    float rest = 0.0f;
    for (uint32_t i = 0; i < topk; ++i) {
        uint32_t b = key[0], bj = 0;
#pragma unroll
        for (int j = 1; j < EPL; ++j) {
            bj = key[j] > b ? j : bj;
            b = max(b, key[j]);
        }
        const uint32_t m = row_max_u(b);
        const uint32_t won = ~row_max_u(b == m ? ~(l + 16 * bj) : 0u);
        if (i == 0) {
            top_k = m;
            if (!renorm)
#pragma unroll
                for (int j = 0; j < EPL; ++j)
                    rest += key[j] ? expf(value_of(key[j]) - value_of(m)) : 0.0f;
        }
        e = l == i ? won : e;
        k = l == i ? m : k;
        n += m != 0;                            // once nothing is left, m stays 0
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            key[j] = l + 16 * j == won ? 0u : key[j];
    }
    const float w = l < n ? expf(value_of(k) - value_of(top_k)) : 0.0f;
    my_e = e;
    my_w = w / row_sum_f(renorm ? w : rest);
    return n;
}

// One token: its experts are the parts and the pairs, in the order chosen.
// Every wave finds and writes the same, so none waits for another; how many
// there are so far is each wave's own (R.up.n and R.plan.down.n are not used).
template <int EPL>
__device__ __forceinline__ void publish(const ChooseOne<EPL> &c, Routing &R)
{
    const uint32_t lane = threadIdx.x & 63;
    if (lane < c.n) {
        R.up.expert[lane] = R.plan.down.expert[lane] = c.e;
        R.plan.token[lane] = 0;
    }
    if (lane <= c.n)
        R.up.first[lane] = R.plan.down.first[lane] = lane;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Fill R with parts of at most SU tokens for the first product and SD for the
// second (every thread of the workgroup calls this; ends with a barrier).
template <uint32_t SU, uint32_t SD>
__device__ void route(const float *__restrict__ logits, uint32_t T, uint32_t E, uint32_t topk,
                      bool renorm, Routing &R)
{
    const uint32_t tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const uint32_t mine_t = 4 * wave + (lane >> 4), l16 = lane & 15;
    for (uint32_t e = tid; e < MAX_E; e += blockDim.x)
        R.mask[e] = 0;
    __syncthreads();
    if (4 * wave < T) {
        uint32_t e, n;
        float w;
        const __amdgpu_buffer_rsrc_t lg = rsrc(logits, T * E * 4);
        n = E <= 64    ? choose_four<4>(lg, mine_t, T, E, topk, renorm, e, w)
            : E <= 128 ? choose_four<8>(lg, mine_t, T, E, topk, renorm, e, w)
            : E <= 256 ? choose_four<16>(lg, mine_t, T, E, topk, renorm, e, w)
                       : choose_four<32>(lg, mine_t, T, E, topk, renorm, e, w);
        if (mine_t < T) {
            if (l16 < n) {
                R.sel_e[mine_t][l16] = e;
                R.sel_w[mine_t][l16] = w;
                atomicOr(&R.mask[e], 1u << mine_t); // an OR: order does not matter
            }
            if (l16 == 0)
                R.nsel[mine_t] = n;
        }
    }
    __syncthreads();
    if (wave < 2) {
        // wave 0 the parts of the first product, wave 1 of the second.  Lane l:
        // experts 8l .. 8l+7; parts (high half) and pairs (low half) before it
        // by an inclusive scan over the lanes
        Parts &P = wave ? R.plan.down : R.up;
        const uint32_t S = wave ? SD : SU;
        uint32_t mk[8], mine = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            mk[j] = R.mask[8 * lane + j];
            const uint32_t c = (uint32_t)__popc(mk[j]);
            mine += ((c + S - 1) / S << 16) + c;
        }
        const uint32_t inc = wave_scan_u(mine);
        uint32_t at = inc - mine;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            R.base[8 * lane + j] = at & 0xFFFFu;    // (both waves write the same)
            for (int left = __popc(mk[j]); left > 0; left -= S) {
                P.expert[at >> 16] = 8 * lane + j;
                P.first[at >> 16] = at & 0xFFFFu;
                at += 0x10000u + min((uint32_t)left, S);
            }
        }
        if (lane == 63) {
            P.n = inc >> 16;
            P.first[inc >> 16] = inc & 0xFFFFu;
        }
    }
    __syncthreads();
    for (uint32_t i = tid; i < T * MAX_TOPK; i += blockDim.x) {
        const uint32_t t = i / MAX_TOPK, s = i % MAX_TOPK;
        if (s < R.nsel[t]) {
            const uint32_t e = R.sel_e[t][s];
            const uint32_t pair = R.base[e] + (uint32_t)__popc(R.mask[e] & ((1u << t) - 1u));
            R.plan.token[pair] = t;
            R.weight[pair] = R.sel_w[t][s];
        }
    }
    __syncthreads();
}

// Four E4M3 codes as BF16, exactly.
__device__ __forceinline__ s16x4 fp8x4_bf16(uint32_t w)
{
    const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, false);
    const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, true);
    return __builtin_bit_cast(s16x4, (u32x2){__builtin_bit_cast(uint32_t, lo),
                                             __builtin_bit_cast(uint32_t, hi)});
}
__device__ __forceinline__ s16x4 half_of(const u32x4 *x, int i)
{
    const u32x4 v = x[i / 2];
    return __builtin_bit_cast(s16x4, i % 2 ? (u32x2){v[2], v[3]} : (u32x2){v[0], v[1]});
}

// p += w (16 codes of a lane) times x (16 BF16 of a lane), over the window.
__device__ __forceinline__ f32x4 window(const s16x4 *w, const u32x4 *x, f32x4 p)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        p = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(half_of(x, i), w[i], p, 0, 0, 0);
    return p;
}

// v of lane l ^ 4, by two moves that write alternate quads.
__device__ __forceinline__ float xor4(float v)
{
    const int u = __float_as_int(v);
    const int down = __builtin_amdgcn_update_dpp(0, u, 0x104, 0xF, 0x5, false);
    return __int_as_float(__builtin_amdgcn_update_dpp(down, u, 0x114, 0xF, 0xA, false));
}
// v of lane l ^ 8: a rotation by half a row.
__device__ __forceinline__ float xor8(float v) { return dpp_f<0x128>(v); }

// Sums of N values (a power of two) over the 16 K slices, lanes of equal l % 4.
// A lane ends with the sums of values first .. first + max(N / 16, 1) - 1 in
// v[0] .. (first is returned), which costs 2 to 3 instructions a pair instead
// of a whole butterfly for each; N < 16: lanes share them, and `owner` is true
// in one of those.
template <int N>
__device__ __forceinline__ uint32_t sum_slices(float *v, bool &owner)
{
    const uint32_t lane = threadIdx.x & 63;
    constexpr int N1 = N > 1 ? N / 2 : 1, N2 = N1 > 1 ? N1 / 2 : 1, N3 = N2 > 1 ? N2 / 2 : 1;
    const bool b5 = lane & 32, b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
#pragma unroll
    for (int i = 0; i < N1; ++i) {              // (halves exchanged: the lower lanes' sum, the upper lanes')
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[N > 1 ? i + N1 : 0]),
                                                        false, false);
        v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
#pragma unroll
    for (int i = 0; i < N2; ++i) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[N1 > 1 ? i + N2 : 0]),
                                                        false, false);
        v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
#pragma unroll
    for (int i = 0; i < N3; ++i) {
        const float keep = N2 > 1 && b3 ? v[N2 > 1 ? i + N3 : 0] : v[i],
                    give = N2 > 1 && !b3 ? v[N2 > 1 ? i + N3 : 0] : v[i];
        v[i] = keep + xor8(give);
    }
    constexpr int N4 = N3 > 1 ? N3 / 2 : 1;
#pragma unroll
    for (int i = 0; i < N4; ++i) {
        const float keep = N3 > 1 && b2 ? v[N3 > 1 ? i + N4 : 0] : v[i],
                    give = N3 > 1 && !b2 ? v[N3 > 1 ? i + N4 : 0] : v[i];
        v[i] = keep + xor4(give);
    }
    owner = (N > 1 || !b5) && (N1 > 1 || !b4) && (N2 > 1 || !b3) && (N3 > 1 || !b2);
    return (N > 1 && b5 ? N1 : 0) + (N1 > 1 && b4 ? N2 : 0) + (N2 > 1 && b3 ? N3 : 0) + (N3 > 1 && b2 ? N4 : 0);
}

struct MoeArgs {
    const uint16_t *x;
    const float *logits;
    const uint8_t *w13, *w2;
    const float *s13, *s2;
    uint16_t *h;                                // [2 pairs, I]: hi and lo of p * h
    Plan *plan;
    uint16_t *out;
    uint32_t T, E, topk, H, I, renorm;
};

// One wave's work: a run of units, each a few weight rows of one expert times
// the operand rows of one part, over windows w0, w0 + WS, ... < w1 (past the K
// range: zeros).
template <int NG>
struct Unit {
    const uint8_t *w;                           // the weight rows' common base
    uint32_t s0, s1;                            // byte offsets of their rows in the scale grid
    uint32_t x[NG];                             // per lane and group: operand row l % 4 at chunk l / 4
    uint32_t w0, w1;
};

// Walk the units u0, u0 + step, ... < n with D windows in flight, across the
// units' ends: RW groups of 4 weight rows (lane l's row l % 4, chunk l / 4 at
// base + ow[g]); unit(u) describes one; sink(u, acc) takes its sums
// acc[g][n][r]: the lane's K slice of its row of weight group g with row r < NR
// of operand group n < NG.
// Groups below split scale by the grid row s0, the others by s1.  started() runs
// once the first D windows are on their way and may change n above those.
template <int RW, int NG, int NR, int D, int WS, class Started, class GetUnit, class Sink>
__device__ __forceinline__ void stream(__amdgpu_buffer_rsrc_t rs, __amdgpu_buffer_rsrc_t rx,
                                       const uint32_t (&ow)[RW], uint32_t split, uint32_t kn,
                                       uint32_t u0, const uint32_t &n, uint32_t step, Started started, GetUnit unit,
                                       Sink sink)
{
    const uint32_t lane = threadIdx.x & 63, c16 = lane >> 2;
    struct Stage {
        u32x4 w[RW], x[NG][2];
        float s0, s1;
    } st[D];
    // the next window to fetch: window fw of unit fu, described by f
    uint32_t fu = u0, fw = 0;
    Unit<NG> f = {};
    if (fu < n) {
        f = unit(fu);
        fw = f.w0;
    }
    auto fetch = [&](Stage &s) {
        // What a lane may not load is moved past the buffers by an addend that
        // the compiler cannot see through: it would turn a select of offsets
        // into branches around the loads, and the wave would then wait for
        // every load in flight.  (No more units: w1 == 0.)
        const bool ok = fw < f.w1 && fw * WIN + 16 * c16 < kn;
        uint32_t dw = ok ? fw * WIN : OOB, dx = ok ? 2 * fw * WIN : OOB;
        uint32_t ds = ok ? 8 * fw + 4 * (lane >> 5) : OOB;
        asm volatile("" : "+v"(dw), "+v"(dx), "+v"(ds));
        const __amdgpu_buffer_rsrc_t rw = rsrc(f.w, NOROW);
#pragma unroll
        for (int g = 0; g < RW; ++g)
            s.w[g] = load16_nt(rw, ow[g] + dw);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            s.x[n][0] = load16(rx, f.x[n] + dx);
            s.x[n][1] = load16(rx, f.x[n] + dx + 16);
        }
        s.s0 = load4(rs, f.s0 + ds);
        s.s1 = load4(rs, f.s1 + ds);
        fw += WS;
        if (fw >= f.w1 && fu < n) {
            fu += step;
            f.w1 = 0;
            if (fu < n) {
                f = unit(fu);
                fw = f.w0;
            }
        }
    };
    f32x4 acc[RW][NG] = {};
    uint32_t uu = u0, left = 0;
    if (uu < n) {
        const Unit<NG> u = unit(uu);
        left = (u.w1 - u.w0 + WS - 1) / WS;
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
        fetch(st[d]);
    started();
    while (uu < n) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const Stage &s = st[d];
#pragma unroll
            for (int g = 0; g < RW; ++g) {
                s16x4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = fp8x4_bf16(s.w[g][i]);
                const float sg = (uint32_t)g < split ? s.s0 : s.s1;
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    const f32x4 p = window(v, s.x[n], (f32x4){0, 0, 0, 0});
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        float a = __builtin_fmaf(p[r], sg, acc[g][n][r]);
                        // pinned here: sunk past the refill, it would make the
                        // compiler copy (and so wait for) the registers being loaded
                        asm volatile("" : "+v"(a));
                        acc[g][n][r] = a;
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            fetch(st[d]);
            __builtin_amdgcn_sched_barrier(0);
            if (--left == 0 && uu < n) {
                sink(uu, acc);
#pragma unroll
                for (int g = 0; g < RW; ++g)
#pragma unroll
                    for (int n = 0; n < NG; ++n)
                        acc[g][n] = (f32x4){0, 0, 0, 0};
                uu += step;
                if (uu < n) {
                    const Unit<NG> u = unit(uu);
                    left = (u.w1 - u.w0 + WS - 1) / WS;
                }
            }
        }
    }
}

// First launch: route, then units of RG * (4 + 4) gate and up rows of a part
// (NTOK tokens at most; in the second launch a part has NTOK / 2).
// A workgroup's four waves share a unit, wave w taking windows w, w + 4, ...,
// and join their sums through LDS in wave order: the rows of a unit are one
// contiguous block (two, gate and up) that is read at one time, which HBM
// serves better than as many separate walks along K.
//
// A single token's experts are known one after another, the last some 1.5 us
// after the first, so a workgroup starts on its unit as soon as that unit's
// expert is chosen and ends the choice under its loads (EPL: of ChooseOne; 0
// for more tokens).
template <int NTOK, int RG, int EPL>
__global__ __launch_bounds__(256) void k_moe_gate_up(MoeArgs A)
{
    __shared__ Routing R;
    __shared__ float part_sum[2][4][2 * RG][4 * NTOK];
    constexpr int D = 2, NG = (NTOK + 3) / 4;   // windows in flight, operand groups
    const uint32_t groups = A.I / (4 * RG);
    uint32_t units = 0;
    ChooseOne<EPL ? EPL : 1> one(rsrc(A.logits, A.E * 4), EPL ? A.E : 0);
    if (EPL) {
        // the experts of this workgroup's first D + 1 units
        uint32_t last = blockIdx.x;
        for (int d = 0; d < D; ++d)
            last += last + gridDim.x < A.topk * groups ? gridDim.x : 0;
        one.until(min(last / groups + 1, A.topk));
        publish(one, R);
    } else {
        route<NTOK, NTOK / 2>(A.logits, A.T, A.E, A.topk, A.renorm != 0, R);
    }
    units = (EPL ? one.n : R.up.n) * groups;
    auto started = [&]() {
        if (EPL) {
            one.until(A.topk);
            publish(one, R);
            const float w = one.weight(A.renorm != 0);
            if ((threadIdx.x & 63) < one.n)
                R.weight[threadIdx.x & 63] = w;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            units = one.n * groups;
        }
        if (blockIdx.x == 0) {
            const uint32_t n = EPL ? one.n : R.plan.down.n, pairs = R.plan.down.first[n];
            for (uint32_t i = threadIdx.x; i <= n; i += blockDim.x)
                A.plan->down.first[i] = R.plan.down.first[i];
            for (uint32_t i = threadIdx.x; i < n; i += blockDim.x)
                A.plan->down.expert[i] = R.plan.down.expert[i];
            for (uint32_t i = threadIdx.x; i < pairs; i += blockDim.x)
                A.plan->token[i] = R.plan.token[i];
            if (threadIdx.x == 0)
                A.plan->down.n = n;
        }
    };
    const uint32_t lane = threadIdx.x & 63, r4 = lane & 3, c16 = lane >> 2;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t HB = A.H / 128, IB = A.I / 128;
    const uint32_t nwq = ((A.H + WIN - 1) / WIN + 3) / 4;   // windows of each wave
    uint32_t ow[2 * RG];
#pragma unroll
    for (int q = 0; q < RG; ++q) {
        ow[q] = (4 * q + r4) * A.H + 16 * c16;
        ow[RG + q] = ow[q] + A.I * A.H;
    }
    // unit u: rows 4 RG (u % groups) of part u / groups
    auto part = [&](uint32_t u, uint32_t &e, uint32_t &first, uint32_t &cnt) {
        const uint32_t p = u / groups;
        e = __builtin_amdgcn_readfirstlane(R.up.expert[p]);
        first = __builtin_amdgcn_readfirstlane(R.up.first[p]);
        cnt = __builtin_amdgcn_readfirstlane(R.up.first[p + 1]) - first;
        return u % groups * (4 * RG);
    };
    auto unit = [&](uint32_t u) {
        uint32_t e, first, cnt;
        const uint32_t row = part(u, e, first, cnt);
        Unit<NG> d;
        d.w = A.w13 + ((size_t)e * 2 * A.I + row) * A.H;
        d.s0 = (e * 2 * IB + row / 128) * HB * 4;
        d.s1 = d.s0 + IB * HB * 4;
#pragma unroll
        for (int n = 0; n < NG; ++n)
            d.x[n] = n && 4u * n >= cnt ? NOROW : R.plan.token[first + min(4 * n + r4, cnt - 1)] * A.H * 2 + 32 * c16;
        d.w0 = wave;
        d.w1 = wave + 4 * nwq;
        return d;
    };
    uint32_t buf = 0;
    auto sink = [&](uint32_t u, const f32x4 (&acc)[2 * RG][NG]) {
        uint32_t e, first, cnt;
        const uint32_t row = part(u, e, first, cnt);
        // value NTOK q + t, of weight row l % 4: in its place as lane 4 t + l % 4 below
        float v[2 * RG * NTOK];
#pragma unroll
        for (int i = 0; i < 2 * RG * NTOK; ++i)
            v[i] = acc[i / NTOK][i % NTOK / 4][i % 4 * (NTOK > 1)];
        bool owner;
        const uint32_t first_v = sum_slices<2 * RG * NTOK>(v, owner);
        if (owner)
#pragma unroll
            for (int i = 0; i < (2 * RG * NTOK + 15) / 16; ++i)
                (&part_sum[buf][wave][0][0])[4 * (first_v + i) + r4] = v[i];
        // (the next unit takes the other buffer, so one barrier is enough)
        __syncthreads();
#pragma unroll
        for (int q = 0; q < RG; ++q) {
            if (c16 >= cnt || (uint32_t)(q % 4) != wave)
                continue;
            float vg = 0.0f, vu = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                vg += part_sum[buf][w][q][lane];
                vu += part_sum[buf][w][RG + q][lane];
            }
            const float h = vg / (1.0f + expf(-vg)) * vu * R.weight[first + c16];
            const uint32_t hi = f32_to_bf16(h);
            const size_t at = (size_t)(2 * (first + c16)) * A.I + row + 4 * q + r4;
            A.h[at] = (uint16_t)hi;
            A.h[at + A.I] = (uint16_t)f32_to_bf16(h - bf16_lo(hi));
        }
        buf ^= 1;
    };
    stream<2 * RG, NG, NTOK == 1 ? 1 : 4, D, 4>(rsrc(A.s13, A.E * 2 * IB * HB * 4), rsrc(A.x, A.T * A.H * 2), ow, RG, A.H,
                               blockIdx.x, units, gridDim.x, started, unit, sink);
}

// Second launch: 4 RG output columns per workgroup; its waves take the parts'
// windows in turn, a few at a time, so that all workgroups move through the
// experts together, and their sums are joined in wave order.
constexpr int NWV = 8;
constexpr int pow2(int n) { return n <= 1 ? 1 : 2 * pow2((n + 1) / 2); }
template <int NTOK, int RG>
__global__ __launch_bounds__(64 * NWV) void k_moe_down(MoeArgs A)
{
    __shared__ Plan P;
    __shared__ float sums[NWV][NTOK == 1 ? 1 : MAX_T][4 * RG];
    const uint32_t tid = threadIdx.x;
    // (read whole, up to the most there can be: its length is then no wait of
    // its own, and what lies past it is not used)
    const uint32_t n = A.plan->down.n, pairs = A.T * A.topk;
    for (uint32_t i = tid; i <= pairs; i += blockDim.x)
        P.down.first[i] = A.plan->down.first[i];
    for (uint32_t i = tid; i < pairs; i += blockDim.x) {
        P.down.expert[i] = A.plan->down.expert[i];
        P.token[i] = A.plan->token[i];
    }
    for (uint32_t i = tid; i < sizeof(sums) / sizeof(float); i += blockDim.x)
        (&sums[0][0][0])[i] = 0.0f;
    __syncthreads();
    const uint32_t lane = tid & 63, r4 = lane & 3, c16 = lane >> 2;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t HB = A.H / 128, IB = A.I / 128, nw = (A.I + WIN - 1) / WIN, c0 = blockIdx.x * 4 * RG;
    // windows to a unit: six, or fewer where that would leave waves without one
    const uint32_t per = min(nw, max(1u, min(6u, n * nw / NWV)));
    const uint32_t live = (nw + per - 1) / per;             // pieces that hold windows
    uint32_t ow[RG];
#pragma unroll
    for (int q = 0; q < RG; ++q)
        ow[q] = c0 + 4 * q < A.H ? (4 * q + r4) * A.I + 16 * c16 : NOROW;
    constexpr int NG = (2 * NTOK + 7) / 8;      // operand groups: two rows for each of NTOK / 2 tokens
    auto unit = [&](uint32_t u) {
        const uint32_t p = u / live;
        const uint32_t e = __builtin_amdgcn_readfirstlane(P.down.expert[p]);
        const uint32_t first = __builtin_amdgcn_readfirstlane(P.down.first[p]);
        const uint32_t cnt = __builtin_amdgcn_readfirstlane(P.down.first[p + 1]) - first;
        Unit<NG> d;
        d.w = A.w2 + ((size_t)e * A.H + c0) * A.I;
        d.s0 = (e * HB + c0 / 128) * IB * 4;
        d.s1 = d.s0 + (c0 / 128 + 1 < HB ? IB * 4 : 0);
#pragma unroll
        for (int n = 0; n < NG; ++n)
            d.x[n] = n && 2u * n >= cnt ? NOROW : (2 * first + min(4 * n + r4, 2 * cnt - 1)) * A.I * 2 + 32 * c16;
        d.w0 = u % live * per;
        d.w1 = min(d.w0 + per, nw);
        return d;
    };
    auto sink = [&](uint32_t u, const f32x4 (&acc)[RG][NG]) {
        const uint32_t p = u / live;
        const uint32_t first = __builtin_amdgcn_readfirstlane(P.down.first[p]);
        const uint32_t cnt = __builtin_amdgcn_readfirstlane(P.down.first[p + 1]) - first;
        // other lanes of this wave may have added to the same sums before
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        // value PER q + i: token i of the part, weight row 4 q + l % 4
        constexpr int PER = NTOK == 1 ? 1 : NTOK / 2, NV = pow2(RG * PER);
        float v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int q = i / PER, s = i % PER;
            v[i] = q < RG ? acc[q < RG ? q : 0][s / 2][s % 2 * 2] + acc[q < RG ? q : 0][s / 2][s % 2 * 2 + 1] : 0.0f;
        }
        bool owner;
        const uint32_t first_v = sum_slices<NV>(v, owner);
#pragma unroll
        for (int i = 0; i < (NV + 15) / 16; ++i) {
            const uint32_t q = (first_v + i) / PER, s = (first_v + i) % PER;
            if (owner && q < RG && s < cnt)
                sums[wave][P.token[first + s]][4 * q + r4] += v[i];  // only this wave's, one lane each
        }
    };
    stream<RG, NG, NTOK == 1 ? 2 : 4, RG * NG <= 5 ? 3 : 2, 1>(
        rsrc(A.s2, A.E * HB * IB * 4), rsrc(A.h, A.T * A.topk * A.I * 4), ow, (128 - c0 % 128) / 4, A.I, wave,
        n * live, NWV, [] {}, unit, sink);
    __syncthreads();
    for (uint32_t i = tid; i < A.T * 4 * RG; i += blockDim.x) {
        const uint32_t t = i / (4 * RG), c = i % (4 * RG);
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < NWV; ++w)
            v += sums[w][t][c];
        if (c0 + c < A.H)
            A.out[(size_t)t * A.H + c0 + c] = (uint16_t)f32_to_bf16(v);
    }
}

template <int NTOK, int RG>
void launch_down(const MoeArgs &A, hipStream_t st)
{
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_moe_down<NTOK, RG>), dim3((A.H + 4 * RG - 1) / (4 * RG)), dim3(64 * NWV),
                       0, st, A);
}

template <int NTOK>
hipError_t launch_moe(const MoeArgs &A, hipStream_t st)
{
    const uint32_t cus = cu_count() ? cu_count() : 256;
    // a workgroup for every unit that may come about, at most as many as fit
    // a CU at once (by registers: four, with parts of eight tokens three)
    constexpr int RGU = 2;
    const uint32_t most = (NTOK == 8 ? 3 : 4) * cus;
    const uint64_t pairs = A.T * A.topk, parts = A.E + pairs / NTOK < pairs ? A.E + pairs / NTOK : pairs;
    const uint64_t units = parts * (A.I / (4 * RGU));
    const dim3 grid(units < most ? (uint32_t)units : most);
    if constexpr (NTOK == 1) {
        if (A.E <= 64)
            hipLaunchKernelGGL(HIP_KERNEL_NAME(k_moe_gate_up<1, RGU, 1>), grid, dim3(256), 0, st, A);
        else if (A.E <= 128)
            hipLaunchKernelGGL(HIP_KERNEL_NAME(k_moe_gate_up<1, RGU, 2>), grid, dim3(256), 0, st, A);
        else if (A.E <= 256)
            hipLaunchKernelGGL(HIP_KERNEL_NAME(k_moe_gate_up<1, RGU, 4>), grid, dim3(256), 0, st, A);
        else
            hipLaunchKernelGGL(HIP_KERNEL_NAME(k_moe_gate_up<1, RGU, 8>), grid, dim3(256), 0, st, A);
    } else {
        hipLaunchKernelGGL(HIP_KERNEL_NAME(k_moe_gate_up<NTOK, RGU, 0>), grid, dim3(256), 0, st, A);
    }
    count_launch();
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return err;
    // The columns dealt evenly over the CUs, at most 32 to a workgroup: with
    // 16 columns each, 5120 columns took 120 us where 20 take 76 (the CUs with
    // two workgroups decide).
    const uint32_t rounds = (A.H + 32 * cus - 1) / (32 * cus);
    switch ((A.H + 4 * cus * rounds - 1) / (4 * cus * rounds)) {
    case 1: launch_down<NTOK, 1>(A, st); break;
    case 2: launch_down<NTOK, 2>(A, st); break;
    case 3: launch_down<NTOK, 3>(A, st); break;
    case 4: launch_down<NTOK, 4>(A, st); break;
    case 5: launch_down<NTOK, 5>(A, st); break;
    case 6: launch_down<NTOK, 6>(A, st); break;
    case 7: launch_down<NTOK, 7>(A, st); break;
    default: launch_down<NTOK, 8>(A, st); break;
    }
    count_launch();
    return hipGetLastError();
}

inline uint64_t planes_bytes(uint64_t T, uint64_t topk, uint64_t I) { return 4 * T * topk * I; }

} // namespace

// I is a multiple of 128, so the plan behind the planes is 16-byte aligned.
uint64_t moe_fp8_workspace(uint32_t T, uint32_t topk, uint32_t I)
{
    return planes_bytes(T, topk, I) + sizeof(Plan);
}

hipError_t launch_moe_fp8(const uint16_t *x, const float *logits, const uint8_t *w13, const float *s13,
                          const uint8_t *w2, const float *s2, void *work, uint16_t *out, uint32_t T,
                          uint32_t E, uint32_t topk, uint32_t H, uint32_t I, bool renorm, hipStream_t st)
{
    uint8_t *const wk = (uint8_t *)work;
    const MoeArgs A = {x, logits, w13, w2, s13, s2, (uint16_t *)wk, (Plan *)(wk + planes_bytes(T, topk, I)),
                       out, T, E, topk, H, I, renorm};
    if (T == 1)
        return launch_moe<1>(A, st);
    // Parts of eight tokens from a mean of three tokens an expert on: the second
    // group of operand rows costs loads and MFMAs whether it holds tokens or
    // not, a second part the weights again.  16 tokens of 8x2, 4096x2048 (mean
    // 4): 56 us against 65; 8 of 16x6, 5120x1024 (3): 57.7 against 62.6; 16 of
    // 48x8, 2048x768 (2.7): 63.0 against 60.4; 16 of 64x6, 5120x1408 (1.5): 196
    // against 192.
    if (T * topk >= 3 * E)
        return launch_moe<8>(A, st);
    return launch_moe<4>(A, st);
}

} // namespace qp
