// attn_decode.hip -- attention of few rows a sequence (decode, verify batches),
// which reads the cache once and has little else to do.
//
// A wave takes 32 keys at a time and needs neither LDS nor barriers for them:
//   S^T [key, row] = K Q^T   two 16x16x32 MFMAs (16 keys each) for every 32 of d;
//                            K goes from memory to the operand's registers, 64
//                            bytes of 16 rows a load
//   P^T = exp2(S^T - m)      a lane holds 8 scores of ONE row, so maximum and sum
//                            are its own; the maximum is shared with the row's
//                            three other lanes only when it grows by more than 2^8
//   O^T [d, row] += V^T P^T  (twice with a BF16 cache: P rounded, and the remainder)
//                            P^T is already in the layout of the operand: key slot
//                            (lane/16, i) stands for key 4 (lane/16) + i of the
//                            first 16 (i < 4) or the second; V is loaded in whole
//                            rows, 4 keys a load, and turned with byte permutes
// so that a wave's only traffic is the cache itself: while one 32 keys are
// worked on, the next are on their way (K is fetched again as soon as its
// products are issued, V as soon as its own are).  The four waves of a workgroup
// take every fourth 32 keys and join through LDS at a unit's end.
//
// Bound by HBM in BF16 (a token each of 48 sequences over 1200 to 12000 positions, 8 kv
// heads of 128, 240 us, 5.6 TB/s; 16 sequences of 9001, 4 kv heads, 32 rows: the kernel
// alone 57 us, 5.3 TB/s) and in E4M3 with up to 16 rows (the same sequences: 30 us, 5.2
// TB/s).  With more the decoding and turning of the codes, which every block of 32 rows
// does again, costs more than their bytes (50 rows: 49 us alone, 3.2 TB/s; with a third
// tile on its way a quarter slower).  The join is 4 to 6 us more.  Over one short
// sequence (700 positions: 10.5 us with the join) it is a chain of trips to memory:
// lengths, pages, keys, parts.
#include "attn_common.hpp"
#include "qp_launch.hpp"

namespace qp {
namespace attn {
namespace {

constexpr uint32_t WAVES = 4, WG = 64 * WAVES;
constexpr uint32_t STEP = 32;              // keys of a wave's step
constexpr uint32_t TILE = STEP * WAVES;    // keys of a workgroup's step, the unit of the shares

__device__ __forceinline__ uint32_t tiles_of(const Seq &q)
{
    if (q.n == 0)
        return 0;
    const uint32_t from = q.first / TILE, to = (q.len + TILE - 1) / TILE;
    return max(to - from, 1u);             // rows that see nothing are still written
}

// W dwords.
template <int W>
__device__ __forceinline__ void load_dwords(__amdgpu_buffer_rsrc_t p, uint32_t at, uint32_t *w)
{
    if constexpr (W == 1) {
        w[0] = __builtin_amdgcn_raw_buffer_load_b32(p, at, 0, 0);
    } else if constexpr (W == 2) {
        const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(p, at, 0, 0));
        w[0] = v[0];
        w[1] = v[1];
    } else {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(p, at + 16 * i, 0, 0));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[4 * i + j] = v[j];
        }
    }
}

// DP: d rounded up to 64, 128 or 256 (what lies past d is zeros of Q and K; of V it is
// read from the head's start and not stored); NQ: 16s of rows of a wave; blocks (1, 2
// or 4): of so many rows a workgroup has, whose waves then go through the same keys
// at the same time, so that a block finds them in the L1 where another has loaded
// them.
template <int DP, int NQ, bool FP8>
__global__ __launch_bounds__(WG, DP <= 128 ? 2 : 1) void k_attn_decode(AttnArgs a, Parts parts, uint32_t max_shares, uint32_t blocks)
{
    constexpr int ROWS = 16 * NQ;
    constexpr int KS = DP / 32;            // MFMAs over d
    constexpr int KL = FP8 ? KS / 2 : KS;  // loads of K over d
    constexpr int ROWB = FP8 ? 1 : 2;      // bytes of an element
    constexpr int EPL = DP / 16;           // elements of V of a lane and key
    constexpr int VW = EPL * ROWB / 4;     // the same in dwords
    constexpr int LD = DP + 4;             // LDS row, so that 16 rows spread over the banks
    __shared__ float o_lds[WAVES][ROWS][LD];
    __shared__ f32x2 ml_lds[WAVES][ROWS];
    __shared__ uint16_t odd_bits[WAVES][STEP][16];      // which of a lane's elements of V are NaN or infinite
    __shared__ uint32_t scan[WAVES];
    __shared__ uint32_t found[2];

    const uint32_t tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const uint32_t col = lane % 16, quad = lane / 16;
    const uint32_t d = a.cache.d, kv = a.cache.heads, group = a.q_heads / kv, pl = a.cache.page_log2;
    const uint32_t hop = STEP * (WAVES / blocks);      // from a wave's step to its next

    // ---- the share: tiles of all sequences in one line, a sequence's heads one after the other
    auto wave_scan = [&](uint32_t v) {                  // inclusive
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const uint32_t up = __shfl_up(v, off, 64);
            v += lane >= (uint32_t)off ? up : 0;
        }
        return v;
    };
    uint32_t sum = 0, mine = 0;
    for (uint32_t s = tid; s < a.seqs; s += WG) {
        mine = tiles_of(read_seq(a, s));
        sum += mine;
    }
    const uint32_t incl = wave_scan(sum);
    if (lane == 63)
        scan[wave] = incl;
    __syncthreads();
    uint64_t total = 0, ahead = 0;
    for (uint32_t w = 0; w < WAVES; ++w) {
        ahead += w < wave ? scan[w] : 0;
        total += scan[w];
    }
    total = uniform(total * kv);
    const uint64_t shares = min((uint64_t)max_shares, total);
    const uint32_t w = blockIdx.x;
    if (w >= shares) {
        if (tid == 0)
            parts.begun[w] = {0, -1, 0, 0, 0, 0, {0, 0}};
        return;
    }
    uint64_t x = uniform(w * total / shares);
    const uint64_t share_end = uniform((w + 1) * total / shares);
    // the sequence that holds tile x, and the first tile of it
    uint32_t seq = 0;
    uint64_t seq_tile = 0;
    if (a.seqs <= WG) {
        const uint64_t to = (ahead + incl) * kv, from = to - (uint64_t)mine * kv;
        if (tid < a.seqs && x >= from && x < to) {
            found[0] = tid;
            found[1] = (uint32_t)(ahead + incl - mine);
        }
        __syncthreads();
        seq = found[0];
        seq_tile = (uint64_t)found[1] * kv;
    } else {
        uint64_t base = 0;
        for (uint32_t s0 = 0; s0 < a.seqs; s0 += WG) {
            __syncthreads();
            const uint32_t t = s0 + tid < a.seqs ? tiles_of(read_seq(a, s0 + tid)) : 0;
            const uint32_t in = wave_scan(t);
            if (lane == 63)
                scan[wave] = in;
            if (tid == 0)
                found[0] = ~0u;
            __syncthreads();
            uint64_t before = base;
            for (uint32_t v = 0; v < WAVES; ++v) {
                before += v < wave ? scan[v] : 0;
                base += scan[v];
            }
            const uint64_t to = (before + in) * kv, from = to - (uint64_t)t * kv;
            if (x >= from && x < to) {
                found[0] = s0 + tid;
                found[1] = (uint32_t)(before + in - t);
            }
            __syncthreads();
            if (found[0] != ~0u)
                break;
        }
        seq = found[0];
        seq_tile = (uint64_t)found[1] * kv;
    }
    seq = min(uniform(seq), a.seqs - 1);
    seq_tile = uniform(seq_tile);

    bool goes_on = false;
    while (x < share_end) {
        if (x < seq_tile)
            break;                         // not reached unless the lengths change under the call
        const Seq q = read_seq_uniform(a, seq);
        const uint32_t tiles = tiles_of(q);
        if (tiles == 0 || x >= seq_tile + (uint64_t)tiles * kv) {
            seq_tile += (uint64_t)tiles * kv;
            if (++seq == a.seqs)
                break;                     // nor this
            continue;
        }
        const uint32_t head = uniform((uint32_t)((x - seq_tile) / tiles));
        const uint64_t unit = seq_tile + (uint64_t)head * tiles;
        const uint32_t off = (uint32_t)(x - unit);
        const uint32_t count = (uint32_t)min((uint64_t)(tiles - off), share_end - x);
        // waves w, w + blocks, ... have the rows of block w % blocks
        const uint32_t row0 = wave % blocks * ROWS, all_rows = q.n * group;
        const int rows = (int)min(all_rows - min(row0, all_rows), (uint32_t)ROWS);

        // ---- the unit's rows
        bf16x8 qf[NQ][KS];
        int pos[NQ];
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
            const uint32_t r = row0 + col + 16 * nq, tok = r / group;
            pos[nq] = q.len - q.n + (int)tok;
            const uint16_t *src = a.q + ((size_t)(q.token + tok) * a.q_heads + head * group + (r - tok * group)) * d;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                // what the lane's 16 bytes of K hold: 8 of every 32 of d, or (E4M3) 16 of every 64
                const uint32_t e = FP8 ? 64 * (ks / 2) + 16 * quad + 8 * (ks % 2) : 32 * ks + 8 * quad;
                u32x4 v = {0, 0, 0, 0};
                if ((int)(col + 16 * nq) < rows && e < d)
                    v = *(const u32x4 *)(src + e);
                qf[nq][ks] = __builtin_bit_cast(bf16x8, v);
            }
        }
        const float scale = a.scale * LOG2E;
        const uint32_t key_from = (q.first / TILE + off) * TILE, key_to = min(key_from + count * TILE, (uint32_t)q.len);
        const int last_pos = q.len - q.n + (int)((row0 + max(rows, 1) - 1) / group);
        const int all_from = a.window ? last_pos + 1 - (int64_t)a.window : 0;              // from here every row sees ...
        const int all_to = q.len - q.n + (int)(row0 / group) + 1;                          // ... up to here (exclusive)
        const int32_t *table = a.table + (size_t)seq * a.width;
        const uint32_t mask = (1u << pl) - 1;

        float m[NQ], base[NQ], l[NQ];
        f32x4 acc[NQ][EPL];
        uint32_t nans[NQ][2];              // bit 16 (i % 2) + j of i / 2: the row's d = EPL (4 quad + i) + j has met NaN or an infinity
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
            m[nq] = -INFINITY;
            base[nq] = l[nq] = 0.0f;
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                acc[nq][j] = (f32x4){0, 0, 0, 0};
            nans[nq][0] = nans[nq][1] = 0;
        }

        // a lane's places in 16 rows of K and of V, in bytes
        uint32_t k_off[KL], v_off[4];
#pragma unroll
        for (int ks = 0; ks < KL; ++ks) {
            const uint32_t e = FP8 ? 64 * ks + 16 * quad : 32 * ks + 8 * quad;
            k_off[ks] = e < d ? (col * d + e) * ROWB : BEYOND;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v_off[j] = ((4 * quad + j) * d + (EPL * col < d ? EPL * col : 0)) * ROWB;

        u32x4 kr[2][KL];
        uint32_t vr[8][VW];
        f32x4 ksc[2], vsc[2];
        // Where the keys of 32 of the wave's steps lie: lane i's are 16 of step i / 2.  In
        // bytes of K (and of V), for E4M3 also of the scales; and which are holes.
        uint32_t step = 0, hole = 0, page_next = 0, at_lo = 0, at_hi = 0, scale_lo = 0, scale_hi = 0;
        uint64_t missing = 0;
        const uint32_t row_bytes = d * ROWB;
        auto look = [&](uint32_t key) {
            const uint32_t k = key + lane / 2 * hop + lane % 2 * 16;
            page_next = k < key_to ? (uint32_t)table[k >> pl] : ~0u;
        };
        // the places of the step at `key`, and their loads; past the end, as of holes,
        // nothing is fetched
        auto places = [&](uint32_t key) {
            if (step % 32 == 0) {
                const bool none = page_next >= a.cache.pages;
                missing = __ballot(none);
                const uint64_t row = (((none ? 0 : page_next) * (uint64_t)kv + head) << pl) +
                                     ((key + lane / 2 * hop + lane % 2 * 16) & mask);
                at_lo = (uint32_t)(row * row_bytes);
                at_hi = (uint32_t)(row * row_bytes >> 32);
                scale_lo = (uint32_t)(4 * row);
                scale_hi = (uint32_t)(4 * row >> 32);
                look(key + 32 * hop);
            }
            hole = (uint32_t)(missing >> 2 * (step % 32)) & 3;
            ++step;
        };
        auto from_lane = [&](uint32_t hi, uint32_t lo, int t) {
            const uint32_t i = 2 * ((step - 1) % 32) + t;
            return (uint64_t)(uint32_t)__builtin_amdgcn_readlane(hi, i) << 32 | (uint32_t)__builtin_amdgcn_readlane(lo, i);
        };
        auto load_k = [&]() {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const __amdgpu_buffer_rsrc_t p = window_at(a.cache.k, from_lane(at_hi, at_lo, t), hole >> t & 1 ? 0 : 16 * row_bytes);
#pragma unroll
                for (int ks = 0; ks < KL; ++ks)
                    kr[t][ks] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(p, k_off[ks], 0, 0));
                if (FP8)
                    ksc[t] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                        window_at(a.cache.ks, from_lane(scale_hi, scale_lo, t), hole >> t & 1 ? 0 : 64), 16 * quad, 0, 0));
            }
        };
        auto load_v = [&]() {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const __amdgpu_buffer_rsrc_t p = window_at(a.cache.v, from_lane(at_hi, at_lo, t), hole >> t & 1 ? 0 : 16 * row_bytes);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    load_dwords<VW>(p, v_off[j], vr[4 * t + j]);
                if (FP8)
                    vsc[t] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                        window_at(a.cache.vs, from_lane(scale_hi, scale_lo, t), hole >> t & 1 ? 0 : 64), 16 * quad, 0, 0));
            }
        };
        // V's fragments of the lane's elements 2 e and 2 e + 1 (E4M3: 4 e .. 4 e + 3): bytes
        // of 8 keys put together
        constexpr int FRAGS = FP8 ? 4 : 2;
        auto fragments = [&](int e, bf16x8 *f) {
            auto mix = [](uint32_t hi, uint32_t lo, uint32_t how) { return __builtin_amdgcn_perm(hi, lo, how); };
            constexpr uint32_t FIRST = 0x05040100u, LAST = 0x07060302u;            // halves of two words
            if constexpr (!FP8) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    u32x4 r;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        r[k] = mix(vr[2 * k + 1][e], vr[2 * k][e], h ? LAST : FIRST);
                    f[h] = __builtin_bit_cast(bf16x8, r);
                }
            } else {
                uint32_t x[4][2];          // element, 4 keys
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t v0 = vr[4 * t][e], v1 = vr[4 * t + 1][e], v2 = vr[4 * t + 2][e], v3 = vr[4 * t + 3][e];
                    const uint32_t a0 = mix(v1, v0, 0x05010400u), a1 = mix(v1, v0, 0x07030602u);
                    const uint32_t b0 = mix(v3, v2, 0x05010400u), b1 = mix(v3, v2, 0x07030602u);
                    x[0][t] = mix(b0, a0, FIRST);
                    x[1][t] = mix(b0, a0, LAST);
                    x[2][t] = mix(b1, a1, FIRST);
                    x[3][t] = mix(b1, a1, LAST);
                }
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    f[h] = __builtin_bit_cast(bf16x8, bf16_of_e4m3((u32x2){x[h][0], x[h][1]}));
            }
        };

        // (a wave whose block has no rows goes past the keys at once)
        uint32_t key = rows > 0 ? key_from + STEP * (wave / blocks) : key_to;
        look(key);
        places(key);
        load_k();
        load_v();
        // (under the first loads)
        if (off + count < tiles) {
            goes_on = true;
            const uint32_t last = min(share_of(unit + tiles - 1, total, shares), (uint32_t)shares - 1);
            if (tid == 0)
                parts.begun[w] = {off == 0 ? (int)w : (int)share_of(unit, total, shares), (int)last, q.token, 0, (int)all_rows, (int)head, {0, 0}};
        }
#pragma unroll 1
        for (; key < key_to; key += hop) {
            const uint32_t hole_now = hole, next = key + hop;
            // ---- scores
            f32x4 s[NQ][2];
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
                s[nq][0] = s[nq][1] = (f32x4){0, 0, 0, 0};
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    u32x4 kw = kr[t][FP8 ? ks / 2 : ks];
                    if constexpr (FP8)
                        kw = bf16_of_e4m3((u32x2){kw[2 * (ks % 2)], kw[2 * (ks % 2) + 1]});
#pragma unroll
                    for (int nq = 0; nq < NQ; ++nq)
                        s[nq][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kw), qf[nq][ks],
                                                                           s[nq][t], 0, 0, 0);
                }
            float unit_scale = scale;
            if constexpr (FP8) {
                unit_scale = 1.0f;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const f32x4 z = ksc[t] * scale;
#pragma unroll
                    for (int nq = 0; nq < NQ; ++nq)
                        s[nq][t] *= z;
                }
            }
            // (always, so that the registers stay the same ones: past the end nothing is fetched)
            places(next);
            load_k();

            // ---- a step that some row sees only in part
            if ((int)key < all_from || (int)(key + STEP) > all_to || hole_now) {
                const int first = (int)key + 4 * (int)here(quad);     // of the lane's keys first + 16 t + i
                uint32_t odd = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int at = first + 16 * (k / 4) + k % 4;
                    const bool whole = !(hole_now >> (k / 4) & 1);
#pragma unroll
                    for (int nq = 0; nq < NQ; ++nq) {
                        const bool sees = whole && at <= pos[nq] && (!a.window || (uint32_t)(pos[nq] - at) < a.window);
                        float x = sees ? s[nq][k / 4][k % 4] : -INFINITY;
                        asm volatile("" : "+v"(x));
                        s[nq][k / 4][k % 4] = x;
                    }
                    // V's rows that no row of Q sees, as zeros (0 times NaN is NaN)
                    const bool any = whole && at >= q.first && at < q.len;
#pragma unroll
                    for (int e = 0; e < VW; ++e) {
                        uint32_t x = any ? vr[k][e] : 0u;
                        asm volatile("" : "+v"(x));
                        vr[k][e] = x;
                        // E4M3's NaN codes are 0x7F and 0xFF: one more carries into their top bits
                        odd |= FP8 ? ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u : odd_tops(x);
                    }
                }
                if (__any(odd != 0)) {
                    // NaN or an infinity that some rows see: noted for them, and kept from the others as a zero
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        uint32_t bits = 0;
#pragma unroll
                        for (int e = 0; e < VW; ++e) {
                            if constexpr (FP8) {
                                const uint32_t z = ((vr[k][e] & 0x7F7F7F7Fu) + 0x01010101u) >> 7 & 0x01010101u;
                                bits |= (z * 0x10204080u >> 28) << 4 * e;         // bytes 0..3 to bits 0..3
                                vr[k][e] &= ~(z * 0xFFu);
                            } else {
                                const uint32_t z = not_finite(vr[k][e]);
                                bits |= ((z & 1u) | z >> 30 & 2u) << 2 * e;
                                vr[k][e] &= ~z;
                            }
                        }
                        odd_bits[wave][16 * (k / 4) + 4 * quad + k % 4][col] = (uint16_t)bits;
                    }
#pragma unroll 1
                    for (int k = 0; k < (int)STEP; ++k) {
                        const int at = (int)key + k;
#pragma unroll
                        for (int nq = 0; nq < NQ; ++nq)
                            if (at <= pos[nq] && (!a.window || (uint32_t)(pos[nq] - at) < a.window) && !(hole_now >> (k / 16) & 1))
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    nans[nq][i / 2] |= (uint32_t)odd_bits[wave][k][4 * quad + i] << 16 * (i % 2);
                    }
                }
            }

            // ---- probabilities
            bf16x8 pf[NQ], rest[NQ];
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) {
                float top = -INFINITY, p[8];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top = __builtin_fmaxf(__builtin_fmaxf(top, s[nq][0][i]), s[nq][1][i]);
                top *= unit_scale;
                if (__any(top > m[nq] + 8.0f)) {
                    // a row's four lanes agree on a new maximum; what was summed under the old one fades.
                    // The other rows keep theirs, so that no row depends on keys that it does not see
                    top = __builtin_fmaxf(top, __shfl_xor(top, 16, 64));
                    top = __builtin_fmaxf(top, __shfl_xor(top, 32, 64));
                    top = top > m[nq] + 8.0f ? top : m[nq];
                    const float to = top == -INFINITY ? 0.0f : top;
                    const float fade = __builtin_amdgcn_exp2f(m[nq] - to);
                    m[nq] = top;
                    base[nq] = to;
                    l[nq] *= fade;
#pragma unroll
                    for (int j = 0; j < EPL; ++j)
                        acc[nq][j] *= fade;
                }
                float row_scale = unit_scale;
                if (!FP8 && __any(far(base[nq]))) {
                    if (far(base[nq])) {
                        s[nq][0] *= unit_scale;
                        s[nq][1] *= unit_scale;
                        row_scale = 1.0f;
                    }
                }
                float part = 0.0f;
                u32x4 w4;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[nq][i / 4][i % 4], row_scale, -base[nq]));
                    part += p[i];
                    if (FP8)
                        p[i] *= finite_scale(vsc[i / 4][i % 4]);
                }
                l[nq] += part;
                // BF16 is the operand's type.  A BF16 cache: the probabilities and what their
                // rounding leaves of them, two products (to 2^-16); an E4M3 cache, whose values
                // are themselves rounded by up to 2^-4: the rounded ones, by up to 2^-8.
                // Measured, distance to 64 bits in the 2-norm: 0.0017, the output's own rounding,
                // for 0.0023 with one product; 16 x 1 over 9001, 32 heads on 8, the same 93 us (d = 64:
                // 43.5 -> 45); in E4M3 16 x 5 over 9001, 40 heads on 4, it would be 52 -> 55.5
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w4[i] = pk_bf16(p[2 * i], p[2 * i + 1]);
                pf[nq] = __builtin_bit_cast(bf16x8, w4);
                if constexpr (!FP8) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w4[i] = pk_bf16(p[2 * i] - bf16_lo(w4[i]), p[2 * i + 1] - bf16_hi(w4[i]));
                    rest[nq] = __builtin_bit_cast(bf16x8, w4);
                }
            }

            // ---- V
#pragma unroll
            for (int e = 0; e < EPL / FRAGS; ++e) {
                bf16x8 f[FRAGS];
                fragments(e, f);
#pragma unroll
                for (int h = 0; h < FRAGS; ++h)
#pragma unroll
                    for (int nq = 0; nq < NQ; ++nq) {
                        f32x4 &o = acc[nq][FRAGS * e + h];
                        o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[h], pf[nq], o, 0, 0, 0);
                        if (!FP8)
                            o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[h], rest[nq], o, 0, 0, 0);
                    }
            }
            load_v();
        }

        // ---- the four waves join; a lane holds d = EPL (4 quad + i) + j of row col
        __syncthreads();                   // the last unit's sums have been read
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
            float sum = l[nq];
            sum += __shfl_xor(sum, 16, 64);
            sum += __shfl_xor(sum, 32, 64);
            if (quad == 0)
                ml_lds[wave][16 * nq + col] = (f32x2){m[nq], sum};
        }
        __syncthreads();
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
            float top = -INFINITY;
            for (uint32_t v = wave % blocks; v < WAVES; v += blocks)
                top = __builtin_fmaxf(top, ml_lds[v][16 * nq + col][0]);
            const float f = __builtin_amdgcn_exp2f(m[nq] - (top == -INFINITY ? 0.0f : top));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float *dst = &o_lds[wave][16 * nq + col][EPL * (4 * quad + i)];
#pragma unroll
                for (int j = 0; j < EPL; ++j)
                    dst[j] = nans[nq][i / 2] >> (16 * (i % 2) + j) & 1 ? __builtin_nanf("") : acc[nq][j][i] * f;
            }
        }
        __syncthreads();
        const bool finished = count == tiles;
        const bool begins = off == 0;
        const size_t slot = (2 * (size_t)w + begins) * ROWS * blocks;
        for (uint32_t i = tid; i < ROWS * blocks * (DP / 8); i += WG) {
            const uint32_t r = i / (DP / 8), e = 8 * (i % (DP / 8)), block = r / ROWS, rb = r % ROWS;
            if (r >= all_rows || e >= d)
                continue;
            float top = -INFINITY, sum = 0.0f, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            for (uint32_t u = block; u < WAVES; u += blocks)
                top = __builtin_fmaxf(top, ml_lds[u][rb][0]);
            const float to = top == -INFINITY ? 0.0f : top;
            for (uint32_t u = block; u < WAVES; u += blocks) {
                sum += ml_lds[u][rb][1] * __builtin_amdgcn_exp2f(ml_lds[u][rb][0] - to);
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    const f32x4 part = *(const f32x4 *)&o_lds[u][rb][e + j];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[j + k] += part[k];
                }
            }
            if (finished) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                const uint32_t tok = r / group;
                u32x4 y;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    y[j] = pk_bf16(v[2 * j] * inv, v[2 * j + 1] * inv);
                *(u32x4 *)(a.out + ((size_t)(q.token + tok) * a.q_heads + head * group + (r - tok * group)) * d + e) = y;
            } else {
                float *dst = parts.o + (slot + r) * d + e;
                *(f32x4 *)dst = (f32x4){v[0], v[1], v[2], v[3]};
                *(f32x4 *)(dst + 4) = (f32x4){v[4], v[5], v[6], v[7]};
                if (e == 0)
                    parts.ml[slot + r] = (f32x2){top, sum};
            }
        }
        x += count;
    }
    if (!goes_on && tid == 0)
        parts.begun[w] = {0, -1, 0, 0, 0, 0, {0, 0}};
}

// A unit's rows go to the workgroups of all its shares but the last (no other unit
// goes on from those).  LP lanes take a row of a part, 16 bytes each, and a
// workgroup has G such groups: of few parts (by_row) each goes through all parts
// of a row of its own; of many, they share a row's parts and join through LDS.
template <int LP>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, Parts parts, uint32_t rows)
{
    constexpr uint32_t G = 256 / LP;
    __shared__ float o_lds[G][4 * LP];
    __shared__ f32x2 ml_lds[G];
    const Begun b = parts.begun[blockIdx.x];
    if (b.last <= b.first)
        return;
    const uint32_t d = a.cache.d, group = a.q_heads / a.cache.heads, g = threadIdx.x / LP, e = 4 * (threadIdx.x % LP);
    const uint32_t from = b.first, count = b.last - from + 1;
    const bool by_row = count <= 4 || (count <= 8 && (uint32_t)b.rows >= G);
    const uint32_t per = by_row ? G : 1, each = (count - 1) * per;
    for (uint32_t r0 = blockIdx.y * each + (blockIdx.x - from) * per; r0 < (uint32_t)b.rows; r0 += gridDim.y * each) {
        const uint32_t r = r0 + (by_row ? g : 0);
        float m = -INFINITY, l = 0.0f;
        f32x4 acc = {0, 0, 0, 0};
        constexpr int U = 4;
        const uint32_t step = by_row ? 1 : G;
        for (uint32_t p0 = by_row ? 0 : g; p0 < count; p0 += U * step) {
            f32x2 ml[U];
            f32x4 o[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t p = p0 + u * step;
                ml[u] = (f32x2){-INFINITY, 0.0f};
                o[u] = (f32x4){0, 0, 0, 0};
                if (p < count && r < (uint32_t)b.rows) {
                    const size_t at = (2 * (size_t)(from + p) + (p == 0)) * rows + r;
                    ml[u] = parts.ml[at];
                    if (e < d)
                        o[u] = *(const f32x4 *)(parts.o + at * d + e);
                }
            }
            float top = m;
#pragma unroll
            for (int u = 0; u < U; ++u)
                top = __builtin_fmaxf(top, ml[u][0]);
            const float to = top == -INFINITY ? 0.0f : top;
            float f = __builtin_amdgcn_exp2f(m - to);
            l *= f;
            acc *= f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                f = __builtin_amdgcn_exp2f(ml[u][0] - to);
                l += ml[u][1] * f;
                acc += o[u] * f;
            }
            m = top;
        }
        if (!by_row) {
            __syncthreads();
            *(f32x4 *)&o_lds[g][e] = acc;
            if (e == 0)
                ml_lds[g] = (f32x2){m, l};
            __syncthreads();
            if (g != 0)
                continue;
            float top = -INFINITY;
            for (uint32_t u = 0; u < G; ++u)
                top = __builtin_fmaxf(top, ml_lds[u][0]);
            const float to = top == -INFINITY ? 0.0f : top;
            l = 0.0f;
            acc = (f32x4){0, 0, 0, 0};
            for (uint32_t u = 0; u < G; ++u) {
                const float f = __builtin_amdgcn_exp2f(ml_lds[u][0] - to);
                l += ml_lds[u][1] * f;
                acc += *(const f32x4 *)&o_lds[u][e] * f;
            }
        }
        if (e < d && r < (uint32_t)b.rows) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const uint32_t flat = b.row + r, tok = flat / group;
            *(u32x2 *)(a.out + ((size_t)(b.token + tok) * a.q_heads + b.head * group + (flat - tok * group)) * d + e) =
                (u32x2){pk_bf16(acc[0] * inv, acc[1] * inv), pk_bf16(acc[2] * inv, acc[3] * inv)};
        }
    }
}

template <int LP>
void join(const AttnArgs &a, const Parts &p, uint32_t shares, uint32_t rows, uint32_t live, hipStream_t st)
{
    constexpr uint32_t G = 256 / LP;
    k_attn_join<LP><<<dim3(shares, (live + G - 1) / G), 256, 0, st>>>(a, p, rows);
}

template <int DP, int NQ>
void launch_rows(const AttnArgs &a, const Parts &p, uint32_t shares, uint32_t blocks, hipStream_t st)
{
    if (a.cache.fp8)
        k_attn_decode<DP, NQ, true><<<shares, WG, 0, st>>>(a, p, shares, blocks);
    else
        k_attn_decode<DP, NQ, false><<<shares, WG, 0, st>>>(a, p, shares, blocks);
}

// Rows of a block: 16, or (more, and as long as they leave two waves a SIMD) 32.
uint32_t room(uint32_t rows, uint32_t d) { return rows <= 16 || d > 128 ? 16 : 32; }

uint32_t blocks_of(uint32_t rows, uint32_t d)
{
    const uint32_t n = (rows + room(rows, d) - 1) / room(rows, d);
    return n <= 2 ? n : 4;
}

template <int DP>
void launch(const AttnArgs &a, const Parts &p, uint32_t rows, uint32_t shares, hipStream_t st)
{
    if constexpr (DP <= 128) {
        if (room(rows, DP) == 32) {
            launch_rows<DP, 2>(a, p, shares, blocks_of(rows, DP), st);
            return;
        }
    }
    launch_rows<DP, 1>(a, p, shares, blocks_of(rows, DP), st);
}

} // namespace

hipError_t launch_attn_join(const AttnArgs &a, const Parts &p, uint32_t shares, uint32_t rows, uint32_t live,
                            hipStream_t st)
{
    if (a.cache.d <= 64)
        join<16>(a, p, shares, rows, live, st);
    else if (a.cache.d <= 128)
        join<32>(a, p, shares, rows, live, st);
    else
        join<64>(a, p, shares, rows, live, st);
    count_launch();
    return hipGetLastError();
}

// As many workgroups as the chip holds at a time.
static uint32_t max_shares(uint32_t d)
{
    return (d <= 128 ? 2 : 1) * (cu_count() ? cu_count() : 256);
}

uint64_t decode_work(uint32_t rows, uint32_t d)
{
    return parts_bytes(max_shares(d), room(rows, d) * blocks_of(rows, d), d);
}

hipError_t launch_attn_decode(const AttnArgs &a, hipStream_t st)
{
    const uint32_t rows = a.max_q * (a.q_heads / a.cache.heads), d = a.cache.d, each = room(rows, d) * blocks_of(rows, d);
    // no more workgroups than the table has room for tiles
    const uint64_t most = (uint64_t)a.seqs * a.cache.heads * ((((uint64_t)a.width << a.cache.page_log2) + TILE - 1) / TILE);
    const uint32_t shares = (uint32_t)min((uint64_t)max_shares(d), most);
    const Parts p = parts_at(a.work, shares, each);
    if (d <= 64)
        launch<64>(a, p, rows, shares, st);
    else if (d <= 128)
        launch<128>(a, p, rows, shares, st);
    else
        launch<256>(a, p, rows, shares, st);
    count_launch();
    if (hipError_t e = hipGetLastError())
        return e;
    return launch_attn_join(a, p, shares, each, rows, st);
}

} // namespace attn
} // namespace qp
