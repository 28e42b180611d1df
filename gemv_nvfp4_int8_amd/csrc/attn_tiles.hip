// attn_tiles.hip -- attention of many rows a sequence (chunks of a prompt, whole
// prompts, large verify batches).
//
// A workgroup takes a unit of 32 rows a wave and goes through its keys 64 at a
// time; K and V of the next 64 are on their way to registers while these are
// worked on from LDS, two buffers in turn with one barrier.  A wave computes
//   S^T [key, row] = K Q^T   32x32x16 MFMAs, K from LDS, Q in registers
//   P^T = exp2(S^T - m)      a lane holds 32 scores of ONE row: its maximum and sum
//                            need one exchange with the lane 32 further, the
//                            maximum's only when it grows by more than 2^8
//   O^T [d, row] += V^T P^T  P^T is already in the operand's layout, if slot i of
//                            lane half h stands for key 4h + i % 4 + 8 (i / 4) of
//                            each 16; V's fragment takes them so with transposing
//                            LDS reads of 4 keys by 16 of d
// LDS rows hold 16-byte pieces in an order turned by the row number (`swizzle`),
// so that both 16 rows of one piece (K) and 4 rows of 64 bytes (V) lie in
// different banks.
#include "attn_common.hpp"
#include "qp_launch.hpp"

namespace qp {
namespace attn {
namespace {

constexpr uint32_t KT = 64;                // keys of a tile

typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// The XOR of row r's piece numbers.
template <int DP>
__device__ __forceinline__ uint32_t swizzle(uint32_t r)
{
    return DP == 64 ? (r >> 1 & 1) << 2 | (r >> 2 & 3) : (r & 3) << 2 | (r >> 2 & 3);
}

// A block of a sequence's rows: which keys any of them sees.
struct Block {
    int from, to;                          // positions
    uint32_t first_tile, tiles;
};

__device__ __forceinline__ Block block_of(const AttnArgs &a, int n, int len, uint32_t row, uint32_t rows, uint32_t group)
{
    Block b;
    const uint32_t end = min(row + rows, (uint32_t)n * group);
    const int lo = len - n + (int)(row / group), hi = len - n + (int)((end - 1) / group);
    const int64_t back = (int64_t)lo - (int64_t)a.window + 1;
    b.from = a.window && back > 0 ? (int)back : 0;
    b.to = max(hi + 1, 0);
    b.first_tile = b.from / KT;
    b.tiles = max((b.to + KT - 1) / KT - min((uint32_t)b.first_tile, (b.to + KT - 1) / KT), 1u);
    return b;
}

template <int DP, int NW, bool FP8>
__global__ __launch_bounds__(64 * NW, DP <= 128 ? 2 : 1) void k_attn_tiles(AttnArgs a, Parts parts, uint32_t max_shares)
{
    constexpr uint32_t WG = 64 * NW;
    constexpr uint32_t ROWS = 32 * NW;
    constexpr int KS = DP / 16;            // MFMAs over d
    constexpr int DB = DP / 32;            // blocks of O's d
    constexpr uint32_t CH = DP / 8;        // 16-byte pieces of a row in LDS
    constexpr uint32_t CPR = FP8 ? DP / 16 : DP / 8;   // 16-byte pieces of a row in memory
    constexpr uint32_t ITEMS = KT * CPR / WG;          // of a thread, of K and of V each
    constexpr uint32_t TILE_BYTES = KT * DP * 2;
    static_assert(ITEMS >= 1 && KT * CPR % WG == 0, "every thread loads as many pieces");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][2][TILE_BYTES];      // buffer; K, V
    __shared__ float scales[2][2][KT];     // of K, of V (E4M3)
    __shared__ uint32_t holes[2][KT / 16], odd[2][NW];
    __shared__ uint8_t odd_bits[2][KT][CH];      // which of a piece of V are NaN or infinite
    __shared__ uint32_t scan[NW], seq_n[WG], seq_len[WG], seq_end[WG];
    __shared__ uint32_t found[4];

    const uint32_t tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const uint32_t col = lane % 32, half = lane / 32;
    const uint32_t d = a.cache.d, kv = a.cache.heads, group = a.q_heads / kv, pl = a.cache.page_log2;

    auto block_scan = [&](uint32_t v, uint32_t &all) {  // inclusive over the workgroup
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const uint32_t up = __shfl_up(v, off, 64);
            v += lane >= (uint32_t)off ? up : 0;
        }
        __syncthreads();
        if (lane == 63)
            scan[wave] = v;
        __syncthreads();
        all = 0;
        uint32_t ahead = 0;
        for (uint32_t w = 0; w < NW; ++w) {
            ahead += w < wave ? scan[w] : 0;
            all += scan[w];
        }
        return v + ahead;
    };
    // Walks all blocks in order, WG sequences and then WG blocks at a time; with
    // `want` below the total, leaves the block that holds that tile in found[]:
    // sequence, first row, the tiles before it.  Returns the tiles walked.
    auto walk = [&](uint64_t want) {
        uint64_t before = 0;
        for (uint32_t s0 = 0; s0 < a.seqs; s0 += WG) {
            const Seq q = s0 + tid < a.seqs ? read_seq(a, s0 + tid) : Seq{0, 0, 0, 0};
            uint32_t blocks;
            const uint32_t end = block_scan((q.n * group + ROWS - 1) / ROWS, blocks);
            seq_n[tid] = q.n;
            seq_len[tid] = q.len;
            seq_end[tid] = end;
            __syncthreads();
            for (uint32_t b0 = 0; b0 < blocks; b0 += WG) {
                const uint32_t b = b0 + tid;
                uint32_t tiles = 0, s = 0, row = 0;
                if (b < blocks) {
                    uint32_t hi = WG - 1;               // the first sequence whose blocks end behind b
                    while (s < hi) {
                        const uint32_t mid = (s + hi) / 2;
                        if (seq_end[mid] > b)
                            hi = mid;
                        else
                            s = mid + 1;
                    }
                    row = (b - (s ? seq_end[s - 1] : 0)) * ROWS;
                    tiles = block_of(a, seq_n[s], seq_len[s], row, ROWS, group).tiles;
                }
                uint32_t all;
                const uint64_t to = before + block_scan(tiles, all), from = to - tiles;
                if (want >= from && want < to) {
                    found[0] = s0 + s;
                    found[1] = row;
                    found[2] = (uint32_t)from;
                    found[3] = (uint32_t)(from >> 32);
                }
                before += all;
                if (want < before)
                    break;
            }
            __syncthreads();
            if (want < before)
                break;
        }
        return before;
    };
    const uint64_t line = uniform(walk(~0ull));     // tiles of one kv head
    const uint64_t total = line * kv, shares = min((uint64_t)max_shares, total);
    const uint32_t w = xcd_remap(blockIdx.x, gridDim.x);
    if (w >= shares) {
        if (tid == 0)
            parts.begun[w].last = -1;
        return;
    }
    uint64_t x = uniform(w * total / shares);
    const uint64_t share_end = uniform((w + 1) * total / shares);
    uint32_t head = uniform((uint32_t)(x / line));
    walk(x % line);
    uint32_t seq = uniform(found[0]), row0 = uniform(found[1]);
    uint64_t unit = (uint64_t)head * line + uniform((uint64_t)found[3] << 32 | found[2]);

    const float scale = a.scale * LOG2E;
    bool began = false;
    // LDS addresses of a lane's fragments: K's piece 2 ks + half of row col, V's
    // pieces of rows 4 half + (lane % 16) / 4 (+ 8) that hold its group's 16 of d
    const uint32_t k_row = col * DP * 2, k_swz = swizzle<DP>(col);
    const uint32_t v_row = 4 * half + lane % 16 / 4, v_piece = 2 * (lane / 16 % 2) + lane % 4 / 2;
    uint32_t v_addr[2][DB];
#pragma unroll
    for (int jj = 0; jj < 2; ++jj)
#pragma unroll
        for (int db = 0; db < DB; ++db) {
            const uint32_t r = v_row + 8 * jj;
            v_addr[jj][db] = r * DP * 2 + ((4 * db + v_piece) ^ swizzle<DP>(r)) * 16 + lane % 2 * 8;
        }

    while (x < share_end) {
        const Seq q = read_seq_uniform(a, seq);
        if (row0 >= (uint32_t)q.n * group) {            // the next sequence, or the next head's first
            row0 = 0;
            if (++seq == a.seqs) {
                seq = 0;
                if (++head == kv)
                    break;                              // not reached unless the lengths change under the call
            }
            continue;
        }
        const Block blk = block_of(a, q.n, q.len, row0, ROWS, group);
        const uint32_t off = (uint32_t)(x - unit);
        if (off >= blk.tiles)
            break;
        const uint32_t count = (uint32_t)min((uint64_t)(blk.tiles - off), share_end - x);
        const uint32_t rows = min(ROWS, (uint32_t)q.n * group - row0);

        // ---- the wave's rows
        const uint32_t first_row = row0 + 32 * wave, my_row = first_row + col;
        const bool wave_live = 32 * wave < rows, row_live = 32 * wave + col < rows;
        const int old = q.len - q.n;
        const int pos = old + (int)(my_row / group);
        const int pos_lo = old + (int)(first_row / group), pos_hi = old + (int)((min(first_row + 32, row0 + rows) - 1) / group);
        const size_t q_at = ((size_t)(q.token + my_row / group) * a.q_heads + head * group + my_row % group) * d;
        bf16x8 qf[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            u32x4 v = {0, 0, 0, 0};
            if (row_live && 16 * ks + 8 * half < d)
                v = *(const u32x4 *)(a.q + q_at + 16 * ks + 8 * half);
            qf[ks] = __builtin_bit_cast(bf16x8, v);
        }
        float m = -INFINITY, base = 0.0f, l = 0.0f;
        f32x16 acc[DB];
#pragma unroll
        for (int db = 0; db < DB; ++db)
            acc[db] = (f32x16)0.0f;

        // ---- loads: a thread's pieces of the tile, its page numbers one tile ahead
        const uint32_t t_end = blk.first_tile + off + count;
        const size_t table = (size_t)seq * a.width, plane = ((size_t)kv * d) << pl;
        const uint32_t mask = (1u << pl) - 1;
        const uint32_t elem = FP8 ? 1 : 2;
        u32x4 kr[ITEMS], vr[ITEMS];
        float ksr = 0.0f, vsr = 0.0f;
        uint32_t ok = 0, hole = 0, page[ITEMS], spage = 0;
        auto look = [&](uint32_t tile) {
#pragma unroll
            for (uint32_t i = 0; i < ITEMS; ++i) {
                const uint32_t key = tile * KT + (tid + WG * i) / CPR;
                page[i] = key < (uint32_t)blk.to ? (uint32_t)a.table[table + (key >> pl)] : ~0u;
            }
            if (FP8 && tid < KT) {
                const uint32_t key = tile * KT + tid;
                spage = key < (uint32_t)blk.to ? (uint32_t)a.table[table + (key >> pl)] : ~0u;
            }
        };
        auto load = [&](uint32_t tile) {
            ok = hole = 0;
#pragma unroll
            for (uint32_t i = 0; i < ITEMS; ++i) {
                const uint32_t it = tid + WG * i, key = tile * KT + it / CPR, c = it % CPR;
                const bool page_ok = page[i] < a.cache.pages;
                const bool fine = page_ok && (int)key >= blk.from && c * (FP8 ? 16 : 8) < d;
                ok |= (uint32_t)fine << i;
                hole |= (uint32_t)!page_ok << i;
                const size_t at = fine ? ((page[i] * plane + (((size_t)head << pl) + (key & mask)) * d) * elem + c * 16) : 0;
                kr[i] = *(const u32x4 *)((const uint8_t *)a.cache.k + at);
                vr[i] = *(const u32x4 *)((const uint8_t *)a.cache.v + at);
            }
            if (FP8 && tid < KT) {
                const uint32_t key = tile * KT + tid;
                const size_t at = spage < a.cache.pages ? ((spage * (size_t)kv + head) << pl) + (key & mask) : 0;
                ksr = a.cache.ks[at];
                vsr = a.cache.vs[at];
            }
        };
        auto store = [&](uint32_t tile, uint32_t buf) {
            uint32_t bad = 0;
            const int k0 = tile * KT;
            // a piece of V; where NaN and infinities have to be kept from some rows, zeros in their places and a note of them
            auto put_v = [&](uint8_t *to, u32x4 v, uint8_t *note, bool edge) {
                if (edge) {
                    uint32_t bits = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t z = not_finite(v[i]);
                        bits |= (z & 1) << (2 * i) | (z >> 31) << (2 * i + 1);
                        v[i] &= ~z;
                    }
                    *note = bits;
                    bad |= bits;
                }
                *(u32x4 *)to = v;
            };
            // some row of the block does not see some key of the tile
            const bool edge = k0 + (int)KT - 1 > old + (int)(row0 / group) ||
                              (a.window && k0 <= old + (int)((row0 + rows - 1) / group) - (int64_t)a.window);
#pragma unroll
            for (uint32_t i = 0; i < ITEMS; ++i) {
                const uint32_t it = tid + WG * i, r = it / CPR, c = it % CPR;
                if (!(ok >> i & 1))
                    kr[i] = vr[i] = (u32x4){0, 0, 0, 0};
                uint8_t *kd = lds[buf][0] + r * DP * 2, *vd = lds[buf][1] + r * DP * 2;
                const uint32_t z = swizzle<DP>(r);
                if constexpr (FP8) {
#pragma unroll
                    for (uint32_t h = 0; h < 2; ++h) {
                        const uint32_t p = ((2 * c + h) ^ z) * 16;
                        *(u32x4 *)(kd + p) = bf16_of_e4m3((u32x2){kr[i][2 * h], kr[i][2 * h + 1]});
                        put_v(vd + p, bf16_of_e4m3((u32x2){vr[i][2 * h], vr[i][2 * h + 1]}), &odd_bits[buf][r][2 * c + h], edge);
                    }
                } else {
                    *(u32x4 *)(kd + (c ^ z) * 16) = kr[i];
                    put_v(vd + (c ^ z) * 16, vr[i], &odd_bits[buf][r][c], edge);
                }
                if (c == 0 && r % 16 == 0)
                    holes[buf][r / 16] = hole >> i & 1;
            }
            if (FP8 && tid < KT) {
                scales[buf][0][tid] = ksr * scale;
                scales[buf][1][tid] = vsr;
            }
            const bool any = __any(bad != 0);
            if (lane == 0)
                odd[buf][wave] = any;
        };

        uint32_t tile = blk.first_tile + off;
        look(tile);
        load(tile);
        if (tile + 1 < t_end)
            look(tile + 1);
        __syncthreads();                   // the last unit's tiles have been read
        store(tile, 0);
        __syncthreads();
        for (uint32_t buf = 0; tile < t_end; ++tile, buf ^= 1) {
            const bool more = tile + 1 < t_end;
            if (more) {
                load(tile + 1);
                if (tile + 2 < t_end)
                    look(tile + 2);
            }
            const int k0 = tile * KT;
            const uint32_t gaps = __builtin_amdgcn_readfirstlane(holes[buf][0] | holes[buf][1] << 1 | holes[buf][2] << 2 |
                                                                 holes[buf][3] << 3);
            const bool none = !wave_live || k0 > pos_hi || (a.window && k0 + (int)KT - 1 <= pos_lo - (int64_t)a.window);
            if (!none) {
                // ---- scores
                f32x16 s[2];
                const uint8_t *kt = lds[buf][0] + k_row, *vt = lds[buf][1];
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    s[kb] = (f32x16)0.0f;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const bf16x8 kf = *(const bf16x8 *)(kt + kb * 32 * DP * 2 + ((2 * ks + half) ^ k_swz) * 16);
                        s[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[ks], s[kb], 0, 0, 0);
                    }
                }
                const float unit_scale = FP8 ? 1.0f : scale;
                if constexpr (FP8) {
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const f32x4 z = *(const f32x4 *)&scales[buf][0][32 * kb + 2 * i + 4 * half];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                s[kb][i + j] *= z[j];
                        }
                }
                const bool whole = k0 + (int)KT - 1 <= pos_lo && (!a.window || k0 > pos_hi - (int64_t)a.window) && gaps == 0;
                uint32_t seen = ~0u;       // bit 16 kb + i: the lane's row sees key 32 kb + 8 (i / 4) + 4 half + i % 4
                if (!whole) {
                    seen = 0;
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int k = 32 * kb + 8 * (i / 4) + 4 * (int)half + i % 4;
                            const bool see = k0 + k <= pos && (!a.window || (uint32_t)(pos - k0 - k) < a.window) &&
                                             !(gaps >> (2 * kb + i / 8) & 1);
                            seen |= (uint32_t)see << (16 * kb + i);
                            s[kb][i] = see ? s[kb][i] : -INFINITY;
                        }
                }
                // ---- probabilities
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    top = __builtin_fmaxf(top, __builtin_fmaxf(s[0][i], s[1][i]));
                top *= unit_scale;
                if (__any(top > m + 8.0f)) {
                    top = __builtin_fmaxf(top, __shfl_xor(top, 32, 64));
                    top = __builtin_fmaxf(top, m);
                    const float to = top == -INFINITY ? 0.0f : top;
                    const float fade = __builtin_amdgcn_exp2f(m - to);
                    m = top;
                    base = to;
                    l *= fade;
#pragma unroll
                    for (int db = 0; db < DB; ++db)
                        acc[db] *= fade;
                }
                float part[4] = {0, 0, 0, 0};
                bf16x8 pf[2][2];
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int sb = 0; sb < 2; ++sb) {
                        float p[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][8 * sb + i], unit_scale, -base));
                            part[i % 4] += p[i];
                        }
                        if constexpr (FP8) {
#pragma unroll
                            for (int i = 0; i < 8; i += 4) {
                                const f32x4 z = *(const f32x4 *)&scales[buf][1][32 * kb + 16 * sb + 2 * i + 4 * half];
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    p[i + j] *= z[j];
                                    if (!whole)
                                        p[i + j] = seen >> (16 * kb + 8 * sb + i + j) & 1 ? p[i + j] : 0.0f;
                                }
                            }
                        }
                        // rounded to BF16, the operand's type (2^-9 of each on average over keys, as the output's own rounding)
                        u32x4 w4;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w4[i] = pk_bf16(p[2 * i], p[2 * i + 1]);
                        pf[kb][sb] = __builtin_bit_cast(bf16x8, w4);
                    }
                l += (part[0] + part[1]) + (part[2] + part[3]);

                // ---- V
                auto v_frag = [&](int kb, int sb, int db) {
                    u32x4 v;
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj) {
                        const uint8_t *p = vt + (32 * kb + 16 * sb) * DP * 2 + v_addr[jj][db];
                        const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
                        const u32x2 t2 = __builtin_bit_cast(u32x2, t);
                        v[2 * jj] = t2[0];
                        v[2 * jj + 1] = t2[1];
                    }
                    return v;
                };
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int sb = 0; sb < 2; ++sb)
#pragma unroll
                        for (int db = 0; db < DB; ++db)
                            acc[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                __builtin_bit_cast(bf16x8, v_frag(kb, sb, db)), pf[kb][sb], acc[db], 0, 0, 0);
                if (!whole) {
                    uint32_t any = 0;
                    for (uint32_t u = 0; u < NW; ++u)
                        any |= odd[buf][u];
                    if (uniform(any)) {
                        // what stood in the places of the zeros, for the rows that see it
                        for (int k = 0; k < (int)KT; ++k) {
                            const bool see = k0 + k <= pos && (!a.window || (uint32_t)(pos - k0 - k) < a.window);
                            for (uint32_t c = 0; c < CH && see; ++c)
#pragma unroll
                                for (int db = 0; db < DB; ++db)
#pragma unroll
                                    for (int i = 0; i < 16; ++i)
                                        if (c == 4u * db + i / 4 && odd_bits[buf][k][c] >> (4 * half + i % 4) & 1)
                                            acc[db][i] = __builtin_nanf("");
                        }
                    }
                }
            }
            if (more)
                store(tile + 1, buf ^ 1);
            __syncthreads();
        }

        // ---- the rows' results: a lane holds d = 32 db + 8 (i / 4) + 4 half + i % 4 of row col
        l += __shfl_xor(l, 32, 64);
        const bool begins = off == 0, finished = count == blk.tiles;
        if (row_live) {
            const size_t slot = (2 * (size_t)w + begins) * ROWS + 32 * wave + col;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            if (!finished && half == 0)
                parts.ml[slot] = (f32x2){m, l};
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const uint32_t e = 32 * db + 2 * i + 4 * half;
                    if (e >= d)
                        continue;
                    const f32x4 v = {acc[db][i], acc[db][i + 1], acc[db][i + 2], acc[db][i + 3]};
                    if (finished)
                        *(u32x2 *)(a.out + q_at + e) = (u32x2){pk_bf16(v[0] * inv, v[1] * inv), pk_bf16(v[2] * inv, v[3] * inv)};
                    else
                        *(f32x4 *)(parts.o + slot * d + e) = v;
                }
        }
        if (begins && !finished) {
            began = true;
            if (tid == 0)
                parts.begun[w] = {(int)share_of(unit + blk.tiles - 1, total, shares), q.token, (int)row0, (int)rows, (int)head, {0, 0, 0}};
        }
        x += count;
        if (x == unit + blk.tiles) {
            unit = x;
            row0 += ROWS;
        }
    }
    if (!began && tid == 0)
        parts.begun[w].last = -1;
}

template <int DP, int NW>
void launch(const AttnArgs &a, const Parts &p, uint32_t shares, hipStream_t st)
{
    if (a.cache.fp8)
        k_attn_tiles<DP, NW, true><<<shares, 64 * NW, 0, st>>>(a, p, shares);
    else
        k_attn_tiles<DP, NW, false><<<shares, 64 * NW, 0, st>>>(a, p, shares);
}

constexpr uint32_t UNIT_ROWS = 128;

uint32_t max_shares(uint32_t d)
{
    // as many workgroups as the chip holds at a time
    return (d <= 128 ? 2 : 1) * (cu_count() ? cu_count() : 256);
}

} // namespace

uint64_t tiles_work(uint32_t d)
{
    return parts_bytes(max_shares(d), UNIT_ROWS, d);
}

hipError_t launch_attn_tiles(const AttnArgs &a, hipStream_t st)
{
    const uint32_t shares = max_shares(a.cache.d);
    const Parts p = parts_at(a.work, shares, UNIT_ROWS);
    if (a.cache.d <= 64)
        launch<64, 4>(a, p, shares, st);
    else if (a.cache.d <= 128)
        launch<128, 4>(a, p, shares, st);
    else
        launch<256, 4>(a, p, shares, st);
    count_launch();
    if (hipError_t e = hipGetLastError())
        return e;
    return launch_attn_join(a, p, shares, UNIT_ROWS, UNIT_ROWS, st);
}

} // namespace attn
} // namespace qp
