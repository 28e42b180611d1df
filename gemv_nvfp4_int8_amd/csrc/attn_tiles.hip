// attn_tiles.hip -- attention of many rows a sequence (chunks of a prompt, whole
// prompts, large verify batches).
//
// A workgroup takes a unit of 32 rows a wave (d > 128: every two waves) and goes
// through its keys a tile at a time; K and V of the next tile are on their way
// (straight to LDS, or through registers where they have to be decoded) while this
// one is worked on, two buffers in turn with one barrier.  A wave computes
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
//
// Where d > 128 a row of O would take twice the registers that leave room for two
// waves a SIMD: two waves have the same 32 rows, each half of O's d, and both compute
// S, which is half as many matrix operations again (4096 rows over themselves, 32
// heads of 256: 560 us, in E4M3 635; one wave a SIMD with all of O took 40% more, in
// E4M3 twice as long).
//
// What bounds it: over long keys, at two waves a SIMD, the softmax's vector work beside
// the matrix operations (an exponential takes 8 cycles of a wave, a product of 32x32x16
// 32), the LDS reads, which 32 rows a wave just balance with the matrix operations, and
// with heads of 128 the part's power (1.84 GHz under 2000 rows over 32000); a tile of
// 256 rows by 64 keys takes 3600 cycles then.  Where units are short, their beginnings
// (lengths, then page numbers, then keys, each a trip to memory, and a masked tile at
// the end) come on top: 8192 rows over themselves are 258 tiles a share, of which the
// first share of a head begins 23 units and the last two, and take 5000 cycles a tile.
// Measured, 32 heads of 128 over 8: 8192 rows over themselves 655 us, 840 TFLOP/s (in
// E4M3 730); 2000 rows over 32000 0.92 to 0.98 ms, 1.04 to 1.10 PFLOP/s; 64
// heads of 64, 7 prompts of 1250 to 2500 in a window of 1024: 280 to 298 us, 470 to 490
// TFLOP/s of what is seen.
#include "attn_common.hpp"
#include "qp_launch.hpp"

namespace qp {
namespace attn {
namespace {

// Keys of a tile: as many as two buffers of them leave room for eight waves a
// compute unit.  (d = 64 with tiles of 64 and three waves a SIMD: 8% slower, 7 prompts
// of 1250 to 2500 in a window of 1024.  d = 128 with tiles of 128: 2000 rows over 32000
// 2% faster, but 32 prompts of 128 9% slower, 2048 rows over themselves the same either
// way, and E4M3 spills.)
constexpr uint32_t tile_keys(uint32_t d) { return d <= 64 ? 128 : d <= 128 ? 64 : 32; }

typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) void lds_void;


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

template <uint32_t KT>
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
__global__ __launch_bounds__(64 * NW, 2) void k_attn_tiles(AttnArgs a, Parts parts, uint32_t max_shares)
{
    constexpr uint32_t WG = 64 * NW, KT = tile_keys(DP), GROUPS = KT / 16, AHEAD_TILES = 64 / GROUPS;
    constexpr uint32_t SPLIT = DP <= 128 ? 1 : 2;      // waves that have the same rows, and each a part of O's d
    constexpr uint32_t ROWS = 32 * NW / SPLIT;
    constexpr int KS = DP / 16;            // MFMAs over d
    constexpr int DB = DP / 32 / SPLIT;    // blocks of a wave's part of O's d
    constexpr uint32_t CH = DP / 8;        // 16-byte pieces of a row in LDS
    constexpr uint32_t CW = CH / SPLIT;    // those of a wave's part of d
    constexpr uint32_t CPR = FP8 ? DP / 16 : DP / 8;   // 16-byte pieces of a row in memory
    constexpr uint32_t ITEMS = KT * CPR / WG;          // of a thread, of K and of V each
    constexpr uint32_t TILE_BYTES = KT * DP * 2;
    static_assert(ITEMS >= 1 && KT * CPR % WG == 0, "every thread loads as many pieces");
    // an array for each buffer: loads on their way to one do not hold up reads of the other
    __shared__ __attribute__((aligned(16))) uint8_t k_lds0[TILE_BYTES], v_lds0[TILE_BYTES], k_lds1[TILE_BYTES], v_lds1[TILE_BYTES];
    __shared__ float scales[2][2][KT];     // of K, of V (E4M3)
    __shared__ uint32_t odd[NW];
    __shared__ uint8_t odd_bits[KT][CH];         // which of a piece of V are NaN or infinite
    __shared__ uint32_t scan[NW], seq_n[WG], seq_len[WG], seq_end[WG];
    __shared__ uint32_t found[4];

    const uint32_t tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const uint32_t col = lane % 32, half = lane / 32;
    const uint32_t strip = wave / SPLIT, part_d = wave % SPLIT * (DP / SPLIT);         // the wave's rows and first d
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
    uint32_t walks = 0, at_seq = 0, at_row = 0;         // runs of WG blocks; the thread's block of the last run
    uint64_t at_from = 0, at_to = 0;
    auto find = [&](uint64_t want) {
        if (want >= at_from && want < at_to) {
            found[0] = at_seq;
            found[1] = at_row;
            found[2] = (uint32_t)at_from;
            found[3] = (uint32_t)(at_from >> 32);
        }
    };
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
                    tiles = block_of<KT>(a, seq_n[s], seq_len[s], row, ROWS, group).tiles;
                }
                uint32_t all;
                at_to = before + block_scan(tiles, all);
                at_from = at_to - tiles;
                at_seq = s0 + s;
                at_row = row;
                ++walks;
                find(want);
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
            parts.begun[w] = {0, -1, 0, 0, 0, 0, {0, 0}};
        return;
    }
    uint64_t x = uniform(w * total / shares);
    const uint64_t share_end = uniform((w + 1) * total / shares);
    uint32_t head = uniform((uint32_t)(x / line));
    if (walks == 1) {                      // all there is was one run
        find(x % line);
        __syncthreads();
    } else {
        walk(x % line);
    }
    uint32_t seq = min(uniform(found[0]), a.seqs - 1), row0 = uniform(found[1]);
    uint64_t unit = (uint64_t)head * line + uniform((uint64_t)found[3] << 32 | found[2]);

    const float scale = a.scale * LOG2E;
    bool goes_on = false;
    // LDS addresses of a lane's fragments: K's piece 2 ks + half of row col, V's
    // pieces of rows 4 half + (lane % 16) / 4 (+ 8) that hold its group's 16 of d
    // (the swizzle turns pieces within 16, so that the next 16 lie 256 bytes on)
    constexpr int KA = KS < 8 ? KS : 8;
    uint32_t k_addr[KA];
#pragma unroll
    for (int ks = 0; ks < KA; ++ks)
        k_addr[ks] = col * DP * 2 + ((2 * ks + half) ^ swizzle<DP>(col)) * 16;
    const uint32_t v_row = 4 * half + lane % 16 / 4, v_piece = 2 * (lane / 16 % 2) + lane % 4 / 2;
    uint32_t v_addr[2][DB];
#pragma unroll
    for (int jj = 0; jj < 2; ++jj)
#pragma unroll
        for (int db = 0; db < DB; ++db) {
            const uint32_t r = v_row + 8 * jj;
            v_addr[jj][db] = r * DP * 2 + ((4 * db + v_piece) ^ swizzle<DP>(r)) * 16 + lane % 2 * 8 + part_d * 2;
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
        const Block blk = block_of<KT>(a, q.n, q.len, row0, ROWS, group);
        const uint32_t off = (uint32_t)(x - unit);
        if (off >= blk.tiles)
            break;
        const uint32_t count = (uint32_t)min((uint64_t)(blk.tiles - off), share_end - x);
        const uint32_t rows = min(ROWS, (uint32_t)q.n * group - row0);

        // ---- the wave's rows
        const uint32_t first_row = row0 + 32 * strip, my_row = first_row + col;
        const bool wave_live = 32 * strip < rows, row_live = 32 * strip + col < rows;
        const int old = q.len - q.n;
        const int my_pos = old + (int)(my_row / group);
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
        float row_scale = FP8 ? 1.0f : scale;
        bool some_far = false;             // of the wave's rows
        uint32_t nans[CW / 8];             // bit 4 c + j: the row's d = part_d + 8 c + 4 half + j has met NaN or an infinity
#pragma unroll
        for (uint32_t i = 0; i < CW / 8; ++i)
            nans[i] = 0;
        f32x16 acc[DB];
#pragma unroll
        for (int db = 0; db < DB; ++db)
            acc[db] = (f32x16)0.0f;

        // ---- loads.  A wave's 64 pieces lie in one 16 keys, so in one page: its
        // address is scalar, the lane's part the same for every tile
        const uint32_t t_end = blk.first_tile + off + count;
        const int32_t *table = a.table + (size_t)seq * a.width;
        const uint32_t page_elems = (kv * d) << pl, head_elems = (head * d) << pl;   // of one page: below 2^31
        const uint32_t mask = (1u << pl) - 1;
        // the lane's bytes of those 16 rows: piece c of LDS row r holds piece
        // c ^ swizzle(r) of the head's row; what lies past d is zeros.  Row r % 16 is the
        // same for every second piece of a thread at least.
        constexpr uint32_t EB = FP8 ? 1 : 2;               // bytes of an element
        uint32_t lane_at[2];
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i) {
            const uint32_t it = tid + WG * i, r = it / CPR;
            const uint32_t e = FP8 ? it % CPR * 16 : (it % CPR ^ swizzle<DP>(r)) * 8;
            lane_at[i] = e < d ? (r % 16 * d + e) * EB : BEYOND;
        }
        u32x4 kr[FP8 ? ITEMS : 1], vr[FP8 ? ITEMS : 1];
        float ksr = 0.0f, vsr = 0.0f;
        // Where 1024 keys lie, in elements: lane i's are the 16 that begin 16 i behind the
        // first tile's (or 1024, 2048, ... further); and which of them are holes.
        uint32_t at_lo = 0, at_hi = 0, page_next = 0;
        uint64_t missing = 0, row_at = 0;                  // (the same in rows, for the scales)
        auto look = [&](uint32_t tile) {
            const uint32_t key = tile * KT + 16 * lane;
            page_next = key < (uint32_t)blk.to && tile < t_end ? (uint32_t)table[key >> pl] : ~0u;
        };
        // Starts a tile's loads; returns its 16s of keys that are holes, as bits.
        auto load = [&](uint32_t tile, uint8_t *kd, uint8_t *vd) {
            const uint32_t nth = (tile - (blk.first_tile + off)) % AHEAD_TILES;
            if (nth == 0) {
                const bool hole = page_next >= a.cache.pages;
                const uint64_t at = (uint64_t)(hole ? 0 : page_next) * page_elems + (head_elems + ((tile * KT + 16 * lane) & mask) * d);
                missing = __ballot(hole);
                at_lo = (uint32_t)at;
                at_hi = (uint32_t)(at >> 32);
                if (FP8)
                    row_at = (((hole ? 0 : page_next) * (uint64_t)kv + head) << pl) + ((tile * KT + 16 * lane) & mask);
                look(tile + AHEAD_TILES);
            }
            const uint32_t gaps = (uint32_t)(missing >> GROUPS * nth) & ((1u << GROUPS) - 1);
#pragma unroll
            for (uint32_t i = 0; i < ITEMS; ++i) {
                // the 16 keys that this wave's pieces are of
                constexpr uint32_t WAVE_ROWS = 64 / CPR;
                const uint32_t g = i * (WG / CPR) / 16 + (WAVE_ROWS * NW > 16 ? wave * WAVE_ROWS / 16 : 0);
                const uint64_t row = (uint64_t)(uint32_t)__builtin_amdgcn_readlane(at_hi, GROUPS * nth + g) << 32 |
                                     (uint32_t)__builtin_amdgcn_readlane(at_lo, GROUPS * nth + g);
                const uint32_t bytes = gaps >> g & 1 ? 0 : 16 * d * EB;                // a hole is read as zeros
                const __amdgpu_buffer_rsrc_t kp = window_at(a.cache.k, row * EB, bytes), vp = window_at(a.cache.v, row * EB, bytes);
                if constexpr (FP8) {
                    kr[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(kp, lane_at[i % 2], 0, 0));
                    vr[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(vp, lane_at[i % 2], 0, 0));
                } else {
                    const uint32_t to = 16 * (64 * wave + WG * i);
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(kp, (lds_void *)(kd + to), 16, lane_at[i % 2], 0, 0, 0);
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(vp, (lds_void *)(vd + to), 16, lane_at[i % 2], 0, 0, 0);
                }
            }
            if (FP8 && 64 * wave < KT) {
                // the first waves: a scale of K and of V each, of the keys' rows of the cache
                // (all lanes take part in the exchange: any may hold the row asked for)
                const uint64_t row = __shfl(row_at, GROUPS * nth + tid / 16, 64) + lane % 16;
                if (tid < KT) {
                    const bool hole = gaps >> tid / 16 & 1;
                    ksr = hole ? 0.0f : a.cache.ks[row];
                    vsr = hole ? 0.0f : a.cache.vs[row];
                }
            }
            return gaps;
        };
        auto store = [&](uint32_t buf, uint8_t *kd, uint8_t *vd) {
            const uint32_t tid = here(threadIdx.x);
#pragma unroll
            for (uint32_t i = 0; i < ITEMS; ++i) {
                const uint32_t it = tid + WG * i, r = it / CPR, c = it % CPR;
                if constexpr (FP8) {
#pragma unroll
                    for (uint32_t h = 0; h < 2; ++h) {
                        const uint32_t p = r * DP * 2 + ((2 * c + h) ^ swizzle<DP>(r)) * 16;
                        *(u32x4 *)(kd + p) = bf16_of_e4m3((u32x2){kr[i][2 * h], kr[i][2 * h + 1]});
                        *(u32x4 *)(vd + p) = bf16_of_e4m3((u32x2){vr[i][2 * h], vr[i][2 * h + 1]});
                    }
                }
            }
            if (FP8 && tid < KT) {
                scales[buf][0][tid] = ksr * scale;
                scales[buf][1][tid] = finite_scale(vsr);
            }
        };
        // One tile; masked: some of the wave's rows do not see some of its keys.
        auto step = [&](const uint8_t *kt, const uint8_t *vt, int k0, uint32_t buf, uint32_t gaps, bool masked, bool poisoned) {
            auto sees = [&](int k) { const int pos = my_pos; return k0 + k <= pos && (!a.window || (uint32_t)(pos - k0 - k) < a.window) && !(gaps >> (k / 16) & 1); };
            // ---- scores; a lane's are of keys 32 kb + 8 (i / 4) + 4 half + i % 4.  K's
            // fragments are read AHEAD products before they are used (the order is pinned:
            // left alone, each read is put right before its product)
            constexpr int AHEAD = 4;
            constexpr int KB = KT / 32;
            f32x16 s[KB];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
                s[kb] = (f32x16)0.0f;
            bf16x8 kf[AHEAD];
            auto k_frag = [&](int n) { return *(const bf16x8 *)(kt + n % KB * 32 * DP * 2 + k_addr[n / KB % KA] + n / KB / KA * 256); };
#pragma unroll
            for (int n = 0; n < AHEAD; ++n)
                kf[n] = k_frag(n);
#pragma unroll
            for (int n = 0; n < KB * KS; ++n) {
                __builtin_amdgcn_sched_barrier(0);
                s[n % KB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[n % AHEAD], qf[n / KB], s[n % KB], 0, 0, 0);
                if (n + AHEAD < KB * KS)
                    kf[n % AHEAD] = k_frag(n + AHEAD);
            }
            __builtin_amdgcn_sched_barrier(0);
            const float unit_scale = FP8 ? 1.0f : scale;
            if constexpr (FP8) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const f32x4 z = *(const f32x4 *)&scales[buf][0][32 * kb + 2 * i + 4 * half];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            s[kb][i + j] *= z[j];
                    }
            }
            if (masked) {
                // key c of the tile is seen if it is 0 to span before the row's own
                const int own = (int)here(my_pos) - k0 - 4 * (int)half;
                const uint32_t span = a.window ? min(a.window - 1, 0x7FFFFFFFu) : 0x7FFFFFFFu;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x = (uint32_t)(own - (32 * kb + 8 * (i / 4) + i % 4)) <= span ? s[kb][i] : -INFINITY;
                        if (gaps >> (2 * kb + i / 8) & 1)
                            x = -INFINITY;
                        asm volatile("" : "+v"(x));     // computed in this branch alone
                        s[kb][i] = x;
                    }
            }
            // ---- probabilities
            float top = -INFINITY;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int i = 0; i < 16; i += 2)
                    top = __builtin_fmaxf(__builtin_fmaxf(top, s[kb][i]), s[kb][i + 1]);
            top *= unit_scale;
            if (__any(top > m + 8.0f)) {
                // (rows whose own has not grown keep theirs: none depends on keys that it does not see)
                top = __builtin_fmaxf(top, __shfl_xor(top, 32, 64));
                top = top > m + 8.0f ? top : m;
                const float to = top == -INFINITY ? 0.0f : top;
                const float fade = __builtin_amdgcn_exp2f(m - to);
                m = top;
                base = to;
                row_scale = !FP8 && far(base) ? 1.0f : unit_scale;
                some_far = __any(far(base));
                l *= fade;
#pragma unroll
                for (int db = 0; db < DB; ++db)
                    acc[db] *= fade;
            }
            if (!FP8 && some_far) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x = far(base) ? s[kb][i] * scale : s[kb][i];
                        asm volatile("" : "+v"(x));
                        s[kb][i] = x;
                    }
            }
            // ---- V: 16 keys' probabilities, then their products with every 32 of d; under
            // these the next 16 keys' probabilities and V's fragments
            // (this wave before the SIMD's other, whose scores and masks then fill the gaps: 3% faster at
            // heads of 64 with a window of 1024, 1.5% at 2000 rows over 32000)
            __builtin_amdgcn_s_setprio(1);
            float part[4] = {0, 0, 0, 0};
            auto probability = [&](int blk, int i) {
                const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[blk / 2][8 * (blk % 2) + i], row_scale, -base));
                part[i % 4] += p;
                return FP8 ? p * scales[buf][1][16 * blk + 8 * (i / 4) + 4 * half + i % 4] : p;
            };
            auto v_frag = [&](int blk, int db) {
                u32x4 v;
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    const uint8_t *p = vt + 16 * blk * DP * 2 + v_addr[jj][db];
                    const u32x2 t = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
                    v[2 * jj] = t[0];
                    v[2 * jj + 1] = t[1];
                }
                return v;
            };
            constexpr int VN = 2 * KB * DB, VR = DB;                    // products; V's fragments in flight
            u32x4 vf[VR], pf, pn;
#pragma unroll
            for (int n = 0; n < VR; ++n)
                vf[n] = v_frag(0, n);
            // rounded to BF16, the operand's type, by up to 2^-8 of each: 0.0023 from 64 bits in the 2-norm
            // where the output's own rounding is 0.0017.  The remainders' products as well, which
            // few rows take, would be half as many matrix operations again, which bound this kernel
#pragma unroll
            for (int i = 0; i < 4; ++i)
                pf[i] = pk_bf16(probability(0, 2 * i), probability(0, 2 * i + 1));
#pragma unroll
            for (int n = 0; n < VN; ++n) {
                const int blk = n / DB, db = n % DB;
                __builtin_amdgcn_sched_barrier(0);
                acc[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vf[n % VR]),
                                                                  __builtin_bit_cast(bf16x8, pf), acc[db], 0, 0, 0);
                if (n + VR < VN)
                    vf[n % VR] = v_frag((n + VR) / DB, (n + VR) % DB);
                if (blk < 2 * KB - 1)
#pragma unroll
                    for (int i = 4 * db / DB; i < 4 * (db + 1) / DB; ++i)
                        pn[i] = pk_bf16(probability(blk + 1, 2 * i), probability(blk + 1, 2 * i + 1));
                if (db == DB - 1)
                    pf = pn;
            }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(0);
            l += (part[0] + part[1]) + (part[2] + part[3]);
            if (poisoned) {
                // NaN and infinities, in whose places V has zeros, for the rows that see them
#pragma unroll 1
                for (int k = 0; k < (int)KT; ++k)
                    if (sees(k)) {
#pragma unroll
                        for (uint32_t c = 0; c < CW; ++c)
                            nans[c / 8] |= (odd_bits[k][part_d / 8 + c] >> 4 * half & 15u) << (4 * (c % 8));
                    }
            }
        };

        uint32_t tile = blk.first_tile + off;
        const int block_lo = old + (int)(row0 / group), block_hi = old + (int)((row0 + rows - 1) / group);
        look(tile);
        __syncthreads();                   // the last unit's tiles have been read
        uint32_t gaps_next = load(tile, k_lds0, v_lds0);
        // (under the first loads)
        if (off + count < blk.tiles) {
            goes_on = true;
            const uint32_t last = min(share_of(unit + blk.tiles - 1, total, shares), (uint32_t)shares - 1);
            if (tid == 0)
                parts.begun[w] = {off == 0 ? (int)w : (int)share_of(unit, total, shares), (int)last, q.token, (int)row0, (int)rows, (int)head, {0, 0}};
        }
        store(0, k_lds0, v_lds0);
        // A tile from one buffer while the next comes to the other.
        auto turn = [&](uint32_t buf, const uint8_t *kt, uint8_t *vt, uint8_t *k_next, uint8_t *v_next) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            const bool more = tile + 1 < t_end;
            const uint32_t gaps = gaps_next;
            if (more)
                gaps_next = load(tile + 1, k_next, v_next);
            const int k0 = tile * KT;
            uint32_t poisoned = 0;
            if (k0 + (int)KT - 1 > block_lo || (a.window && k0 <= block_hi - (int64_t)a.window) || gaps) {
                // some row of the block does not see some key, and 0 times NaN would be NaN
                uint32_t bad = 0;
#pragma unroll 2
                for (uint32_t i = here(threadIdx.x); i < KT * CH; i += WG) {
                    const u32x4 v = *(const u32x4 *)(vt + 16 * i);
                    bad |= odd_tops(v[0]) | odd_tops(v[1]) | odd_tops(v[2]) | odd_tops(v[3]);
                }
                const bool any = __any(bad != 0);
                if (lane == 0)
                    odd[wave] = any;
                __syncthreads();
                uint32_t some = 0;
                for (uint32_t u = 0; u < NW; ++u)
                    some |= odd[u];
                poisoned = uniform(some);
                if (poisoned) {
                    // those of V go, and are noted for the rows that see them
                    for (uint32_t i = here(threadIdx.x); i < KT * CH; i += WG) {
                        u32x4 v = *(const u32x4 *)(vt + 16 * i);
                        uint32_t bits = 0;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t z = not_finite(v[j]);
                            bits |= (z & 1) << (2 * j) | (z >> 31) << (2 * j + 1);
                            v[j] &= ~z;
                        }
                        const uint32_t r = i / CH;
                        odd_bits[r][i % CH ^ swizzle<DP>(r)] = bits;
                        *(u32x4 *)(vt + 16 * i) = v;
                    }
                    __syncthreads();
                }
            }
            const bool none = !wave_live || k0 > pos_hi || (a.window && k0 + (int)KT - 1 <= pos_lo - (int64_t)a.window);
            const bool whole = k0 + (int)KT - 1 <= pos_lo && (!a.window || k0 > pos_hi - (int64_t)a.window) && gaps == 0;
            const int way = uniform(none ? 0u : whole ? 1u : 2u);
            if (way != 0)
                step(kt, vt, k0, buf, gaps, way == 2, poisoned != 0);
            if (more)
                store(buf ^ 1, k_next, v_next);
            ++tile;
        };
        while (true) {
            turn(0, k_lds0, v_lds0, k_lds1, v_lds1);
            if (tile >= t_end)
                break;
            turn(1, k_lds1, v_lds1, k_lds0, v_lds0);
            if (tile >= t_end)
                break;
        }

        // ---- the rows' results: a lane holds d = 32 db + 8 (i / 4) + 4 half + i % 4 of row col
        l += __shfl_xor(l, 32, 64);
        const bool begins = off == 0, finished = count == blk.tiles;
        if (row_live) {
            const size_t slot = (2 * (size_t)w + begins) * ROWS + 32 * strip + col;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            if (!finished && half == 0 && part_d == 0)
                parts.ml[slot] = (f32x2){m, l};
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const uint32_t e = part_d + 32 * db + 2 * i + 4 * half;
                    if (e >= d)
                        continue;
                    f32x4 v = {acc[db][i], acc[db][i + 1], acc[db][i + 2], acc[db][i + 3]};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = nans[db / 2] >> (16 * (db % 2) + i + j) & 1 ? __builtin_nanf("") : v[j];
                    if (finished)
                        *(u32x2 *)(a.out + q_at + e) = (u32x2){pk_bf16(v[0] * inv, v[1] * inv), pk_bf16(v[2] * inv, v[3] * inv)};
                    else
                        *(f32x4 *)(parts.o + slot * d + e) = v;
                }
        }
        x += count;
        if (x == unit + blk.tiles) {
            unit = x;
            row0 += ROWS;
        }
    }
    if (!goes_on && tid == 0)
        parts.begun[w] = {0, -1, 0, 0, 0, 0, {0, 0}};
}

template <int DP, int NW>
void launch(const AttnArgs &a, const Parts &p, uint32_t shares, hipStream_t st)
{
    if (a.cache.fp8)
        k_attn_tiles<DP, NW, true><<<shares, 64 * NW, 0, st>>>(a, p, shares);
    else
        k_attn_tiles<DP, NW, false><<<shares, 64 * NW, 0, st>>>(a, p, shares);
}

// Waves of a workgroup.  Eight read K and V half as often as four; at d <= 64 two
// workgroups of four fit side by side, so that one's start and barriers are the
// other's time to work, which counts where units are short.  Measured there, four
// waves and eight, 64 heads on 8, us: 32 prompts of 128 42 and 53; 8 of 512 83 and
// 76, 1 of 4096 275 and 270, 7 of 250 to 2500 in a window of 1024 276 and 265.
uint32_t waves_of(uint32_t d, uint32_t max_q) { return d <= 64 && max_q <= 256 ? 4 : 8; }

// Rows of a unit (two waves share them for d > 128).
uint32_t unit_rows(uint32_t d, uint32_t max_q) { return 32 * waves_of(d, max_q) / (d <= 128 ? 1 : 2); }

// As many workgroups as the chip holds at a time.
uint32_t max_shares(uint32_t d, uint32_t max_q)
{
    return 8 / waves_of(d, max_q) * (cu_count() ? cu_count() : 256);
}

} // namespace

uint64_t tiles_work(uint32_t d)
{
    // enough for any max_q: what serves a large one serves a smaller
    return max(parts_bytes(max_shares(d, 1), unit_rows(d, 1), d), parts_bytes(max_shares(d, ~0u), unit_rows(d, ~0u), d));
}

hipError_t launch_attn_tiles(const AttnArgs &a, hipStream_t st)
{
    const uint32_t d = a.cache.d, shares = max_shares(d, a.max_q), rows = unit_rows(d, a.max_q);
    const Parts p = parts_at(a.work, shares, rows);
    if (waves_of(d, a.max_q) == 4)
        launch<64, 4>(a, p, shares, st);
    else if (d <= 64)
        launch<64, 8>(a, p, shares, st);
    else if (d <= 128)
        launch<128, 8>(a, p, shares, st);
    else
        launch<256, 8>(a, p, shares, st);
    count_launch();
    if (hipError_t e = hipGetLastError())
        return e;
    return launch_attn_join(a, p, shares, rows, rows, st);
}

} // namespace attn
} // namespace qp
