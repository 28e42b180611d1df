// gemm_fp8_block.hip -- block-scaled FP8 GEMM:
//
//   C[i,j] = bf16( sum_b as[i,b] * ws[j/128,b] * P_b[i,j] ),
//   P_b[i,j] = sum_{t in block b} e4m3(a[i,t]) * e4m3(w[j,t]),  128 K per block.
//
// P_b is formed on the matrix core in F32 from zero; as[i,b] * ws[j/128,b] is
// one F32 product per row and block, and acc += P_b * that one FMA per output
// and block on the vector ALU.
//
// The MFMAs compute C^T tiles (W fragment as the first operand): a lane then
// holds one row of C, so its scale is one value per lane and block and needs
// no broadcast.
#include "gemm_common.hpp"
#include "qp_launch.hpp"
#include "../../include/qproj_layer.h"
#include <algorithm>
#include <type_traits>

namespace qp {
namespace {

// ---------------------------------------------------------------------------
// Large tiles: MW x NW waves, each 64 rows of A by 16*TJ rows of W, as 4 x TJ
// MFMAs v_mfma_f32_16x16x128 per K block: one instruction is one whole P_b of
// a 16 x 16 tile, so P_b costs four registers for a moment and its fold, four
// FMAs, runs under the next tiles' MFMAs.  The running sums stay in ordinary
// registers (the vector ALU cannot reach accumulator registers), which caps a
// wave at 64 x 128; two waves share a SIMD so that one's folds, LDS reads and
// waits run under the other's MFMAs.
//
// Operand panels of one K block (128 bytes per row of A or of W) arrive by
// 16-byte buffer loads to LDS, swizzled as in gemm_common.hpp, into a ring of
// five slots: panel i of A0, W0, A1, W1, ... in slot i % 5.  A block's A
// fragments are all in registers soon after it starts, its W fragments at
// three quarters of it; each time a barrier says so and the slot is refilled
// at once, W two blocks ahead and A three, so that a panel has 1.65 to 2
// blocks' time to come (with one block's time, 475 against 371 us without any
// loads; 8192 x 12288 x 5120).
// Rows past M or N lie past the buffer and read as zeros, so tiles at the
// edges need no clamping; where 128 does not divide K (TAIL), both operands'
// chunks past K are given an offset past the buffer (A's zeros alone would not
// do: W's row goes on with the next row, which may hold a NaN); a live row's
// offset on top leaves it past the buffer, a row past M or N is never stored.
// Where 128 divides K, W's loads go without the select: 512 x 5120 x 17408 94.4
// us, with it 95.4.
//
// The scales of five K blocks are loaded at once: lane l holds as * ws of its
// wave's row l for each; a block's four values per lane (its rows 16t + l%16)
// come from three lane swaps.
//
// Measured: 8192 x 12288 x 5120: 445 to 490 us from box to box, 2.1 to 2.3
// PFLOP/s; 4096 x 5120 x 17408: 327 to 340 us, 2.2; 600 x 4104 x 2368 (128 x 128
// tiles): 15.0 us.  Bound by issue and power: the MFMAs take 57% of the cycles and the vector ALU 48%, four of its
// 6.7 instructions per MFMA being the fold, at a shader clock of 1.77 GHz.
// ---------------------------------------------------------------------------
constexpr uint32_t FB_OOB = 0x80000000u;

// C's rows start at any multiple of 2 bytes, which global stores allow.
typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4_any;
typedef __attribute__((ext_vector_type(2), aligned(2))) uint32_t u32x2_any;

// s_waitcnt immediates: vmcnt <= n alone, lgkmcnt == 0 alone
constexpr int waitcnt_vm(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }
constexpr int WAIT_LGKM0 = 15 | (7 << 4) | (3 << 14);

__device__ __forceinline__ __amdgpu_buffer_rsrc_t fb_rsrc(const void *p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, 0x00020000);
}

// v's four rows of 16 lanes, each spread over all four.
__device__ __forceinline__ void spread_rows(float v, float *s)
{
    const uint32_t u = __float_as_uint(v);
    const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const auto a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
    s[0] = __uint_as_float(a[0]);
    s[1] = __uint_as_float(a[1]);
    s[2] = __uint_as_float(b[0]);
    s[3] = __uint_as_float(b[1]);
}

template <int MW, int NW, int TJ, bool TAIL>
__global__ __launch_bounds__(64 * MW * NW) void k_fp8_gemm_block_tiles(
    const uint8_t *__restrict__ A, const float *__restrict__ as,
    const uint8_t *__restrict__ W, const float *__restrict__ ws,
    uint16_t *__restrict__ out, uint32_t M, uint32_t N, uint32_t K,
    uint32_t mtiles, uint32_t ntiles, uint32_t first, uint32_t quarters)
{
    constexpr int NWV = MW * NW, TM = 64 * MW, TN = 16 * TJ * NW;
    constexpr int AL = TM / 8 / NWV, WL = TN / 8 / NWV;     // DMA loads per wave and stage
    static_assert(TM / 8 % NWV == 0 && TN / 8 % NWV == 0 && AL % 2 == 0 && WL % 2 == 0, "whole DMA");
    static_assert(128 % (16 * TJ) == 0 && TN % 128 == 0, "a wave's columns share a scale block");
    constexpr int SLOT = (TM > TN ? TM : TN) * BIG_KB;
    // separate variables: see gemm_fp8.hip
    __shared__ __attribute__((aligned(1024))) uint8_t S0[SLOT];
    __shared__ __attribute__((aligned(1024))) uint8_t S1[SLOT];
    __shared__ __attribute__((aligned(1024))) uint8_t S2[SLOT];
    __shared__ __attribute__((aligned(1024))) uint8_t S3[SLOT];
    __shared__ __attribute__((aligned(1024))) uint8_t S4[SLOT];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % MW, wn = wave / MW;
    // Tiles first .. of the banded order, or, with `quarters`, four workgroups
    // to each of them, one for each quarter of a tile twice as long and wide.
    uint32_t tm, tn, id = xcd_remap(blockIdx.x, gridDim.x);
    banded_tile(first + (quarters ? id / 4 : id), mtiles, ntiles, tm, tn);
    if (quarters) {
        tm = 2 * tm + (id & 1);
        tn = 2 * tn + (id >> 1 & 1);
    }
    const uint32_t m0 = tm * TM, n0 = tn * TN;
    if (m0 >= M || n0 >= N)
        return;                          // a quarter past the edge
    const uint32_t nst = (K + 127) / 128;

    const __amdgpu_buffer_rsrc_t ra = fb_rsrc(A, M * K), rw = fb_rsrc(W, N * K);
    const __amdgpu_buffer_rsrc_t ras = fb_rsrc(as, M * nst * 4);

    // DMA: load j of wave w fills kilobyte L*w + j of a slot, rows 8(Lw+j) +
    // lane/8; the lane's physical chunk lane%8 takes logical chunk
    // (lane%8) ^ ((row/2) % 8) of its row.
    // The three lane offsets everything else follows from are hidden from the
    // compiler once per block (launder): it would keep every sum of them and a
    // row's or a slot's address in a register of its own across the loop.
    const int r16 = lane & 15, g = lane >> 4;
    uint32_t dcol = 16u * ((lane & 7) ^ (lane >> 4)), drow = (uint32_t)(lane >> 3) * K;
    uint32_t f0 = r16 * BIG_KB + 16 * (g ^ ((r16 >> 1) & 7));
    auto launder = [&]() { asm volatile("" : "+v"(dcol), "+v"(drow), "+v"(f0)); };
    // loads [lo, hi) of a panel's AL (WL) per wave
    auto dma_a = [&](uint32_t st, uint8_t *slot, int lo, int hi) {
        const uint32_t k0 = st * 128;
#pragma unroll
        for (int j = lo; j < hi; ++j) {
            const uint32_t c = k0 + (j & 1 ? dcol ^ 64 : dcol);
            const uint32_t o = c < K ? drow + c : FB_OOB;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void *)(slot + 1024 * (AL * wave + j)), 16,
                                                     o + (m0 + 8 * (AL * wave + j)) * K, 0, 0, 0);
        }
    };
    auto dma_w = [&](uint32_t st, uint8_t *slot, int lo, int hi) {
        const uint32_t k0 = st * 128;
#pragma unroll
        for (int j = lo; j < hi; ++j) {
            const uint32_t c = k0 + (j & 1 ? dcol ^ 64 : dcol);
            const uint32_t o = !TAIL || c < K ? drow + c : FB_OOB;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void *)(slot + 1024 * (WL * wave + j)), 16,
                                                     o + (n0 + 8 * (WL * wave + j)) * K, 0, 0, 0);
        }
    };

    // Fragment of 16 rows: lane l takes row l%16 and chunks l/16 and l/16 + 4
    // (both operands in the same order, so the sum over K is whole).
    auto frag = [&](const uint8_t *rows16) {
        const i32x4 p = *reinterpret_cast<const i32x4 *>(rows16 + f0);
        const i32x4 q = *reinterpret_cast<const i32x4 *>(rows16 + (f0 ^ 64));
        return (i32x8){p[0], p[1], p[2], p[3], q[0], q[1], q[2], q[3]};
    };
    auto frag_a = [&](const uint8_t *slot, int t) { return frag(slot + (wm * 64 + 16 * t) * BIG_KB); };
    auto frag_w = [&](const uint8_t *slot, int t) { return frag(slot + (wn * 16 * TJ + 16 * t) * BIG_KB); };

    // A's scales of five blocks from b on, of the wave's row `lane` (past the
    // end of the row: values of no use; past the buffer: zeros), and their
    // products with the weight's
    struct Scales {
        f32x4 v;
        float l;
    };
    const uint32_t oas = (m0 + wm * 64 + lane) * nst * 4;
    auto load_scales = [&](uint32_t b) {
        Scales s;
        s.v = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(ras, oas + 4 * b, 0, 0));
        s.l = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(ras, oas + 4 * b + 16, 0, 0));
        return s;
    };
    const float *const wsr = ws + (size_t)min((n0 + wn * 16 * TJ) / 128, (N - 1) / 128) * nst;
    auto times_ws = [&](Scales s, uint32_t b) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s.v[i] *= wsr[min(b + i, nst - 1)];
        s.l *= wsr[min(b + 4, nst - 1)];
        return s;
    };

    f32x4 acc[4][TJ];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j)
            acc[i][j] = (f32x4){0, 0, 0, 0};

    i32x8 a[4], w0;
    auto mfma = [&](const i32x8 &w, const i32x8 &x) {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, (f32x4){0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
    };
    auto fold = [&](f32x4 &c, const f32x4 &p, float s) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            c[r] = __builtin_fmaf(p[r], s, c[r]);
    };
    // One K block: a[] and w0 hold its first fragments.  Its MFMAs run in the
    // order j = 0 .. TJ-3, t = 0 .. 3, then t = 0 .. 3, j = TJ-2, TJ-1; the
    // fold of each follows the fourth MFMA after it (from one block into the
    // next), so no fold waits for its own.  After j = 0 a barrier: A's slot is
    // read out and takes W(st+2).  After the last LDS read every wave waits for
    // its part of the next block's panels, then for all waves; W's slot takes
    // A(st+3), and the last eight MFMAs run while the next block's fragments
    // replace a[].
    constexpr int LAG = 4, NM = 4 * TJ;
    f32x4 p[LAG];
    float sp[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < LAG; ++i)
        p[i] = (f32x4){0, 0, 0, 0};
    constexpr auto tile_t = [](int i) { return i < NM - 8 ? i % 4 : (i - (NM - 8)) / 2; };
    constexpr auto tile_j = [](int i) { return i < NM - 8 ? i / 4 : TJ - 2 + i % 2; };
    Scales sq, sn;
    auto stage = [&](auto in_five, uint32_t st, uint8_t *ca, uint8_t *cw, const uint8_t *na, const uint8_t *nw) {
        constexpr int I5 = decltype(in_five)::value;
        const float s64 = I5 == 4 ? sq.l : sq.v[I5 & 3];
        float s[4];
        launder();
        spread_rows(s64, s);
        auto step = [&](int i, const i32x8 &wf) {
            const int f = i < LAG ? NM - LAG + i : i - LAG;
            const float sf = i < LAG ? sp[tile_t(f)] : s[tile_t(f)];
            const f32x4 old = p[i % LAG];
            p[i % LAG] = mfma(wf, a[tile_t(i)]);
            fold(acc[tile_t(f)][tile_j(f)], old, sf);
        };
        i32x8 w[TJ];
        w[0] = w0;
#pragma unroll
        for (int j = 0; j < TJ - 2; ++j) {
            w[j + 1] = frag_w(cw, j + 1);
            if (j == TJ - 3)
                w[TJ - 1] = frag_w(cw, TJ - 1);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                step(4 * j + t, w[j]);
                if (j == 1) {
                    // one load of the refill under each MFMA: the address unit
                    // holds a burst of them, and the wave behind it
                    dma_w(st + 2, ca, t * WL / 4, (t + 1) * WL / 4);
                    if (t == 0)
                        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
                    __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (j != 1) {
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                if (j == TJ - 3)
                    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (j == 0) {
                // (a[] has been waited for by its MFMAs)
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // A(st+2) and W(st+2) may stay in flight.  Nothing is allowed for the
        // scales' loads: the compiler may move those or drop them, and a
        // count that expects them would then let the next panels be late.
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(AL + WL));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if (I5 == 0)
            sn = load_scales(st + 5);
        if (I5 == 4)
            sq = times_ws(sn, st + 1);
        w0 = frag_w(nw, 0);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            step(NM - 8 + 2 * t, w[TJ - 2]);
            step(NM - 8 + 2 * t + 1, w[TJ - 1]);
            a[t] = frag_a(na, t);
            dma_a(st + 3, cw, t * AL / 4, (t + 1) * AL / 4);
            __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            if (t == 0)
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 13, 0);
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
            sp[t] = s[t];
    };

    sq = load_scales(0);
    dma_a(0, S0, 0, AL);
    dma_w(0, S1, 0, WL);
    dma_a(1, S2, 0, AL);
    dma_w(1, S3, 0, WL);
    dma_a(2, S4, 0, AL);
    sq = times_ws(sq, 0);
    sn = sq;
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(2 * AL + WL));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    w0 = frag_w(S1, 0);
#pragma unroll
    for (int t = 0; t < 4; ++t)
        a[t] = frag_a(S0, t);
    // (a loop left in its middle would join its exits with its back edge, and
    // the compiler then waits for every load in flight at its head)
    uint32_t st = 0;
    for (; st + 5 <= nst; st += 5) {
        stage(std::integral_constant<int, 0>(), st, S0, S1, S2, S3);
        stage(std::integral_constant<int, 1>(), st + 1, S2, S3, S4, S0);
        stage(std::integral_constant<int, 2>(), st + 2, S4, S0, S1, S2);
        stage(std::integral_constant<int, 3>(), st + 3, S1, S2, S3, S4);
        stage(std::integral_constant<int, 4>(), st + 4, S3, S4, S0, S1);
    }
    if (st < nst)
        stage(std::integral_constant<int, 0>(), st, S0, S1, S2, S3);
    if (st + 1 < nst)
        stage(std::integral_constant<int, 1>(), st + 1, S2, S3, S4, S0);
    if (st + 2 < nst)
        stage(std::integral_constant<int, 2>(), st + 2, S4, S0, S1, S2);
    if (st + 3 < nst)
        stage(std::integral_constant<int, 3>(), st + 3, S1, S2, S3, S4);
#pragma unroll
    for (int i = 0; i < LAG; ++i)
        fold(acc[tile_t(NM - LAG + i)][tile_j(NM - LAG + i)], p[i], sp[tile_t(NM - LAG + i)]);
    // the loads past the end must land before the slots are used again
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
    __syncthreads();

    // Lane l holds, of tile (t, j), row 16t + l%16 and columns 16j + 4(l/16) .. +3.
    const uint32_t rb = m0 + wm * 64, cb = n0 + wn * 16 * TJ;
    // Stage the wave's 64 x 16TJ block in LDS (RB = 32TJ bytes per row;
    // 8-byte unit u of row r at u ^ x(r), so that 16 rows' writes spread over
    // the banks) and store it in whole rows, 16 bytes per lane.
    constexpr int RB = 32 * TJ, UN = RB / 8, PU = RB / 16, RPI = 64 / PU;
    constexpr int OWN = 64 * RB;                       // this wave's bytes
    constexpr int PS = SLOT / OWN;                     // waves per slot
    static_assert(PS >= 1 && NWV <= 5 * PS, "fits");
    const int es = wave / PS;
    uint8_t *const ep = (es == 0 ? S0 : es == 1 ? S1 : es == 2 ? S2 : es == 3 ? S3 : S4) + wave % PS * OWN;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const f32x4 &c = acc[t][j];
            const u32x2 v = {pk_bf16(c[0], c[1]), pk_bf16(c[2], c[3])};
            const int r = 16 * t + r16;
            *reinterpret_cast<u32x2 *>(ep + r * RB + 8 * ((4 * j + g) ^ (2 * (r & (UN / 2 - 1))))) = v;
        }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int pu = lane % PU;
    const uint32_t col = cb + 8 * pu;
    auto row = [&](int it) { return RPI * it + lane / PU; };
    auto chunk = [&](int r) {
        return *reinterpret_cast<const u32x4 *>(ep + r * RB + 16 * (pu ^ (r & (UN / 2 - 1))));
    };
    if (N % 8 == 0) {
#pragma unroll 4
        for (int it = 0; it < 64 / RPI; ++it) {
            const int r = row(it);
            const u32x4 v = chunk(r);
            if (rb + r < M && col < N)
                *reinterpret_cast<u32x4 *>(out + (size_t)(rb + r) * N + col) = v;
        }
        return;
    }
    // Rows of C are aligned to 2 bytes only.  Global stores need no more; element
    // by element 7218 x 1641 x 384 took 31.7 us, where this takes 13.4.
    const uint32_t live = col < N ? min(N - col, 8u) : 0;
#pragma unroll 4
    for (int it = 0; it < 64 / RPI; ++it) {
        const int r = row(it);
        const u32x4 v = chunk(r);
        uint16_t *const to = out + (size_t)(rb + r) * N + col;
        if (rb + r >= M)
            continue;
        if (live == 8)
            *reinterpret_cast<u32x4_any *>(to) = v;
        else
            for (uint32_t i = 0; i < live; ++i)        // the row's last chunk
                to[i] = (uint16_t)(v[i / 2] >> 16 * (i % 2));
    }
}

// ---------------------------------------------------------------------------
// Small tiles, K split over the waves: 16*MT rows of A by rpw <= 16*NT rows of
// W per workgroup (rpw a multiple of 4, so that a problem's columns can be
// dealt evenly over the CUs), for problems with too few large tiles to fill
// them.  The waves take runs of four K blocks in turn (512 bytes of a row, some
// of it in flight at once: 28.2 us against 29.0 with single blocks in turn, 28.9
// with runs of eight; 37 x 5120 x 17408), or single ones where there is at most
// one for each (75 x 4224 x 224: 6.1 against 7.4 when that came in, 4.3 with the
// choice of rows that followed); each wave DMAs its blocks' panels into its own ring of D slots and waits for nothing but its own loads, so there is
// no barrier until the NW partial tiles are joined through LDS, in wave order.
// (Fragments loaded straight to registers, 16 rows of 64 bytes to an
// instruction, were half as fast: 8 rows of whole 128-byte lines are what the
// address unit and HBM serve best.)
// Scales come four of the wave's blocks at a time, lane group g (quad lane
// l%4) holding the g-th's: a load touches a cache line per row of A, and a line
// holds many blocks' scales.
//
// Bound by W's way from HBM and, behind that, the waves' own work on a block,
// which overlap in part: 37 x 5120 x 17408 takes 28 us, with W in the caches
// (the same instructions) 17; the bytes alone 14.5.  4 x 17408 x 5120: 16.4 us,
// 5.4 TB/s; 16 x 152064 x 5120: 129 to 136 us, 5.8 to 6.1 TB/s.
// ---------------------------------------------------------------------------
template <int MT, int NT, int NW, int D, bool ONCE>
__global__ __launch_bounds__(64 * NW) void k_fp8_gemm_block_ksplit(
    const uint8_t *__restrict__ A, const float *__restrict__ as,
    const uint8_t *__restrict__ W, const float *__restrict__ ws,
    uint16_t *__restrict__ out, uint32_t M, uint32_t N, uint32_t K, uint32_t mtiles, uint32_t rpw)
{
    static_assert(D == 2 || D == 3, "ring");
    constexpr int L = 2 * (MT + NT), SLOT = 1024 * L;      // DMA loads and bytes of a block
    // one variable per ring position: see gemm_fp8.hip
    __shared__ __attribute__((aligned(1024))) uint8_t R0[NW * SLOT];
    __shared__ __attribute__((aligned(1024))) uint8_t R1[NW * SLOT];
    __shared__ __attribute__((aligned(16))) uint8_t R2[D > 2 ? NW * SLOT : 16];
    // (positions past D are never named, so their variables take no LDS)
    auto ring = [&](int d) -> uint8_t * {
        if constexpr (D > 2)
            if (d == 2)
                return R2;
        return d == 1 ? R1 : R0;
    };
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // workgroups that share W's rows are neighbours behind one L2
    const uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
    const uint32_t m0 = id % mtiles * (16 * MT), n0 = id / mtiles * rpw;
    const uint32_t nb = (K + 127) / 128;
    const __amdgpu_buffer_rsrc_t ra = fb_rsrc(A, M * K), rw = fb_rsrc(W, N * K);
    const __amdgpu_buffer_rsrc_t ras = fb_rsrc(as, M * nb * 4);
    const __amdgpu_buffer_rsrc_t rws = fb_rsrc(ws, (N + 127) / 128 * nb * 4);

    // 1 KB = 8 rows x 128 bytes per load, chunks swizzled as in gemm_common.hpp
    const uint32_t dcol = 16u * ((lane & 7) ^ (lane >> 4)), drow = lane >> 3;
    const uint32_t oa = (m0 + drow) * K, ow = (n0 + drow) * K;
    auto dma = [&](uint32_t b, uint8_t *r) {
        uint8_t *const slot = r + wave * SLOT;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const bool of_a = j < 2 * MT;
            const int q = of_a ? j : j - 2 * MT;
            const uint32_t c = b * 128 + (q & 1 ? dcol ^ 64 : dcol);
            const uint32_t o = (of_a ? oa : ow) + 8 * q * K + c;
            if (of_a)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void *)(slot + 1024 * j), 16,
                                                         c < K ? o : FB_OOB, 0, 0, 0);
            else                         // (aux 2: nontemporal)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void *)(slot + 1024 * j), 16,
                                                         c < K && drow + 8 * q < rpw ? o : FB_OOB, 0, 0, ONCE ? 2 : 0);
        }
    };
    // the wave's i-th block; past the last: blocks past K, which are zeros
    const uint32_t rlog = nb > NW ? 2 : 0, rlen = 1u << rlog;
    auto nth = [&](uint32_t i) { return (i >> rlog) * (rlen * NW) + rlen * wave + (i & (rlen - 1)); };
    // raw scales of the wave's blocks i .. i+3: a[t] of row 16t + l%16 and block
    // i + l/16, w[j] of rows 16j + 4(l/16) .. +3 and block i + l%4
    struct Scales {
        float a[MT], w[NT];
    } next;
    auto load_scales = [&](uint32_t i) {
        const uint32_t ba = nth(i + g), bw = nth(i + (lane & 3));
#pragma unroll
        for (int t = 0; t < MT; ++t)
            next.a[t] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                ras, ba < nb ? ((m0 + 16 * t + r16) * nb + ba) * 4 : FB_OOB, 0, 0));
#pragma unroll
        for (int j = 0; j < NT; ++j)
            next.w[j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                rws, bw < nb ? ((n0 + 16 * j + 4 * g) / 128 * nb + bw) * 4 : FB_OOB, 0, 0));
    };
    const uint32_t f0 = r16 * BIG_KB + 16 * (g ^ ((r16 >> 1) & 7));
    f32x4 acc[MT][NT] = {};
    float sa[MT][4], sw[NT];
    auto block = [&](auto u_, uint32_t i) {
        constexpr int U = decltype(u_)::value, Q = U % 4;
        const uint8_t *const slot = ring(U % D) + wave * SLOT;
        if (Q == 0) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
                spread_rows(next.a[t], sa[t]);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                sw[j] = next.w[j];
            load_scales(i + 4);
        }
        // all but the D - 1 newest blocks' panels have landed (the scales'
        // loads are not counted on: the compiler may move them)
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(waitcnt_vm((D - 1) * L));
        __builtin_amdgcn_sched_barrier(0);
        i32x8 f[MT + NT];
#pragma unroll
        for (int e = 0; e < MT + NT; ++e) {
            const i32x4 p = *reinterpret_cast<const i32x4 *>(slot + 2048 * e + f0);
            const i32x4 q = *reinterpret_cast<const i32x4 *>(slot + 2048 * e + (f0 ^ 64));
            f[e] = (i32x8){p[0], p[1], p[2], p[3], q[0], q[1], q[2], q[3]};
        }
        // the slot is refilled only after its reads have returned
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(WAIT_LGKM0);
        __builtin_amdgcn_sched_barrier(0);
        dma(nth(i + D), ring(U % D));
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const float swq = __int_as_float(__builtin_amdgcn_update_dpp(
                0, __float_as_int(sw[j]), Q * 0x55, 0xF, 0xF, true));       // quad lane Q to its quad
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    f[MT + j], f[t], (f32x4){0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
                const float c = sa[t][Q] * swq;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[t][j][r] = __builtin_fmaf(p[r], c, acc[t][j][r]);
            }
        }
    };
    load_scales(0);
#pragma unroll
    for (int d = 0; d < D; ++d)
        dma(nth(d), ring(d));
    const uint32_t runs = (nb + rlen - 1) >> rlog;
    const uint32_t mine = runs > (uint32_t)wave ? (runs - wave + NW - 1) / NW * rlen : 0;
    constexpr int UN = D == 3 ? 12 : 4;
    uint32_t i = 0;
    auto run = [&](auto self, auto u_) {
        constexpr int U = decltype(u_)::value;
        if constexpr (U < UN) {
            if (i + U >= mine)
                return;
            block(u_, i + U);
            self(self, std::integral_constant<int, U + 1>());
        }
    };
    for (; i < mine; i += UN)
        run(run, std::integral_constant<int, 0>());
    // the loads past the end must land before the ring is used again
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
    __syncthreads();
    constexpr int PB = MT * NT * 1024;                     // a wave's partial tile
    constexpr int PER = NW * SLOT / PB;                    // of which a ring position holds
    static_assert(PER * D >= NW, "partial tiles fit in the ring");
    auto part = [&](int w) { return ring(w / PER) + w % PER * PB; };
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            *reinterpret_cast<f32x4 *>(part(wave) + (t * NT + j) * 1024 + 16 * lane) = acc[t][j];
    __syncthreads();
    // unit e of the tile: a lane's four columns of one row
    for (uint32_t e = threadIdx.x; e < 64 * MT * NT; e += 64 * NW) {
        const uint32_t tile = e / 64, l = e % 64;
        const uint32_t r = m0 + tile / NT * 16 + l % 16, c = tile % NT * 16 + l / 16 * 4;
        f32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < NW; ++w)
            v += *reinterpret_cast<const f32x4 *>(part(w) + tile * 1024 + 16 * l);
        if (r >= M || c >= rpw || n0 + c >= N)
            continue;
        uint16_t *const to = out + (size_t)r * N + n0 + c;
        const u32x2 o = {pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
        if (n0 + c + 4 <= N)                 // (rpw is a multiple of 4; rows of C are aligned to 2 bytes)
            *reinterpret_cast<u32x2_any *>(to) = o;
        else
            for (uint32_t i = 0; i < N - (n0 + c); ++i)
                to[i] = (uint16_t)(o[i / 2] >> 16 * (i % 2));
    }
}

// Waves and ring depth of a ksplit workgroup: what 160 KB of LDS hold of
// 2 (MT + NT) KB blocks, waves first (measured at every MT + NT: more waves
// beat a deeper ring).
constexpr int ks_waves(int s) { return s <= 5 ? 8 : s == 6 ? 6 : s <= 8 ? 5 : 4; }
constexpr int ks_depth(int s) { return s <= 3 ? 3 : 2; }
// NT of a workgroup of rpw rows of W
constexpr uint32_t ks_columns(uint32_t rpw) { return rpw <= 16 ? 1 : rpw <= 32 ? 2 : rpw <= 48 ? 3 : 5; }

struct GemmArgs {
    const uint8_t *a;
    const float *as;
    const uint8_t *w;
    const float *ws;
    uint16_t *out;
    uint32_t m, n, k;
    hipStream_t st;
};

template <int MT, int NT>
void launch_ksplit(const GemmArgs &g, uint32_t rpw, bool once)
{
    constexpr int NW = ks_waves(MT + NT), D = ks_depth(MT + NT);
    const uint32_t mt = (g.m + 16 * MT - 1) / (16 * MT), nt = (g.n + rpw - 1) / rpw;
    auto go = [&](auto k) {
        hipLaunchKernelGGL(k, dim3(mt * nt), dim3(64 * NW), 0, g.st, g.a, g.as, g.w, g.ws, g.out, g.m, g.n, g.k, mt,
                           rpw);
    };
    if (once)
        go(k_fp8_gemm_block_ksplit<MT, NT, NW, D, true>);
    else
        go(k_fp8_gemm_block_ksplit<MT, NT, NW, D, false>);
}

template <int MT>
void launch_ksplit_rows(const GemmArgs &g, uint32_t rpw, bool once)
{
    switch (ks_columns(rpw)) {
    case 1: launch_ksplit<MT, 1>(g, rpw, once); break;
    case 2: launch_ksplit<MT, 2>(g, rpw, once); break;
    case 3: launch_ksplit<MT, 3>(g, rpw, once); break;
    default: launch_ksplit<MT, 5>(g, rpw, once); break;
    }
}

template <int MW, int NW, int TJ>
hipError_t launch_tiles(const GemmArgs &g, uint32_t mt, uint32_t nt, uint32_t first, uint32_t tiles,
                        bool quarters)
{
    auto go = [&](auto k) {
        hipLaunchKernelGGL(k, dim3(quarters ? 4 * tiles : tiles), dim3(64 * MW * NW), 0, g.st, g.a, g.as, g.w, g.ws,
                           g.out, g.m, g.n, g.k, mt, nt, first, (uint32_t)quarters);
    };
    if (g.k % 128)
        go(k_fp8_gemm_block_tiles<MW, NW, TJ, true>);
    else
        go(k_fp8_gemm_block_tiles<MW, NW, TJ, false>);
    count_launch();
    return hipGetLastError();
}

// Which kernel, with which tiles, serves a shape.
struct Choice {
    int kernel;                      // QP_BLOCKSCALE_*
    uint32_t mt, rpw;                // ksplit: MT and rows of W per workgroup
    bool once;                       // ksplit: W past the caches
    uint32_t mtiles, ntiles;         // tiles: the grid of them,
    uint32_t full;                   // 256 x 256: those before the quarters
};

Choice choose(uint32_t m, uint32_t n, uint32_t k)
{
    const uint32_t cus = cu_count() ? cu_count() : 256, nb = (k + 127) / 128;

    // Time estimates in tenths of a nanosecond, fitted to 36 shapes from 17 x 512
    // x 4096 to 6599 x 256 x 8448 with every kernel on each (one MI355X).  The
    // choice costs 1% against the best of them in the mean, at the worst 13 to
    // 20% (989 x 296 x 16384).  They rank the kernels and are no forecast: there is
    // no term for the bytes that a share takes from L2 and HBM, so that where those
    // bound a call the estimate is low (37 x 17408 x 5120 16.8 for 22.9 us, 16 x
    // 152064 x 5120 75 for 129, 7218 x 1641 x 384 8.6 for 13.9).  ksplit, per round of its
    // workgroups: a start and an end that grow with the tile, and per K block
    // 8.5 ns for 8 rows of A, 12.9 for 8 of W and 9.1 for a 16 x 16 tile.  It
    // takes 16 to 64 rows of A a workgroup, whatever suits the shape: 64 x 5120
    // x 17408 36 us with 64, 30 with 32; 284 x 223 x 14336 17 with 64, 9 with 16.
    // 128 x 128 tiles: 598 ns a K block alone on a CU, 1100 for two.  256 x 256
    // tiles: 1680.
    uint64_t t_ks = ~0ull;
    uint32_t mtk = 1, rpw = 16;
    for (uint32_t mt = 1; mt <= 4 && 16 * (mt - 1) < m; ++mt) {
        // W rows per workgroup: the columns dealt over the CUs, at most 80, in
        // as few rounds as that allows
        const uint32_t mwg = (m + 16 * mt - 1) / (16 * mt), per = cus > mwg ? cus / mwg : 1;
        const uint32_t rounds_n = (uint32_t)((n + 80ull * per - 1) / (80ull * per));
        const uint32_t share = (uint32_t)((n + (uint64_t)rounds_n * per - 1) / ((uint64_t)rounds_n * per));
        const uint32_t rows = (share + 3) / 4 * 4, nt = ks_columns(rows);
        const uint64_t wgs = (uint64_t)mwg * ((n + rows - 1) / rows);
        const uint64_t t = 23000 + (wgs + cus - 1) / cus *
                                       (8800 + 1180 * mt * nt +
                                        nb * (85ull * ((std::min(16 * mt, m) + 7) / 8) +
                                              129 * ((rows + 7) / 8) + 91 * mt * nt));
        if (t < t_ks) {
            t_ks = t;
            mtk = mt;
            rpw = rows;
        }
    }
    auto t_small = [&](uint64_t tiles) {
        const uint64_t last = tiles % (2 * cus);
        return 35100 + (tiles / (2 * cus) * 11000 + (last > cus ? 11000 : last ? 5980 : 0)) * nb;
    };
    const uint32_t ms = (m + 127) / 128, ns = (n + 127) / 128, ml = (m + 255) / 256, nl = (n + 255) / 256;
    const uint64_t small = (uint64_t)ms * ns, large = (uint64_t)ml * nl;
    // the 256 x 256 tiles past the last whole round run as 128 x 128 quarters
    // if that is faster than another round
    const uint64_t tail = large % cus;
    const bool quarter = tail && t_small(4 * tail) < 16800ull * nb;
    const uint64_t full = quarter ? large - tail : large;
    const uint64_t t_large = 58000 + (full + cus - 1) / cus * 16800ull * nb + (quarter ? t_small(4 * tail) : 0);

    if (t_ks <= t_small(small) && t_ks <= t_large) {
        // W past the caches (nontemporal) where it is read once and no cache would
        // have kept it: 16 x 152064 x 5120 136 us against 151; 4 x 17408 x 5120, cold,
        // 17.1 against 19.1.  A small weight that is in the 256 MB memory-side cache
        // stays there otherwise (1 x 5120 x 5120: 6.7 us against 8.0), and with more
        // rows the gain is small (37 x 5120 x 17408, cold: 27.6 against 28.6; cached:
        // 26.6 against 24.1), so those pass it only when larger than that cache.
        const bool once = m <= 16 * mtk && (uint64_t)n * k >= (mtk == 1 ? 1u << 26 : 1u << 28);
        return {QP_BLOCKSCALE_KSPLIT, mtk, rpw, once, 0, 0, 0};
    }
    if (full == 0 || t_small(small) <= t_large)
        return {QP_BLOCKSCALE_TILES_128, 0, 0, false, ms, ns, (uint32_t)small};
    return {quarter ? QP_BLOCKSCALE_TILES_256_QUARTERS : QP_BLOCKSCALE_TILES_256, 0, 0, false, ml, nl, (uint32_t)full};
}

} // namespace

int fp8_gemm_blockscale_kernel(uint32_t m, uint32_t n, uint32_t k)
{
    const Choice c = choose(m, n, k);
    return c.kernel == QP_BLOCKSCALE_KSPLIT ? c.kernel + (int)(c.mt + 8 * ks_columns(c.rpw) + 64 * c.once) : c.kernel;
}

hipError_t launch_fp8_gemm_blockscale(const uint8_t *a, const float *as, const uint8_t *w,
                                      const float *ws, uint16_t *out, uint32_t m, uint32_t n,
                                      uint32_t k, hipStream_t st)
{
    const GemmArgs g = {a, as, w, ws, out, m, n, k, st};
    const Choice c = choose(m, n, k);
    if (c.kernel == QP_BLOCKSCALE_KSPLIT) {
        if (c.mt == 1)
            launch_ksplit_rows<1>(g, c.rpw, c.once);
        else if (c.mt == 2)
            launch_ksplit_rows<2>(g, c.rpw, c.once);
        else if (c.mt == 3)
            launch_ksplit_rows<3>(g, c.rpw, c.once);
        else
            launch_ksplit_rows<4>(g, c.rpw, c.once);
        count_launch();
        return hipGetLastError();
    }
    if (c.kernel == QP_BLOCKSCALE_TILES_128)
        return launch_tiles<2, 2, 4>(g, c.mtiles, c.ntiles, 0, c.full, false);
    if (const hipError_t e = launch_tiles<4, 2, 8>(g, c.mtiles, c.ntiles, 0, c.full, false))
        return e;
    if (c.kernel == QP_BLOCKSCALE_TILES_256)
        return hipSuccess;
    return launch_tiles<2, 2, 4>(g, c.mtiles, c.ntiles, c.full, c.mtiles * c.ntiles - c.full, true);
}

} // namespace qp
