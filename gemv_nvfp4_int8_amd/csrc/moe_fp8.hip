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
//    from L2, topk wave maxima): cheaper than a launch of its own.  It leaves
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
//  * h_e stays at F32's precision between the launches as a sum of two BF16
//    planes, hi = bf16(h), lo = bf16(h - hi) (error 2^-17 of h): the second
//    product then takes two MFMAs where one would read a rounded h.
//  * The second launch's workgroups own output columns for all experts, so a
//    token's sum over its experts needs no atomics and has a fixed order.
#include "qp_device.hpp"
#include "qp_launch.hpp"

namespace qp {
namespace {

typedef __attribute__((ext_vector_type(4))) short s16x4;

constexpr int MAX_T = 16, MAX_TOPK = 16, MAX_E = 512, MAX_PAIRS = MAX_T * MAX_TOPK;
constexpr int WIN = 256;                        // K elements per window
// Past every buffer (each is below 2^31 bytes): such a load returns zero.
constexpr uint32_t OOB = 0x80000000u;

// What the first launch leaves for the second (behind the two planes of h).
struct Plan {
    uint32_t nact;
    uint32_t expert[MAX_PAIRS];                 // active experts, ascending
    uint32_t first[MAX_PAIRS + 1];              // their first pair
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

__device__ __forceinline__ uint32_t wave_max_u(uint32_t v)
{
    v = max(v, dpp_u<0xB1>(v));                 // pairs, quads, eights, sixteens
    v = max(v, dpp_u<0x4E>(v));
    v = max(v, dpp_u<0x141>(v));
    v = max(v, dpp_u<0x140>(v));
    v = max(v, (uint32_t)__shfl_xor((int)v, 16, WAVE));
    return max(v, (uint32_t)__shfl_xor((int)v, 32, WAVE));
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
    float weight[MAX_PAIRS];                    // p of each pair
    // scratch
    uint32_t sel_e[MAX_T][MAX_TOPK], nsel[MAX_T];
    float sel_w[MAX_T][MAX_TOPK];
    uint32_t mask[MAX_E], base[MAX_E];          // tokens of an expert; its first pair
};

// The topk of one token by a wave: lane l holds experts l*EPL .. l*EPL+EPL-1,
// so among equal keys the lowest lane, and in it the lowest slot, is the
// lowest expert.
template <int EPL>
__device__ __forceinline__ void route_token(const float *__restrict__ logits, uint32_t E,
                                            uint32_t topk, bool renorm, uint32_t t, Routing &R)
{
    const uint32_t lane = threadIdx.x & 63;
    uint32_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const uint32_t e = lane * EPL + j;
        key[j] = e < E ? key_of(logits[(size_t)t * E + e] + 0.0f) : 0u;   // (-0 ties with +0)
    }
    float top = 0.0f, all = 0.0f;
    if (!renorm) {
        uint32_t b = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            b = max(b, key[j]);
        top = value_of(wave_max_u(b));
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            all += key[j] ? expf(value_of(key[j]) - top) : 0.0f;
        for (int o = 1; o < 64; o <<= 1)
            all += __shfl_xor(all, o, WAVE);
    }
    uint32_t n = 0, my_e = 0;
    float sum = 0.0f, my_w = 0.0f;
    for (uint32_t i = 0; i < topk; ++i) {
        uint32_t b = key[0], bj = 0;
#pragma unroll
        for (int j = 1; j < EPL; ++j)
            if (key[j] > b) {
                b = key[j];
                bj = j;
            }
        const uint32_t m = wave_max_u(b);
        if (m == 0)
            break;                              // uniform: nothing left to choose
        const uint32_t who = (uint32_t)__builtin_ctzll(__ballot(b == m));
        const uint32_t j = (uint32_t)__builtin_amdgcn_readlane((int)bj, (int)who);
        if (i == 0)
            top = value_of(m);
        const float w = expf(value_of(m) - top);
        sum += w;
        if (lane == i) {
            my_e = who * EPL + j;
            my_w = w;
        }
        if (lane == who) {
#pragma unroll
            for (int q = 0; q < EPL; ++q)
                if (q == (int)j)
                    key[q] = 0;
        }
        n = i + 1;
    }
    if (lane < n) {
        R.sel_e[t][lane] = my_e;
        R.sel_w[t][lane] = my_w / (renorm ? sum : all);
        atomicOr(&R.mask[my_e], 1u << t);       // an OR: order does not matter
    }
    if (lane == 0)
        R.nsel[t] = n;
}

// Fill R (every thread of the workgroup calls this; ends with a barrier).
__device__ void route(const float *__restrict__ logits, uint32_t T, uint32_t E, uint32_t topk,
                      bool renorm, Routing &R)
{
    const uint32_t tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, nw = blockDim.x >> 6;
    for (uint32_t e = tid; e < MAX_E; e += blockDim.x)
        R.mask[e] = 0;
    __syncthreads();
    for (uint32_t t = wave; t < T; t += nw) {
        if (E <= 64)
            route_token<1>(logits, E, topk, renorm, t, R);
        else if (E <= 128)
            route_token<2>(logits, E, topk, renorm, t, R);
        else if (E <= 256)
            route_token<4>(logits, E, topk, renorm, t, R);
        else
            route_token<8>(logits, E, topk, renorm, t, R);
    }
    __syncthreads();
    if (wave == 0) {
        // lane l: experts 8l .. 8l+7; active experts (high half) and pairs
        // (low half) before it, by an inclusive scan over the lanes
        uint32_t mk[8], mine = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            mk[j] = R.mask[8 * lane + j];
            mine += (mk[j] ? 0x10000u : 0u) + (uint32_t)__popc(mk[j]);
        }
        uint32_t inc = mine;
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t v = (uint32_t)__shfl_up((int)inc, o, WAVE);
            inc += lane >= (uint32_t)o ? v : 0u;
        }
        uint32_t at = inc - mine;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (mk[j]) {
                R.plan.expert[at >> 16] = 8 * lane + j;
                R.plan.first[at >> 16] = at & 0xFFFFu;
                R.base[8 * lane + j] = at & 0xFFFFu;
                at += 0x10000u + (uint32_t)__popc(mk[j]);
            }
        if (lane == 63) {
            R.plan.nact = inc >> 16;
            R.plan.first[inc >> 16] = inc & 0xFFFFu;
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

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
__device__ __forceinline__ float load4(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
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

// The sum over the 16 K slices (lanes of equal l % 4), in every lane.
__device__ __forceinline__ float sum_slices(float v)
{
    v += dpp_f<0x128>(v);                       // rotate by 8 and by 4 in a row of 16
    v += dpp_f<0x124>(v);
    v += __shfl_xor(v, 16, WAVE);
    return v + __shfl_xor(v, 32, WAVE);
}

struct MoeArgs {
    const uint16_t *x;
    const float *logits;
    const uint8_t *w13, *w2;
    const float *s13, *s2;
    uint16_t *hi, *lo;                          // [pairs, I] planes of p * h
    Plan *plan;
    uint16_t *out;
    uint32_t T, E, topk, H, I, renorm;
};

// Gate rows 4g .. 4g+3 and their up rows of one expert, for its cnt <= 4*TG
// tokens.
template <int TG>
__device__ __forceinline__ void gate_up(const MoeArgs &A, const Routing &R, uint32_t e, uint32_t first,
                                        uint32_t cnt, uint32_t g)
{
    constexpr int D = TG == 1 ? 4 : 2;          // windows in flight
    const uint32_t lane = threadIdx.x & 63, r4 = lane & 3, c16 = lane >> 2;
    const uint32_t HB = A.H / 128, IB = A.I / 128, nw = (A.H + WIN - 1) / WIN;
    const __amdgpu_buffer_rsrc_t rw = rsrc(A.w13 + (size_t)e * 2 * A.I * A.H, 2 * A.I * A.H);
    const __amdgpu_buffer_rsrc_t rs = rsrc(A.s13 + (size_t)e * 2 * IB * HB, 2 * IB * HB * 4);
    const __amdgpu_buffer_rsrc_t rx = rsrc(A.x, A.T * A.H * 2);
    const uint32_t og = (4 * g + r4) * A.H + 16 * c16, ou = og + A.I * A.H;
    const uint32_t sg = (4 * g / 128) * HB * 4 + 4 * (lane >> 5), su = sg + IB * HB * 4;
    uint32_t ox[TG];
#pragma unroll
    for (int t = 0; t < TG; ++t)
        ox[t] = R.plan.token[first + min(4u * t + r4, cnt - 1)] * A.H * 2 + 32 * c16;

    struct Stage {
        u32x4 g, u, x[TG][2];
        float sg, su;
    } st[D];
    auto fetch = [&](Stage &s, uint32_t w) {
        const bool ok = w * WIN + 16 * c16 < A.H;
        s.g = load16(rw, ok ? og + w * WIN : OOB);
        s.u = load16(rw, ok ? ou + w * WIN : OOB);
        s.sg = load4(rs, ok ? sg + 8 * w : OOB);
        s.su = load4(rs, ok ? su + 8 * w : OOB);
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            s.x[t][0] = load16(rx, ok ? ox[t] + 2 * w * WIN : OOB);
            s.x[t][1] = load16(rx, ok ? ox[t] + 2 * w * WIN + 16 : OOB);
        }
    };
    f32x4 ag[TG] = {}, au[TG] = {};
    auto use = [&](const Stage &s) {
        s16x4 wg[4], wu[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            wg[i] = fp8x4_bf16(s.g[i]);
            wu[i] = fp8x4_bf16(s.u[i]);
        }
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            const f32x4 pg = window(wg, s.x[t], (f32x4){});
            const f32x4 pu = window(wu, s.x[t], (f32x4){});
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                ag[t][r] = __builtin_fmaf(pg[r], s.sg, ag[t][r]);
                au[t][r] = __builtin_fmaf(pu[r], s.su, au[t][r]);
            }
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d)
        fetch(st[d], d);
    for (uint32_t w = 0; w < nw; w += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            use(st[d]);
            fetch(st[d], w + d + D);
        }
    }
    // lane l takes token l / 4 of weight row l % 4
    float vg = 0.0f, vu = 0.0f;
#pragma unroll
    for (int t = 0; t < 4 * TG; ++t) {
        const float a = sum_slices(ag[t / 4][t % 4]), b = sum_slices(au[t / 4][t % 4]);
        vg = c16 == (uint32_t)t ? a : vg;
        vu = c16 == (uint32_t)t ? b : vu;
    }
    if (c16 < cnt) {
        const float h = vg / (1.0f + expf(-vg)) * vu * R.weight[first + c16];
        const uint32_t hi = f32_to_bf16(h);
        const size_t at = (size_t)(first + c16) * A.I + 4 * g + r4;
        A.hi[at] = (uint16_t)hi;
        A.lo[at] = (uint16_t)f32_to_bf16(h - bf16_lo(hi));
    }
}

// First launch: route, then gate/up tasks of 4 + 4 rows, one wave each.
__global__ __launch_bounds__(256) void k_moe_gate_up(MoeArgs A)
{
    __shared__ Routing R;
    route(A.logits, A.T, A.E, A.topk, A.renorm != 0, R);
    if (blockIdx.x == 0) {
        const uint32_t n = R.plan.nact, pairs = R.plan.first[n];
        for (uint32_t i = threadIdx.x; i <= n; i += blockDim.x)
            A.plan->first[i] = R.plan.first[i];
        for (uint32_t i = threadIdx.x; i < n; i += blockDim.x)
            A.plan->expert[i] = R.plan.expert[i];
        for (uint32_t i = threadIdx.x; i < pairs; i += blockDim.x)
            A.plan->token[i] = R.plan.token[i];
        if (threadIdx.x == 0)
            A.plan->nact = n;
    }
    const uint32_t groups = A.I / 4, tasks = R.plan.nact * groups;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (uint32_t task = blockIdx.x * 4 + wave; task < tasks; task += gridDim.x * 4) {
        const uint32_t slot = task / groups, g = task % groups;
        const uint32_t e = __builtin_amdgcn_readfirstlane(R.plan.expert[slot]);
        const uint32_t first = __builtin_amdgcn_readfirstlane(R.plan.first[slot]);
        const uint32_t cnt = __builtin_amdgcn_readfirstlane(R.plan.first[slot + 1]) - first;
        if (cnt <= 4)
            gate_up<1>(A, R, e, first, cnt, g);
        else if (cnt <= 8)
            gate_up<2>(A, R, e, first, cnt, g);
        else
            gate_up<4>(A, R, e, first, cnt, g);
    }
}

constexpr int DOWN_WAVES = 8, DOWN_ROWS = 8;

// Columns c0 .. c0+7 of the output over windows [w0, w1) of one expert's I,
// for its cnt <= 4*TG tokens, added to acc[token][column].
template <int TG>
__device__ __forceinline__ void down(const MoeArgs &A, const Plan &P, uint32_t e, uint32_t first,
                                     uint32_t cnt, uint32_t c0, uint32_t w0, uint32_t w1,
                                     float (*acc)[DOWN_ROWS])
{
    constexpr int D = 2;
    const uint32_t lane = threadIdx.x & 63, r4 = lane & 3, c16 = lane >> 2;
    const uint32_t HB = A.H / 128, IB = A.I / 128;
    const __amdgpu_buffer_rsrc_t rw = rsrc(A.w2 + (size_t)e * A.H * A.I, A.H * A.I);
    const __amdgpu_buffer_rsrc_t rs = rsrc(A.s2 + (size_t)e * HB * IB, HB * IB * 4);
    const uint32_t plane = A.T * A.topk * A.I * 2;
    const __amdgpu_buffer_rsrc_t rhi = rsrc(A.hi, plane), rlo = rsrc(A.lo, plane);
    const uint32_t ow = (c0 + r4) * A.I + 16 * c16;
    const uint32_t os = (c0 / 128) * IB * 4 + 4 * (lane >> 5);
    uint32_t ox[TG];
#pragma unroll
    for (int t = 0; t < TG; ++t)
        ox[t] = (first + min(4u * t + r4, cnt - 1)) * A.I * 2 + 32 * c16;
    struct Stage {
        u32x4 w[2], hi[TG][2], lo[TG][2];
        float s;
    } st[D];
    auto fetch = [&](Stage &s, uint32_t w) {
        const bool ok = w < w1 && w * WIN + 16 * c16 < A.I;
        s.w[0] = load16(rw, ok ? ow + w * WIN : OOB);
        s.w[1] = load16(rw, ok ? ow + 4 * A.I + w * WIN : OOB);
        s.s = load4(rs, ok ? os + 8 * w : OOB);
#pragma unroll
        for (int t = 0; t < TG; ++t)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                s.hi[t][q] = load16(rhi, ok ? ox[t] + 2 * w * WIN + 16 * q : OOB);
                s.lo[t][q] = load16(rlo, ok ? ox[t] + 2 * w * WIN + 16 * q : OOB);
            }
    };
    f32x4 a[TG][2] = {};
    auto use = [&](const Stage &s) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            s16x4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = fp8x4_bf16(s.w[q][i]);
#pragma unroll
            for (int t = 0; t < TG; ++t) {
                const f32x4 p = window(w, s.hi[t], window(w, s.lo[t], (f32x4){}));
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    a[t][q][r] = __builtin_fmaf(p[r], s.s, a[t][q][r]);
            }
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d)
        fetch(st[d], w0 + d);
    for (uint32_t w = w0; w < w1; w += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            use(st[d]);
            fetch(st[d], w + d + D);
        }
    }
    // other lanes of this wave may have added to the same sums before
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float v = 0.0f;
#pragma unroll
        for (int t = 0; t < 4 * TG; ++t) {
            const float s = sum_slices(a[t / 4][q][t % 4]);
            v = c16 == (uint32_t)t ? s : v;
        }
        if (c16 < cnt)
            acc[P.token[first + c16]][4 * q + r4] += v;   // only this wave's, one lane each
    }
}

// Second launch: 8 output columns per workgroup; its waves take the active
// experts in turn (in pieces of the K range where there are fewer experts
// than two per wave), and their sums are joined in wave order.
__global__ __launch_bounds__(64 * DOWN_WAVES) void k_moe_down(MoeArgs A)
{
    __shared__ Plan P;
    __shared__ float acc[DOWN_WAVES][MAX_T][DOWN_ROWS];
    const uint32_t tid = threadIdx.x;
    const uint32_t n = A.plan->nact;
    for (uint32_t i = tid; i <= n; i += blockDim.x)
        P.first[i] = A.plan->first[i];
    for (uint32_t i = tid; i < n; i += blockDim.x)
        P.expert[i] = A.plan->expert[i];
    for (uint32_t i = tid; i < A.T * A.topk; i += blockDim.x)
        P.token[i] = A.plan->token[i];
    for (uint32_t i = tid; i < DOWN_WAVES * MAX_T * DOWN_ROWS; i += blockDim.x)
        (&acc[0][0][0])[i] = 0.0f;
    __syncthreads();
    const uint32_t nw = (A.I + WIN - 1) / WIN, c0 = blockIdx.x * DOWN_ROWS;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint32_t pieces = n ? (2 * DOWN_WAVES + n - 1) / n : 1;
    pieces = min(pieces, nw);
    const uint32_t per = (nw + pieces - 1) / pieces;
    for (uint32_t u = wave; u < n * pieces; u += DOWN_WAVES) {
        const uint32_t slot = u / pieces, w0 = (u % pieces) * per, w1 = min(w0 + per, nw);
        if (w0 >= w1)
            continue;
        const uint32_t e = __builtin_amdgcn_readfirstlane(P.expert[slot]);
        const uint32_t first = __builtin_amdgcn_readfirstlane(P.first[slot]);
        const uint32_t cnt = __builtin_amdgcn_readfirstlane(P.first[slot + 1]) - first;
        if (cnt <= 4)
            down<1>(A, P, e, first, cnt, c0, w0, w1, acc[wave]);
        else if (cnt <= 8)
            down<2>(A, P, e, first, cnt, c0, w0, w1, acc[wave]);
        else
            down<4>(A, P, e, first, cnt, c0, w0, w1, acc[wave]);
    }
    __syncthreads();
    for (uint32_t i = tid; i < A.T * DOWN_ROWS; i += blockDim.x) {
        const uint32_t t = i / DOWN_ROWS, c = i % DOWN_ROWS;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < DOWN_WAVES; ++w)
            v += acc[w][t][c];
        A.out[(size_t)t * A.H + c0 + c] = (uint16_t)f32_to_bf16(v);
    }
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
    const uint64_t planes = planes_bytes(T, topk, I);
    uint8_t *const wk = (uint8_t *)work;
    const MoeArgs A = {x, logits, w13, w2, s13, s2, (uint16_t *)wk, (uint16_t *)(wk + planes / 2),
                       (Plan *)(wk + planes), out, T, E, topk, H, I, renorm};
    // one wave per task while the tasks of all experts that may be chosen
    // leave CUs idle, else four workgroups per CU walk them
    const uint64_t slots = E < T * topk ? E : T * topk;
    const uint64_t groups = (slots * (I / 4) + 3) / 4;
    const uint32_t cus = cu_count(), cap = 4 * (cus ? cus : 256);
    hipLaunchKernelGGL(k_moe_gate_up, dim3(groups < cap ? (uint32_t)groups : cap), dim3(256), 0, st, A);
    count_launch();
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return err;
    hipLaunchKernelGGL(k_moe_down, dim3(H / DOWN_ROWS), dim3(64 * DOWN_WAVES), 0, st, A);
    count_launch();
    return hipGetLastError();
}

} // namespace qp
