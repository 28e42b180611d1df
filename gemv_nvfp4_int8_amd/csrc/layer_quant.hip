// layer_quant.hip -- the two operators that feed a product: residual addition
// + RMS norm, and the gated activation silu(g) * u, each with an 8-bit output
// (E4M3 per row or per 128, int8 per 32) in the same pass, or a BF16 one.
//
// Both stream HBM (7 and 5 bytes per element), so every input byte is read
// once: a row's values stay in registers between its reductions and the
// encode.  A thread owns 16-byte chunks of 8 elements, neighbouring lanes
// neighbouring chunks, so a 128-block is one DPP row of 16 lanes and a
// 32-block one quad; block maxima never leave the registers.
#include <algorithm>
#include <type_traits>

#include "qp_device.hpp"
#include "qp_launch.hpp"

namespace qp {
namespace {

enum { FMT_ROW = 0, FMT_BLOCK128 = 1, FMT_INT8 = 2, FMT_BF16 = 16 };

template <int CTRL>
__device__ __forceinline__ float dpp_mov(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}

// DPP controls whose four applications, one after another, pair every lane of
// a row of 16 with all others: swap in pairs, swap pairs in quads, mirror in
// halves of 8, mirror in 16.
constexpr int DPP_X1 = 0xB1, DPP_X2 = 0x4E, DPP_HALF_MIRROR = 0x141, DPP_MIRROR = 0x140;

__device__ __forceinline__ float max4(float v)
{
    v = __builtin_fmaxf(v, dpp_mov<DPP_X1>(v));
    return __builtin_fmaxf(v, dpp_mov<DPP_X2>(v));
}
__device__ __forceinline__ float max16(float v)
{
    v = max4(v);
    v = __builtin_fmaxf(v, dpp_mov<DPP_HALF_MIRROR>(v));
    return __builtin_fmaxf(v, dpp_mov<DPP_MIRROR>(v));
}
__device__ __forceinline__ float sum16(float v)
{
    v += dpp_mov<DPP_X1>(v);
    v += dpp_mov<DPP_X2>(v);
    v += dpp_mov<DPP_HALF_MIRROR>(v);
    return v + dpp_mov<DPP_MIRROR>(v);
}
__device__ __forceinline__ float sum64(float v)
{
    v = sum16(v);
    v += __shfl_xor(v, 16, WAVE);
    return v + __shfl_xor(v, 32, WAVE);
}
__device__ __forceinline__ float max64(float v)
{
    v = max16(v);
    v = __builtin_fmaxf(v, __shfl_xor(v, 16, WAVE));
    return __builtin_fmaxf(v, __shfl_xor(v, 32, WAVE));
}

__device__ __forceinline__ void unpack8(u32x4 r, float *v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(r[i]);
        v[2 * i + 1] = bf16_hi(r[i]);
    }
}

__device__ __forceinline__ float amax8(const float *y)
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = __builtin_fmaxf(m, __builtin_fabsf(y[i]));
    return m;
}

// bf16(x + r), element by element.
__device__ __forceinline__ u32x4 add_bf16(u32x4 x, u32x4 r)
{
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = pk_bf16(bf16_lo(x[i]) + bf16_lo(r[i]), bf16_hi(x[i]) + bf16_hi(r[i]));
    return o;
}

// Sum of squares of a chunk, in element order.
__device__ __forceinline__ float ssq8(u32x4 h)
{
    float v[8], s = 0.0f;
    unpack8(h, v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        s = __builtin_fmaf(v[i], v[i], s);
    return s;
}

__device__ __forceinline__ void norm8(u32x4 h, u32x4 w, float rstd, float *y)
{
    float a[8], b[8];
    unpack8(h, a);
    unpack8(w, b);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y[i] = a[i] * rstd * b[i];
}

// silu(g) * u with the hardware's exp2 and reciprocal (1 ulp each).  The
// argument's rounding costs |g| * 2^-24 relative on exp(-g): at most 2e-7 of
// y where exp(-g) <= 1 counts, and only for negative g, whose y is small,
// more.  exp(-g) = inf gives -0, the limit.  The reciprocal is that of a
// quarter of 1 + exp(-g), and g enters as a quarter (both exact): of the whole
// it would be subnormal from g = -87.4 down to where exp(-g) is inf, -88.7,
// and the instruction returns 0 in place of a subnormal.
__device__ __forceinline__ void silu8(u32x4 g, u32x4 u, float *y)
{
    float a[8], b[8];
    unpack8(g, a);
    unpack8(u, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float e = __builtin_amdgcn_exp2f(a[i] * -0x1.715476p+0f);
        y[i] = a[i] * 0.25f * __builtin_amdgcn_rcpf(__builtin_fmaf(e, 0.25f, 0.25f)) * b[i];
    }
}

template <int FMT>
__device__ __forceinline__ float scale_of(float amax)
{
    return div_by_const<FMT == FMT_INT8 ? 127 : 448>(amax);
}

// Eight codes of y under scale sc (0: all +0).  |y| <= amax, so a quotient
// passes the top code by a few ulp at most, unless the scale is subnormal:
// then it is saturated first.
template <int FMT>
__device__ __forceinline__ u32x2 encode8(const float *y, float sc)
{
    const ScaleDiv d(sc);
    float t[8];
    u32x2 o;
    if (__all(d.fast || sc == 0.0f)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[i] = d.quick(y[i]);
        if (FMT == FMT_INT8)
            o = (u32x2){pack_i8x4(&t[0]), pack_i8x4(&t[4])};
        else
            o = (u32x2){cvt_e4m3x4_nosat(t[0], t[1], t[2], t[3]),
                        cvt_e4m3x4_nosat(t[4], t[5], t[6], t[7])};
    } else {
        constexpr float TOP = FMT == FMT_INT8 ? 127.0f : 448.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[i] = __builtin_amdgcn_fmed3f(d(y[i]), -TOP, TOP);
        if (FMT == FMT_INT8)
            o = (u32x2){pack_i8x4(&t[0]), pack_i8x4(&t[4])};
        else
            o = (u32x2){cvt_e4m3x4(t[0], t[1], t[2], t[3]), cvt_e4m3x4(t[4], t[5], t[6], t[7])};
    }
    return sc == 0.0f ? (u32x2){0, 0} : o;
}

__host__ __device__ __forceinline__ constexpr uint32_t scales_per_row(int fmt, uint32_t k)
{
    return fmt == FMT_ROW ? 1 : fmt == FMT_BLOCK128 ? (k + 127) / 128 : fmt == FMT_INT8 ? k / 32 : 0;
}

// Quantize and store chunk c of a row: block formats find their own scale,
// the row format gets it, BF16 has none.  Every lane of the wave calls this
// (DPP).
template <int FMT>
__device__ __forceinline__ void emit8(const float *y, float row_scale, uint32_t c, bool live,
                                      uint8_t *__restrict__ qr, float *__restrict__ sr)
{
    if (FMT == FMT_BF16) {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = pk_bf16(y[2 * i], y[2 * i + 1]);
        if (live)
            __builtin_nontemporal_store(o, reinterpret_cast<u32x4 *>(qr + (size_t)c * 16));
        return;
    }
    float sc = row_scale;
    if (FMT == FMT_BLOCK128)
        sc = scale_of<FMT>(max16(amax8(y)));
    if (FMT == FMT_INT8)
        sc = scale_of<FMT>(max4(amax8(y)));
    const u32x2 o = encode8<FMT>(y, sc);
    if (live) {
        __builtin_nontemporal_store(o, reinterpret_cast<u32x2 *>(qr + (size_t)c * 8));
        if (FMT == FMT_BLOCK128 && (c & 15) == 0)
            sr[c >> 4] = sc;
        if (FMT == FMT_INT8 && (c & 3) == 0)
            sr[c >> 2] = sc;
    }
}

struct RowArgs {
    const uint16_t *x;          // norm: x; activation: gate_up
    const uint16_t *res;        // norm: residual or null
    const uint16_t *w;          // norm: weight
    uint16_t *res_out;
    uint8_t *q;
    float *s;
    float eps;
    uint32_t rows, k;
    uint32_t parts;             // workgroups per row
};

// 1 / sqrt(mean + eps) from the block sums sm[0 .. nb): lane l adds blocks l,
// l + 64, ... and one butterfly joins the lanes.  Every kernel below forms
// the same block sums (16 lanes of one chunk each), so a row's norm does not
// depend on how many threads share it.
__device__ __forceinline__ float rstd_of(const float *sm, uint32_t nb, uint32_t k, float eps)
{
    float v = 0.0f;
    for (uint32_t i = threadIdx.x & 63; i < nb; i += 64)
        v += sm[i];
    return 1.0f / __builtin_sqrtf(sum64(v) / (float)k + eps);
}

// Scales and codes of a thread's chunks; m is its maximum (row format).
template <int FMT, int CPL, class V>
__device__ __forceinline__ void finish(const RowArgs &A, uint32_t row, uint32_t first, uint32_t T,
                                       float m, float *tops, V value)
{
    const uint32_t nch = A.k / 8;
    float sc = 0.0f;
    if (FMT == FMT_ROW) {
        m = max64(m);
        if ((threadIdx.x & 63) == 0)
            tops[threadIdx.x >> 6] = m;
        __syncthreads();
        for (uint32_t i = 0; i < T / 64; ++i)
            m = __builtin_fmaxf(m, tops[i]);
        sc = scale_of<FMT>(m);
        if (first == 0)
            A.s[row] = sc;
    }
    float *sr = A.s + (size_t)row * scales_per_row(FMT, A.k);
    uint8_t *qr = A.q + (size_t)row * A.k * (FMT == FMT_BF16 ? 2 : 1);
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
        const uint32_t c = first + T * j;
        float y[8];
        value(j, y);
        emit8<FMT>(y, sc, c, c < nch, qr, sr);
    }
}

// The row held in registers, CPL chunks per thread: chunk t + T j of the row,
// T threads, a workgroup.  An activation whose scales are per block has no sum
// over its row, so its rows are also cut into `parts` pieces of T CPL chunks.
//
// Bound by HBM: what counts is that every load of the row is in flight before
// the first use and that no lane idles, so T follows the row (a fixed 256
// threads of 8 chunks left 5 of 8 idle at k = 5120: 8192 x 5120 took 60 us).
// 8192 x 5120 (norm, residual): 49 us, 6.0 TB/s; 4096 x 17408 (activation):
// 56.5 us per 128, 56.0 per row, 57.6 int8, 6.2 to 6.4 TB/s, and 65.5 BF16, 6.5
// TB/s; one row of 5120: 2.9 us in a graph, of which an empty kernel is about 2.
template <bool NORM, int FMT, int CPL>
__global__ __launch_bounds__(1024) void k_row_quant(RowArgs A)
{
    constexpr bool ALONE = !NORM && FMT != FMT_ROW;       // no sum over the row
    __shared__ float sm[NORM ? 1024 * CPL / 16 : 1];
    __shared__ float tops[16];
    const uint32_t T = blockDim.x, t = threadIdx.x, nch = A.k / 8;
    const uint32_t row = ALONE ? blockIdx.x / A.parts : blockIdx.x;
    const uint32_t first = t + (ALONE ? blockIdx.x % A.parts * (T * CPL) : 0);
    const size_t at = (size_t)row * A.k;
    const u32x4 z = (u32x4){0, 0, 0, 0};
    u32x4 h[CPL], w[CPL];                // norm: h and the weight; activation: g and u
    if (NORM) {
        u32x4 r[CPL];
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            const uint32_t c = first + T * j;
            h[j] = r[j] = w[j] = z;
            if (c < nch) {
                h[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(A.x + at + 8 * (size_t)c));
                if (A.res)
                    r[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(A.res + at + 8 * (size_t)c));
                w[j] = *reinterpret_cast<const u32x4 *>(A.w + 8 * (size_t)c);
            }
        }
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            const uint32_t c = first + T * j;
            if (A.res) {
                h[j] = add_bf16(h[j], r[j]);
                if (c < nch)
                    __builtin_nontemporal_store(h[j], reinterpret_cast<u32x4 *>(A.res_out + at + 8 * (size_t)c));
            }
            const float s = sum16(ssq8(h[j]));
            if ((t & 15) == 0)
                sm[c >> 4] = s;          // c / 16 < T CPL / 16; past the row: 0
        }
        __syncthreads();
        const float rstd = rstd_of(sm, T * CPL / 16, A.k, A.eps);
        float m = 0.0f, y[8];
        if (FMT == FMT_ROW) {
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                norm8(h[j], w[j], rstd, y);
                m = __builtin_fmaxf(m, amax8(y));
            }
        }
        finish<FMT, CPL>(A, row, first, T, m, tops,
                               [&](int j, float *v) { norm8(h[j], w[j], rstd, v); });
    } else {
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            const uint32_t c = first + T * j;
            h[j] = w[j] = z;
            if (c < nch) {
                h[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(A.x + 2 * at + 8 * (size_t)c));
                w[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(A.x + 2 * at + A.k + 8 * (size_t)c));
            }
        }
        if (FMT == FMT_ROW) {
            float y[CPL][8], m = 0.0f;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                silu8(h[j], w[j], y[j]);
                m = __builtin_fmaxf(m, amax8(y[j]));
            }
            finish<FMT, CPL>(A, row, first, T, m, tops, [&](int j, float *v) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = y[j][i];
            });
        } else {
            finish<FMT, CPL>(A, row, first, T, 0.0f, tops,
                                   [&](int j, float *v) { silu8(h[j], w[j], v); });
        }
    }
}

// Rows of more than 32768 values, which the registers do not hold (and which
// are not cut): 1024 threads walk the row once per step (sum, for the row
// format the maximum, encode) and recompute y.  With a residual, h is read
// back from residual_out: each thread reads only what it wrote itself.
template <bool NORM, int FMT>
__global__ __launch_bounds__(1024) void k_row_quant_long(RowArgs A)
{
    __shared__ float sums[(1u << 18) / 128];
    __shared__ float tops[16];
    const uint32_t row = blockIdx.x, t = threadIdx.x, nch = A.k / 8, nb = (nch + 15) / 16;
    const uint32_t steps = (nch + 1023) / 1024;
    const size_t at = (size_t)row * A.k;
    const uint16_t *h_src = NORM && A.res ? A.res_out : A.x;
    float rstd = 0.0f;
    if (NORM) {
        for (uint32_t i = 0; i < steps; ++i) {
            const uint32_t c = t + 1024 * i;
            u32x4 h = (u32x4){0, 0, 0, 0};
            if (c < nch) {
                h = *reinterpret_cast<const u32x4 *>(A.x + at + 8 * (size_t)c);
                if (A.res) {
                    h = add_bf16(h, *reinterpret_cast<const u32x4 *>(A.res + at + 8 * (size_t)c));
                    *reinterpret_cast<u32x4 *>(A.res_out + at + 8 * (size_t)c) = h;
                }
            }
            const float s = sum16(ssq8(h));
            if ((t & 15) == 0 && c / 16 < nb)
                sums[c >> 4] = s;
        }
        __syncthreads();
        rstd = rstd_of(sums, nb, A.k, A.eps);
    }
    auto value = [&](uint32_t c, float *y) {
        const u32x4 z = (u32x4){0, 0, 0, 0};
        if (NORM) {
            const u32x4 h = c < nch ? *reinterpret_cast<const u32x4 *>(h_src + at + 8 * (size_t)c) : z;
            const u32x4 w = c < nch ? *reinterpret_cast<const u32x4 *>(A.w + 8 * (size_t)c) : z;
            norm8(h, w, rstd, y);
        } else {
            const uint16_t *p = A.x + 2 * at + 8 * (size_t)c;
            const u32x4 g = c < nch ? *reinterpret_cast<const u32x4 *>(p) : z;
            const u32x4 u = c < nch ? *reinterpret_cast<const u32x4 *>(p + A.k) : z;
            silu8(g, u, y);
        }
    };
    float y[8], sc = 0.0f;
    if (FMT == FMT_ROW) {
        float m = 0.0f;
        for (uint32_t i = 0; i < steps; ++i) {
            value(t + 1024 * i, y);
            m = __builtin_fmaxf(m, amax8(y));
        }
        m = max64(m);
        if ((t & 63) == 0)
            tops[t >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i)
            m = __builtin_fmaxf(m, tops[i]);
        sc = scale_of<FMT>(m);
        if (t == 0)
            A.s[row] = sc;
    }
    float *sr = A.s + (size_t)row * scales_per_row(FMT, A.k);
    uint8_t *qr = A.q + at * (FMT == FMT_BF16 ? 2 : 1);
    for (uint32_t i = 0; i < steps; ++i) {
        const uint32_t c = t + 1024 * i;
        value(c, y);
        emit8<FMT>(y, sc, c, c < nch, qr, sr);
    }
}

template <bool NORM, int FMT, int CPL>
void launch_row(RowArgs A, uint32_t threads, hipStream_t st)
{
    A.parts = (A.k / 8 + threads * CPL - 1) / (threads * CPL);   // 1 unless the row may be cut
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_row_quant<NORM, FMT, CPL>), dim3(A.rows * A.parts), dim3(threads), 0,
                       st, A);
}

// Chunks per thread: one while the whole grid is resident at once (8192
// waves): then the call is latency, and a second chunk only adds to it (16 x
// 5120, norm: 3.5 against 3.9 us; 16 x 17408, activation per 128: 2.5 against
// 3.0).  Two beyond (8192 x 5120: 49.2 against 55.7; 4 chunks 51.3; 4096 x
// 17408: 56.7 against 59.5; 4 chunks 59.9), more only for rows that 1024
// threads do not cover with two; 8 would spill.
template <bool NORM, int FMT>
hipError_t launch_fmt(const RowArgs &A, hipStream_t st)
{
    const uint32_t nch = A.k / 8, waves = (nch + 63) / 64;
    constexpr bool cut = !NORM && FMT != FMT_ROW;
    uint32_t cpl = waves > 1 && (uint64_t)A.rows * waves > 8192 ? 2 : 1;
    if constexpr (cut) {
        const uint32_t threads = std::min((waves + cpl - 1) / cpl * 64, 256u);
        cpl == 1 ? launch_row<NORM, FMT, 1>(A, threads, st) : launch_row<NORM, FMT, 2>(A, threads, st);
    } else {
        cpl = std::max(cpl, (nch + 1023) / 1024);
        const uint32_t threads = (waves + cpl - 1) / cpl * 64;
        if (cpl == 1)
            launch_row<NORM, FMT, 1>(A, threads, st);
        else if (cpl == 2)
            launch_row<NORM, FMT, 2>(A, threads, st);
        else if (cpl == 3)
            launch_row<NORM, FMT, 3>(A, threads, st);
        else if (cpl == 4)
            launch_row<NORM, FMT, 4>(A, threads, st);
        else
            hipLaunchKernelGGL(HIP_KERNEL_NAME(k_row_quant_long<NORM, FMT>), dim3(A.rows), dim3(1024), 0, st, A);
    }
    count_launch();
    return hipGetLastError();
}

template <bool NORM>
hipError_t launch_any(const RowArgs &A, int fmt, hipStream_t st)
{
    return fmt == FMT_ROW        ? launch_fmt<NORM, FMT_ROW>(A, st)
           : fmt == FMT_BLOCK128 ? launch_fmt<NORM, FMT_BLOCK128>(A, st)
           : fmt == FMT_INT8     ? launch_fmt<NORM, FMT_INT8>(A, st)
                                 : launch_fmt<NORM, FMT_BF16>(A, st);
}

} // namespace

hipError_t launch_rmsnorm_residual_quant(const uint16_t *x, const uint16_t *res, const uint16_t *w,
                                         float eps, int fmt, void *q, float *s, uint16_t *res_out,
                                         uint32_t rows, uint32_t k, hipStream_t st)
{
    // A launch holds fewer than 2^32 threads (one with more loses rows without
    // an error), and a row takes 64 of them or more: rows of 16 values, which
    // may number 2^26 and more, go in several launches.
    constexpr uint32_t MOST = 1u << 25;
    for (uint32_t at = 0; at < rows; at += MOST) {
        const size_t e = (size_t)at * k;
        const RowArgs A = {x + e, res ? res + e : nullptr, w, res ? res_out + e : nullptr,
                           (uint8_t *)q + e * (fmt == FMT_BF16 ? 2 : 1), s + (size_t)at * scales_per_row(fmt, k), eps,
                           std::min(rows - at, MOST), k, 1};
        if (const hipError_t err = launch_any<true>(A, fmt, st))
            return err;
    }
    return hipSuccess;
}

hipError_t launch_silu_mul_quant(const uint16_t *gate_up, int fmt, void *q, float *s, uint32_t rows,
                                 uint32_t k, hipStream_t st)
{
    return launch_any<false>({gate_up, nullptr, nullptr, nullptr, (uint8_t *)q, s, 0.0f, rows, k, 1}, fmt, st);
}

} // namespace qp
