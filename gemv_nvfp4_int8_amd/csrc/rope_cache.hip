// rope_cache.hip -- norms of queries and keys, rotary positions, and the paged
// cache's new entries, in one pass over the output of the q/k/v product.
//
// A head is taken by G lanes (8, 16 or 32: the next power of two of d/8), 16
// bytes each, so that its sum of squares and its largest magnitude are a few
// cross-lane steps and no value is read twice from memory.  A lane's partners
// of the half layout lie rot/2 further on or back, in another lane's 16 bytes:
// they are loaded once more (from L1) rather than passed between lanes, because
// rot/2 need not be a multiple of 8.  Cosines and sines are the same for all
// heads of a token: one thread a pair computes them into LDS while the heads'
// loads are on their way.
#include "qp_device.hpp"
#include "qp_launch.hpp"
#include "decoder.hpp"

namespace qp {
namespace {

constexpr uint32_t WG = 256;
constexpr uint32_t MAX_TOKENS = 8;         // of a workgroup

template <int G>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int off = G / 2; off >= 1; off >>= 1)
        v += __shfl_xor(v, off, WAVE);
    return v;
}

template <int G>
__device__ __forceinline__ float group_max(float v)
{
#pragma unroll
    for (int off = G / 2; off >= 1; off >>= 1)
        v = __builtin_fmaxf(v, __shfl_xor(v, off, WAVE));
    return v;
}

__device__ __forceinline__ void unpack(u32x4 w, float *x)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ u32x4 pack(const float *x)
{
    return (u32x4){pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3]), pk_bf16(x[4], x[5]), pk_bf16(x[6], x[7])};
}

// One head's 16 bytes of one lane, and what the rotation needs beside them.
struct Piece {
    u32x4 own, partner;
};

// tokens * heads items are dealt to the workgroup's groups of G lanes, U at a
// time so that a lane has that many loads in flight.
template <bool FP8, int G, int U>
__global__ __launch_bounds__(WG) void k_qk_norm_rope(RopeArgs a, uint32_t tokens, uint32_t heads)
{
    __shared__ f32x2 turn[MAX_TOKENS * 128];
    const uint32_t d = a.cache.d, kv = a.cache.heads, half = a.rot / 2;
    const uint32_t t0 = blockIdx.x * tokens, nt = min(tokens, a.t - t0);
    const uint32_t items = nt * heads, group = threadIdx.x / G, c0 = 8 * (threadIdx.x % G);
    const bool live = c0 < d;
    const bool chunked = half % 8 == 0 && !a.interleaved;
    constexpr uint32_t NG = WG / G;

    Piece p[U];
    auto load = [&](uint32_t first) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = first + u * NG;
            p[u].own = p[u].partner = (u32x4){0, 0, 0, 0};
            if (i >= items || !live)
                continue;
            const uint16_t *x = a.qkv + ((size_t)t0 * heads + i) * d;
            p[u].own = *(const u32x4 *)(x + c0);
            if (chunked && c0 < a.rot && i % heads < heads - kv)
                p[u].partner = *(const u32x4 *)(x + (c0 < half ? c0 + half : c0 - half));
        }
    };
    load(group);
    for (uint32_t i = threadIdx.x; i < nt * half; i += WG) {
        // the angle in turns, in 64 bits: the whole turns of far positions drop
        // out before anything is rounded to 32
        const double turns = (double)a.pos[t0 + i / half] * (double)a.inv_freq[i % half] * 0.15915494309189533577;
        float s, c;
        sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
        turn[i] = (f32x2){c * a.rope_scale, s * a.rope_scale};
    }
    __syncthreads();

    for (uint32_t first = group; first < items; first += U * NG) {
        if (first != group)
            load(first);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = first + u * NG;
            if (i >= items)
                break;                                  // whole groups leave together
            const uint32_t tok = i / heads, h = i - tok * heads;
            float x[8];
            unpack(p[u].own, x);
            if (h < heads - kv) {
                const uint16_t *w = h < a.q_heads ? a.qw : a.kw;
                float rstd = 1.0f;
                if (w) {
                    float ss = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        ss = __builtin_fmaf(x[j], x[j], ss);
                    rstd = __builtin_amdgcn_rsqf(group_sum<G>(ss) / (float)d + a.eps);
                    if (live) {
                        float g[8];
                        unpack(*(const u32x4 *)(w + c0), g);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            x[j] = x[j] * rstd * g[j];
                    }
                }
                if (live && c0 < a.rot) {
                    const f32x2 *cs = turn + tok * half;
                    if (a.interleaved) {
#pragma unroll
                        for (int j = 0; j < 8; j += 2)
                            if (c0 + j < a.rot) {
                                const f32x2 t = cs[(c0 + j) / 2];
                                const float lo = x[j], hi = x[j + 1];
                                x[j] = __builtin_fmaf(lo, t[0], -(hi * t[1]));
                                x[j + 1] = __builtin_fmaf(hi, t[0], lo * t[1]);
                            }
                    } else {
                        float y[8];
                        unpack(p[u].partner, y);
                        const uint16_t *raw = a.qkv + ((size_t)t0 * heads + i) * d;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint32_t e = c0 + j;
                            if (e >= a.rot)
                                continue;
                            const uint32_t o = e < half ? e + half : e - half;
                            if (!chunked)
                                y[j] = __uint_as_float((uint32_t)raw[o] << 16);
                            if (w)
                                y[j] = y[j] * rstd * __uint_as_float((uint32_t)w[o] << 16);
                            const f32x2 t = cs[e < half ? e : e - half];
                            x[j] = __builtin_fmaf(x[j], t[0], (e < half ? -y[j] : y[j]) * t[1]);
                        }
                    }
                }
            }
            if (h < a.q_heads) {
                if (live)
                    *(u32x4 *)(a.q_out + ((size_t)(t0 + tok) * a.q_heads + h) * d + c0) = pack(x);
                continue;
            }
            const int32_t slot = a.slots[t0 + tok];
            const bool kept = (uint32_t)slot < a.cache.pages << a.cache.page_log2;   // a slot below 0 wraps far past it
            const bool key = h < heads - kv;
            const uint32_t head = h - a.q_heads - (key ? 0 : kv);
            const size_t at = (((size_t)(slot >> a.cache.page_log2) * kv + head) << a.cache.page_log2) +
                              (slot & ((1 << a.cache.page_log2) - 1));
            void *cache = key ? a.cache.k : a.cache.v;
            if (!FP8) {
                if (live && kept)
                    *(u32x4 *)((uint16_t *)cache + at * d + c0) = pack(x);
                continue;
            }
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top = __builtin_fmaxf(top, __builtin_fabsf(live ? x[j] : 0.0f));
            const float scale = div_by_const<448>(group_max<G>(top));
            float q[8];
            div_all<8>(ScaleDiv(scale), x, q);
            u32x2 codes = {cvt_e4m3x4(q[0], q[1], q[2], q[3]), cvt_e4m3x4(q[4], q[5], q[6], q[7])};
            if (scale == 0.0f)
                codes = (u32x2){0, 0};
            if (live && kept) {
                *(u32x2 *)((uint8_t *)cache + at * d + c0) = codes;
                if (c0 == 0)
                    (key ? a.cache.ks : a.cache.vs)[at] = scale;
            }
        }
    }
}

template <int G>
void launch(const RopeArgs &a, hipStream_t st)
{
    const uint32_t heads = a.q_heads + 2 * a.cache.heads;
    // tokens of a workgroup: one, or as many as give every group of lanes an item
    const uint32_t tokens = max(1u, min(MAX_TOKENS, WG / G / heads));
    const dim3 grid((a.t + tokens - 1) / tokens);
    if (a.cache.fp8)
        k_qk_norm_rope<true, G, 2><<<grid, WG, 0, st>>>(a, tokens, heads);
    else
        k_qk_norm_rope<false, G, 2><<<grid, WG, 0, st>>>(a, tokens, heads);
}

} // namespace

hipError_t launch_qk_norm_rope_cache(const RopeArgs &a, hipStream_t st)
{
    if (a.cache.d <= 64)
        launch<8>(a, st);
    else if (a.cache.d <= 128)
        launch<16>(a, st);
    else
        launch<32>(a, st);
    count_launch();
    return hipGetLastError();
}

} // namespace qp
