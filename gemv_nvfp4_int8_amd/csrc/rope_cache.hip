// rope_cache.hip -- norms of queries and keys, rotary positions, and the paged
// cache's new entries, in one pass over the output of the q/k/v product.
//
// A head is taken by G lanes (8, 16 or 32: the next power of two of d/8), 16
// bytes each, so that its sum of squares and its largest magnitude are a few
// cross-lane steps.  A lane's partners of the half layout lie rot/2 further on or
// back, in another lane's 16 bytes, and come from that lane when they are normed
// (8192 tokens of 32 + 2 * 8 heads of 128: 33 us; loaded and normed once more, 41:
// the vector instructions bound it then).  Cosines
// and sines are the same for all heads of a token: one thread a pair computes them
// into LDS while the heads' loads are on their way; what is not turned has the
// angle 0 there and a partner of 0, so that all lanes do the same (in neighbouring
// pairs, whose partners are what they are, it is kept by a choice instead).
//
// Bound by HBM when large: 8192 tokens of 32 + 2 * 8 heads of 128 take 33 us, 6.1 TB/s
// read and written; 2047 of 40 + 2 * 4 with an E4M3 cache 9.9 us (4.9 TB/s).  A single
// token takes 4 us: a launch, one trip to memory, the sums across lanes.
#include <type_traits>

#include "qp_device.hpp"
#include "qp_launch.hpp"
#include "decoder.hpp"

namespace qp {
namespace {

constexpr uint32_t WG = 256;
constexpr uint32_t MAX_TOKENS = 8;         // of a workgroup
constexpr uint32_t MAX_HALF = 128;

// How pairs lie: 8 partners in one lane's 16 bytes (rot/2 a multiple of 8), in the
// same lane, anywhere, or (rot = d = 64 or 128) in the lane G/2 further on or back,
// from which data-parallel moves bring them (d = 128, E4M3: 33.5 us where the general
// exchange through LDS' crossbar takes 35.2; at d = 256, where such a move would cross
// rows of 16 lanes, nothing is gained).
enum Layout { HALF, PAIRS, HALF_ANY, FULL };

// All lanes of G: op over their values, within 16 lanes by data-parallel moves.
template <int G, typename Op>
__device__ __forceinline__ float over_group(float v, Op op)
{
    auto moved = [](float x, auto ctrl) {
        return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), decltype(ctrl)::value, 0xf, 0xf, false));
    };
    v = op(v, moved(v, std::integral_constant<int, 0xB1>()));           // lane ^ 1
    v = op(v, moved(v, std::integral_constant<int, 0x4E>()));           // lane ^ 2
    v = op(v, moved(v, std::integral_constant<int, 0x141>()));          // 7 - lane, of 8
    if (G >= 16)
        v = op(v, moved(v, std::integral_constant<int, 0x140>()));      // 15 - lane, of 16
    if (G >= 32)
        v = op(v, __shfl_xor(v, 16, WAVE));
    return v;
}

// The value of the lane G/2 further on or back in the group.
template <int G>
__device__ __forceinline__ float across(float x)
{
    auto moved = [](float x, auto ctrl) {
        return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), decltype(ctrl)::value, 0xf, 0xf, false));
    };
    if constexpr (G == 8)                  // 7 - lane, then that of 4 turned round
        return moved(moved(x, std::integral_constant<int, 0x141>()), std::integral_constant<int, 0x1B>());
    else
        return moved(x, std::integral_constant<int, 0x128>());          // turned by 8, of 16
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

// A workgroup has one token, whose heads its groups of G lanes take in turn, U at a
// time so that a lane has their loads in flight together; or (fewer heads than
// groups) `tokens` of them, a head a group.
template <bool FP8, int G, Layout L>
__global__ __launch_bounds__(WG) void k_qk_norm_rope(RopeArgs a, uint32_t tokens, uint32_t heads)
{
    constexpr uint32_t NG = WG / G;
    constexpr int U = 3;
    // a token's cosines and sines, then eight times those of the angle 0
    __shared__ __attribute__((aligned(16))) f32x2 turn[MAX_TOKENS][MAX_HALF + 8];
    const uint32_t d = a.cache.d, kv = a.cache.heads, half = a.rot / 2;
    const uint32_t t0 = blockIdx.x * tokens, nt = min(tokens, a.t - t0);
    const uint32_t group = threadIdx.x / G, c0 = 8 * (threadIdx.x % G);
    const bool live = c0 < d;
    const uint32_t nth = tokens == 1 ? 0 : group / heads, tok = t0 + nth;
    const uint32_t h0 = tokens == 1 ? group : group - nth * heads;
    // where the lane's angles are, and its partners
    const bool turned = live && c0 < a.rot;
    const uint32_t angle = L == PAIRS ? c0 / 2 : !turned ? MAX_HALF : c0 < half ? c0 : c0 - half;
    const uint32_t from = threadIdx.x % WAVE / G * G + (turned ? c0 < half ? c0 + half : c0 - half : c0) / 8;

    u32x4 own[U];
    auto load = [&](uint32_t h) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            own[u] = (u32x4){0, 0, 0, 0};
            const uint32_t head = h + u * NG;
            if (head >= heads || nth >= nt || !live)
                continue;
            own[u] = *(const u32x4 *)(a.qkv + ((size_t)tok * heads + head) * d + c0);
        }
    };
    load(h0);
    for (uint32_t i = threadIdx.x; i < nt * (MAX_HALF + 8); i += WG) {
        const uint32_t n = i / (MAX_HALF + 8), j = i % (MAX_HALF + 8);
        f32x2 cs = {1.0f, -0.0f};          // x * 1 + 0 * -0 is x, -0 too
        if (j < half) {
            // the angle in turns, in 64 bits: the whole turns of far positions drop
            // out before anything is rounded to 32
            const double turns = (double)a.pos[t0 + n] * (double)a.inv_freq[j] * 0.15915494309189533577;
            float s, c;
            sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
            cs = (f32x2){c * a.rope_scale, s * a.rope_scale};
        }
        turn[n][j] = cs;
    }
    int32_t slot = -1;
    if (nth < nt)
        slot = a.slots[tok];
    __syncthreads();
    if (nth >= nt)
        return;

    float c[8], s[8];                      // of the lane's eight entries (PAIRS: of its four pairs)
    if (L != HALF_ANY) {
#pragma unroll
        for (int j = 0; j < (L == PAIRS ? 4 : 8); j += 2) {
            const f32x4 v = *(const f32x4 *)&turn[nth][angle + j];
            c[j] = v[0];
            s[j] = v[1];
            c[j + 1] = v[2];
            s[j + 1] = v[3];
        }
        if ((L == HALF || L == FULL) && c0 < half) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[j] = -s[j];
        }
    }
    const bool kept = (uint32_t)slot < a.cache.pages << a.cache.page_log2;       // a slot below 0 wraps far past it
    const float of_d = 1.0f / (float)d;
    for (uint32_t h = h0; h < heads; h += U * NG) {
        if (h != h0)
            load(h);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t head = h + u * NG;
            if (head >= heads)
                break;                                  // whole groups leave together
            const bool value = head >= heads - kv;
            float x[8];
            unpack(own[u], x);
            if (!value) {
                const uint16_t *w = head < a.q_heads ? a.qw : a.kw;
                float rstd = 1.0f, y[8];
                if (w) {
                    float ss = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        ss = __builtin_fmaf(x[j], x[j], ss);
                    ss = over_group<G>(ss, [](float p, float q) { return p + q; });
                    rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, of_d, a.eps));
                    u32x4 g = {0, 0, 0, 0};
                    if (live)
                        g = *(const u32x4 *)(w + c0);
                    unpack(g, y);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[j] = x[j] * rstd * y[j];
                }
                if constexpr (L == PAIRS) {
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        // (a pair that is not turned may hold an infinity, which times 0 is NaN)
                        const float lo = x[j], hi = x[j + 1];
                        const bool pair = c0 + j < a.rot;
                        x[j] = pair ? __builtin_fmaf(lo, c[j / 2], -(hi * s[j / 2])) : lo;
                        x[j + 1] = pair ? __builtin_fmaf(hi, c[j / 2], lo * s[j / 2]) : hi;
                    }
                } else if constexpr (L == FULL) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[j] = __builtin_fmaf(x[j], c[j], across<G>(x[j]) * s[j]);
                } else if constexpr (L == HALF) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float z = __shfl(x[j], from, WAVE);
                        x[j] = __builtin_fmaf(x[j], c[j], (turned ? z : 0.0f) * s[j]);
                    }
                } else if (turned) {
                    const uint16_t *raw = a.qkv + ((size_t)tok * heads + head) * d;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t e = c0 + j;
                        if (e >= a.rot)
                            continue;
                        const uint32_t o = e < half ? e + half : e - half;
                        const f32x2 t = turn[nth][e < half ? e : e - half];
                        float z = __uint_as_float((uint32_t)raw[o] << 16);
                        if (w)
                            z = z * rstd * __uint_as_float((uint32_t)w[o] << 16);
                        x[j] = __builtin_fmaf(x[j], t[0], (e < half ? -z : z) * t[1]);
                    }
                }
            }
            if (head < a.q_heads) {
                if (live)
                    *(u32x4 *)(a.q_out + ((size_t)tok * a.q_heads + head) * d + c0) = pack(x);
                continue;
            }
            const uint32_t kv_head = head - a.q_heads - (value ? kv : 0);
            const size_t at = (((size_t)((uint32_t)slot >> a.cache.page_log2) * kv + kv_head) << a.cache.page_log2) +
                              ((uint32_t)slot & ((1u << a.cache.page_log2) - 1));
            void *cache = value ? a.cache.v : a.cache.k;
            if (!FP8) {
                if (live && kept)
                    *(u32x4 *)((uint16_t *)cache + at * d + c0) = pack(x);
                continue;
            }
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top = __builtin_fmaxf(top, __builtin_fabsf(live ? x[j] : 0.0f));
            const float scale = div_by_const<448>(over_group<G>(top, [](float p, float q) { return __builtin_fmaxf(p, q); }));
            float q[8];
            div_all<8>(ScaleDiv(scale), x, q);
            u32x2 codes = {cvt_e4m3x4(q[0], q[1], q[2], q[3]), cvt_e4m3x4(q[4], q[5], q[6], q[7])};
            if (scale == 0.0f)
                codes = (u32x2){0, 0};
            if (live && kept) {
                *(u32x2 *)((uint8_t *)cache + at * d + c0) = codes;
                if (c0 == 0)
                    (value ? a.cache.vs : a.cache.ks)[at] = scale;
            }
        }
    }
}

template <int G, Layout L>
void launch_layout(const RopeArgs &a, hipStream_t st)
{
    const uint32_t heads = a.q_heads + 2 * a.cache.heads;
    const uint32_t tokens = max(1u, min(MAX_TOKENS, WG / G / heads));
    const dim3 grid((a.t + tokens - 1) / tokens);
    if (a.cache.fp8)
        k_qk_norm_rope<true, G, L><<<grid, WG, 0, st>>>(a, tokens, heads);
    else
        k_qk_norm_rope<false, G, L><<<grid, WG, 0, st>>>(a, tokens, heads);
}

template <int G>
void launch(const RopeArgs &a, hipStream_t st)
{
    if (a.interleaved)
        launch_layout<G, PAIRS>(a, st);
    else if (G <= 16 && a.rot == 8 * G && a.cache.d == 8 * G)
        launch_layout<(G < 16 ? G : 16), FULL>(a, st);
    else if (a.rot % 16 == 0)
        launch_layout<G, HALF>(a, st);
    else
        launch_layout<G, HALF_ANY>(a, st);
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
