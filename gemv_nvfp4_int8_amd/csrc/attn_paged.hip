// attn_paged.hip -- attention of new tokens over a paged cache.
//
// One wave per row and query head: 64 keys at a time, one a lane, with the
// running maximum and sum of the softmax; then each lane sums its columns of V.
#include "qp_device.hpp"
#include "qp_launch.hpp"
#include "decoder.hpp"

namespace qp {
namespace {

constexpr float LOG2E = 1.4426950408889634f;

template <bool FP8>
__global__ __launch_bounds__(64) void k_attn_rows(AttnArgs a)
{
    __shared__ float qs[256], ps[64];
    const uint32_t row = blockIdx.x, head = blockIdx.y, lane = threadIdx.x, d = a.cache.d;
    const uint32_t kv_head = head / (a.q_heads / a.cache.heads), pl = a.cache.page_log2;
    int seq = -1;
    for (uint32_t s0 = 0; s0 < a.seqs && seq < 0; s0 += 64) {
        const uint32_t s = s0 + lane;
        bool here = false;
        if (s < a.seqs) {
            const int lo = a.q_start[s], hi = a.q_start[s + 1], len = a.kv_len[s];
            here = lo >= 0 && hi >= lo && (uint32_t)hi <= a.t && (uint32_t)(hi - lo) <= a.max_q && len >= 0 &&
                   (uint32_t)len <= a.width << pl && (uint32_t)lo <= row && row < (uint32_t)hi;
        }
        const uint64_t who = __ballot(here);
        if (who)
            seq = s0 + __builtin_ctzll(who);
    }
    if (seq < 0)
        return;
    const int pos = a.kv_len[seq] - a.q_start[seq + 1] + (int)row;
    const int first = a.window && pos >= (int)a.window ? pos - (int)a.window + 1 : 0;
    for (uint32_t i = lane; i < d; i += 64)
        qs[i] = __uint_as_float((uint32_t)a.q[((size_t)row * a.q_heads + head) * d + i] << 16);
    __syncthreads();
    float m = -INFINITY, l = 0.0f, acc[4] = {0, 0, 0, 0};
    for (int k0 = first; k0 <= pos; k0 += 64) {
        const int key = k0 + (int)lane;
        float s = -INFINITY, vs = 1.0f;
        uint32_t page = 0;
        bool seen = key <= pos;
        if (seen) {
            page = (uint32_t)a.table[(size_t)seq * a.width + (key >> pl)];
            seen = page < a.cache.pages;
        }
        size_t r = 0;
        if (seen) {
            r = (((size_t)page * a.cache.heads + kv_head) << pl) + (key & ((1 << pl) - 1));
            float dot = 0.0f;
            for (uint32_t i = 0; i < d; ++i)
                dot = __builtin_fmaf(qs[i], FP8 ? dec_e4m3(((const uint8_t *)a.cache.k)[r * d + i])
                                                : __uint_as_float((uint32_t)((const uint16_t *)a.cache.k)[r * d + i] << 16), dot);
            if (FP8) {
                dot *= a.cache.ks[r];
                vs = a.cache.vs[r];
            }
            s = dot * (a.scale * LOG2E);
        }
        const float top = __builtin_fmaxf(m, wave_max(s));
        const float base = top == -INFINITY ? 0.0f : top;
        const float p = seen ? exp2f(s - base) : 0.0f;
        const float fade = exp2f(m - base);
        m = top;
        float sum = p;
        for (int off = 32; off; off >>= 1)
            sum += __shfl_xor(sum, off, WAVE);
        l = l * fade + sum;
        for (int c = 0; c < 4; ++c)
            acc[c] *= fade;
        const uint64_t live = __ballot(seen);
        ps[lane] = p * vs;
        __syncthreads();
        for (int j = 0; j < 64; ++j) {
            if (!(live >> j & 1))
                continue;
            const size_t rj = ((size_t)__shfl((uint32_t)(r >> 32), j, WAVE) << 32) | __shfl((uint32_t)r, j, WAVE);
            for (uint32_t c = 0; c < 4; ++c)
                if (lane + 64 * c < d) {
                    const size_t e = rj * d + lane + 64 * c;
                    const float v = FP8 ? dec_e4m3(((const uint8_t *)a.cache.v)[e])
                                        : __uint_as_float((uint32_t)((const uint16_t *)a.cache.v)[e] << 16);
                    acc[c] = __builtin_fmaf(ps[j], v, acc[c]);
                }
        }
        __syncthreads();
    }
    for (uint32_t c = 0; c < 4; ++c)
        if (lane + 64 * c < d)
            a.out[((size_t)row * a.q_heads + head) * d + lane + 64 * c] = (uint16_t)f32_to_bf16(l > 0.0f ? acc[c] / l : l == 0.0f ? 0.0f : l);
}

} // namespace

uint64_t paged_attention_work(uint32_t, uint32_t, uint32_t, uint32_t, uint32_t, uint32_t)
{
    return 16;
}

hipError_t launch_paged_attention(const AttnArgs &a, hipStream_t st)
{
    const dim3 grid(a.t, a.q_heads);
    if (a.cache.fp8)
        k_attn_rows<true><<<grid, 64, 0, st>>>(a);
    else
        k_attn_rows<false><<<grid, 64, 0, st>>>(a);
    count_launch();
    return hipGetLastError();
}

} // namespace qp
