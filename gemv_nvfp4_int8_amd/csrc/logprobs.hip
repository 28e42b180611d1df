// logprobs.hip -- log probabilities of given tokens, entropy and the most
// probable tokens of rows of logits.
//
// One workgroup per row: the largest logit, then the sums, then `top` times the
// next largest (of equal ones the lowest token).
#include "qp_device.hpp"
#include "qp_launch.hpp"
#include "decoder.hpp"

namespace qp {
namespace {

constexpr uint32_t WG = 256;

template <bool F32>
__global__ __launch_bounds__(WG) void k_logprobs(LogprobArgs a)
{
    __shared__ uint64_t best[WG];
    __shared__ float sums[2][WG];
    const uint32_t row = blockIdx.x, tid = threadIdx.x;
    auto logit = [&](uint32_t i) {
        const size_t e = (size_t)row * a.vocab + i;
        return F32 ? ((const float *)a.logits)[e] : __uint_as_float((uint32_t)((const uint16_t *)a.logits)[e] << 16);
    };
    // larger key: larger value, or the same and a lower index; never 0
    auto key = [](float x, uint32_t i) {
        const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);
        return (uint64_t)(u >> 31 ? ~u : u | 0x80000000u) << 32 | (0xFFFFFFFFu - i);
    };
    auto largest_below = [&](uint64_t limit) {
        uint64_t k = 0;
        for (uint32_t i = tid; i < a.vocab; i += WG) {
            const uint64_t c = key(logit(i), i);
            if (c < limit && c > k)
                k = c;
        }
        best[tid] = k;
        __syncthreads();
        for (uint32_t h = WG / 2; h; h >>= 1) {
            if (tid < h && best[tid + h] > best[tid])
                best[tid] = best[tid + h];
            __syncthreads();
        }
        k = best[0];
        __syncthreads();
        return k;
    };
    uint64_t k = largest_below(~0ull);
    const float m = logit(0xFFFFFFFFu - (uint32_t)k), base = m == -INFINITY ? 0.0f : m;
    float s = 0.0f, t = 0.0f;
    for (uint32_t i = tid; i < a.vocab; i += WG) {
        const float y = logit(i) - base, e = expf(y);
        s += e;
        t += e > 0.0f ? e * y : 0.0f;
    }
    sums[0][tid] = s;
    sums[1][tid] = t;
    __syncthreads();
    for (uint32_t h = WG / 2; h; h >>= 1) {
        if (tid < h)
            for (int j = 0; j < 2; ++j)
                sums[j][tid] += sums[j][tid + h];
        __syncthreads();
    }
    s = sums[0][0];
    t = sums[1][0];
    const float norm = s > 0.0f ? logf(s) : 0.0f;
    if (tid == 0 && a.targets) {
        const uint32_t at = (uint32_t)a.targets[row];
        a.logprob[row] = at < a.vocab ? logit(at) - base - norm : 0.0f;
    }
    if (tid == 0 && a.entropy)
        a.entropy[row] = s > 0.0f ? norm - t / s : 0.0f;
    for (uint32_t n = 0; n < a.top; ++n) {
        const uint32_t id = 0xFFFFFFFFu - (uint32_t)k;
        if (tid == 0 && id < a.vocab) {
            a.ids[(size_t)row * a.top + n] = (int32_t)id;
            a.top_logprobs[(size_t)row * a.top + n] = logit(id) - base - norm;
        }
        if (n + 1 < a.top)
            k = largest_below(k);
    }
}

} // namespace

uint64_t token_logprobs_work(uint32_t, uint32_t, uint32_t)
{
    return 16;
}

hipError_t launch_token_logprobs(const LogprobArgs &a, hipStream_t st)
{
    if (a.f32)
        k_logprobs<true><<<a.rows, WG, 0, st>>>(a);
    else
        k_logprobs<false><<<a.rows, WG, 0, st>>>(a);
    count_launch();
    return hipGetLastError();
}

} // namespace qp
