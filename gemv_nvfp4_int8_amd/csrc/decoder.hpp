// decoder.hpp -- host-side launchers of the operators of qproj_decoder.h.
// Arguments are assumed validated by capi_decoder.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qp {

// A paged cache: [pages, heads, 1 << page_log2, d], K and V each.
struct PagedCache {
    void *k, *v;
    float *ks, *vs;               // null for BF16
    uint32_t pages, heads, d, page_log2;
    bool fp8;
};

struct RopeArgs {
    const uint16_t *qkv, *qw, *kw;
    const int32_t *pos, *slots;
    const float *inv_freq;
    uint16_t *q_out;
    float eps, rope_scale;
    uint32_t t, q_heads, rot;
    bool interleaved;
    PagedCache cache;
};
hipError_t launch_qk_norm_rope_cache(const RopeArgs &a, hipStream_t st);

struct AttnArgs {
    const uint16_t *q;
    uint16_t *out;
    const int32_t *table, *q_start, *kv_len;
    void *work;
    float scale;
    uint32_t window, t, seqs, max_q, q_heads, width;
    PagedCache cache;
};
uint64_t paged_attention_work(uint32_t t, uint32_t seqs, uint32_t max_q, uint32_t q_heads,
                              uint32_t kv_heads, uint32_t d);
hipError_t launch_paged_attention(const AttnArgs &a, hipStream_t st);

struct LogprobArgs {
    const void *logits;
    const int32_t *targets;
    float *logprob, *entropy;
    int32_t *ids;
    float *top_logprobs;
    void *work;
    uint32_t rows, vocab, top;
    bool f32;
};
uint64_t token_logprobs_work(uint32_t rows, uint32_t vocab, uint32_t top);
hipError_t launch_token_logprobs(const LogprobArgs &a, hipStream_t st);

} // namespace qp
