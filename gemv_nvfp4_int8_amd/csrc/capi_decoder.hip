// capi_decoder.hip -- the extern "C" boundary of the operators declared in
// include/qproj_decoder.h.  As in capi.hip, every argument is checked on the
// host before anything is enqueued; nothing allocates or synchronises.
#include <cfloat>
#include <cmath>

#include "capi_check.hpp"
#include "decoder.hpp"
#include "../../include/qproj_decoder.h"

using namespace qp::capi;

namespace {

int check_cache(int fmt, const void *k, const void *v, const float *ks, const float *vs,
                uint32_t kv_heads, uint32_t d, uint32_t pages, uint32_t page_size)
{
    if (fmt != QP_KV_BF16 && fmt != QP_KV_FP8_ROW)
        return QP_ERR_FORMAT;
    if (int e = check_ptrs({k, v}))
        return e;
    if (fmt == QP_KV_FP8_ROW)
        if (int e = check_ptrs({ks, vs}))
            return e;
    if (kv_heads == 0 || kv_heads > 65535 || d == 0 || d > 256 || d % 16 != 0 || pages == 0 || page_size < 16 ||
        page_size > 4096 || (page_size & (page_size - 1)) != 0 || !fits(pages, page_size) ||
        !fits(kv_heads, (uint64_t)page_size * d))
        return QP_ERR_SHAPE;
    return QP_OK;
}

qp::PagedCache cache_of(int fmt, const void *k, const void *v, const float *ks, const float *vs,
                        uint32_t kv_heads, uint32_t d, uint32_t pages, uint32_t page_size)
{
    const bool fp8 = fmt == QP_KV_FP8_ROW;
    return {const_cast<void *>(k), const_cast<void *>(v), fp8 ? const_cast<float *>(ks) : nullptr,
            fp8 ? const_cast<float *>(vs) : nullptr, pages, kv_heads, d,
            (uint32_t)__builtin_ctz(page_size), fp8};
}

bool attention_shape(uint32_t t, uint32_t seqs, uint32_t q_heads, uint32_t kv_heads, uint32_t d)
{
    return t != 0 && seqs != 0 && q_heads != 0 && kv_heads != 0 && kv_heads <= 65535 &&
           q_heads % kv_heads == 0 && d != 0 && d <= 256 && d % 16 == 0 && (uint64_t)t * q_heads <= MAX_ELEMS &&
           fits((uint64_t)t * q_heads, d) && seqs <= MAX_ELEMS - 1;
}

// (a launch has a workgroup of 256 a row, and holds fewer than 2^32 threads)
bool logits_shape(uint32_t rows, uint32_t vocab)
{
    return rows != 0 && vocab != 0 && rows < 1u << 24 && fits(rows, vocab);
}

} // namespace

extern "C" {

int rope_inv_freq(float *inv_freq, uint32_t rot, double base, int scaling, double factor, double low,
                  double high, uint32_t original)
{
    if (!inv_freq)
        return QP_ERR_NULL;
    if (scaling < QP_ROPE_PLAIN || scaling > QP_ROPE_RAMP)
        return QP_ERR_FORMAT;
    if (rot < (scaling == QP_ROPE_BASE ? 4u : 2u) || rot % 2 != 0 || rot > QP_ROPE_MAX_ROT)
        return QP_ERR_SHAPE;
    const bool blend = scaling == QP_ROPE_WAVELENGTH || scaling == QP_ROPE_RAMP;
    if (!(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor) ||
        (blend && (!(low > 0.0) || !(high > low) || !std::isfinite(high) || original < 1)))
        return QP_ERR_RANGE;
    const double two_pi = 6.283185307179586476925286766559;
    if (scaling == QP_ROPE_BASE)
        base *= std::pow(factor, (double)rot / (rot - 2));
    // the pair (a real number) that makes `turns` turns over the original context
    auto pair_of = [&](double turns) {
        return rot * std::log(original / (turns * two_pi)) / (2.0 * std::log(base));
    };
    double from = 0.0, to = 1.0;
    if (scaling == QP_ROPE_RAMP) {
        from = std::fmax(std::floor(pair_of(high)), 0.0);
        to = std::fmin(std::ceil(pair_of(low)), rot - 1.0);      // (may lie behind the last pair)
        to = std::fmax(to, from + 1e-3);          // both in one pair: a step behind it
    }
    for (uint32_t i = 0; i < rot / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot);
        double keep = 1.0;                        // the share that is not divided
        if (scaling == QP_ROPE_LINEAR)
            keep = 0.0;
        else if (scaling == QP_ROPE_WAVELENGTH)
            keep = std::fmin(std::fmax((original * f / two_pi - low) / (high - low), 0.0), 1.0);
        else if (scaling == QP_ROPE_RAMP)
            keep = 1.0 - std::fmin(std::fmax((i - from) / (to - from), 0.0), 1.0);
        inv_freq[i] = (float)(f * keep + f / factor * (1.0 - keep));
    }
    return QP_OK;
}

int qk_norm_rope_cache(const uint16_t *qkv, const uint16_t *q_norm, const uint16_t *k_norm, float eps,
                       const int32_t *positions, const float *inv_freq, float rope_scale, int layout,
                       uint32_t rot, const int32_t *slots, int kv_format, void *k_cache, void *v_cache,
                       float *k_scale, float *v_scale, uint16_t *q_out, uint32_t t, uint32_t q_heads,
                       uint32_t kv_heads, uint32_t d, uint32_t pages, uint32_t page_size, void *stream)
{
    if (int e = check_ptrs({qkv, positions, slots, q_out}))
        return e;
    if (int e = check_cache(kv_format, k_cache, v_cache, k_scale, v_scale, kv_heads, d, pages, page_size))
        return e;
    if ((q_norm == nullptr) != (k_norm == nullptr) || (rot != 0 && !inv_freq))
        return QP_ERR_NULL;
    if (!aligned16(q_norm) || !aligned16(k_norm) || !aligned16(inv_freq))
        return QP_ERR_ALIGN;
    if (layout != QP_ROPE_HALF && layout != QP_ROPE_INTERLEAVED)
        return QP_ERR_FORMAT;
    const uint64_t row = ((uint64_t)q_heads + 2 * (uint64_t)kv_heads) * d;
    if (t == 0 || q_heads == 0 || rot % 2 != 0 || rot > d || row > MAX_ELEMS || !fits(t, row))
        return QP_ERR_SHAPE;
    if ((q_norm && (!(eps >= FLT_MIN) || !std::isfinite(eps))) || !std::isfinite(rope_scale))
        return QP_ERR_RANGE;               // (a smaller eps is 0 to the reciprocal root, and a head of zeros NaN)
    return done(qp::launch_qk_norm_rope_cache(
        {qkv, q_norm, k_norm, positions, slots, inv_freq, q_out, eps, rope_scale, t, q_heads, rot,
         layout == QP_ROPE_INTERLEAVED,
         cache_of(kv_format, k_cache, v_cache, k_scale, v_scale, kv_heads, d, pages, page_size)},
        S(stream)));
}

uint64_t paged_attention_workspace(uint32_t t, uint32_t seqs, uint32_t max_q, uint32_t q_heads,
                                   uint32_t kv_heads, uint32_t d)
{
    if (!attention_shape(t, seqs, q_heads, kv_heads, d) || max_q < 1 || max_q > t)
        return 0;
    return qp::paged_attention_work(t, seqs, max_q, q_heads, kv_heads, d);
}

int paged_attention(const uint16_t *q, int kv_format, const void *k_cache, const void *v_cache,
                    const float *k_scale, const float *v_scale, const int32_t *page_table,
                    const int32_t *q_start, const int32_t *kv_len, float scale, uint32_t window,
                    void *workspace, uint64_t workspace_bytes, uint16_t *out, uint32_t t, uint32_t seqs,
                    uint32_t max_q, uint32_t q_heads, uint32_t kv_heads, uint32_t d, uint32_t pages,
                    uint32_t page_size, uint32_t table_width, void *stream)
{
    if (int e = check_ptrs({q, page_table, q_start, kv_len, workspace, out}))
        return e;
    if (int e = check_cache(kv_format, k_cache, v_cache, k_scale, v_scale, kv_heads, d, pages, page_size))
        return e;
    if (!attention_shape(t, seqs, q_heads, kv_heads, d) || table_width == 0 || !fits(seqs, table_width) ||
        (uint64_t)table_width * page_size >= 1u << 27 || (uint64_t)seqs * table_width * page_size >= 1ull << 38)
        return QP_ERR_SHAPE;               // (tiles of 32 keys or more are counted in 32 bits, 512 blocks at a time)
    if (max_q < 1 || max_q > t || !(scale > 0.0f) || !std::isfinite(scale * 1.4426950408889634f))
        return QP_ERR_RANGE;               // (scores are kept in base 2)
    if (workspace_bytes < qp::paged_attention_work(t, seqs, max_q, q_heads, kv_heads, d))
        return QP_ERR_SCRATCH;
    return done(qp::launch_paged_attention(
        {q, out, page_table, q_start, kv_len, workspace, scale, window < 1u << 27 ? window : 0, t, seqs, max_q, q_heads, table_width,
         cache_of(kv_format, k_cache, v_cache, k_scale, v_scale, kv_heads, d, pages, page_size)},
        S(stream)));
}

uint64_t token_logprobs_workspace(uint32_t rows, uint32_t vocab, uint32_t top)
{
    if (!logits_shape(rows, vocab) || top > QP_LOGPROBS_MAX_TOP || top > vocab)
        return 0;
    return qp::token_logprobs_work(rows, vocab, top);
}

int token_logprobs(const void *logits, int logits_format, const int32_t *targets, float *logprob,
                   float *entropy, int32_t *top_ids, float *top_logprobs, void *workspace,
                   uint64_t workspace_bytes, uint32_t rows, uint32_t vocab, uint32_t top, void *stream)
{
    if (int e = check_ptrs({logits, workspace}))
        return e;
    if ((targets == nullptr) != (logprob == nullptr) || (top != 0 && (!top_ids || !top_logprobs)) ||
        (!targets && !entropy && top == 0))
        return QP_ERR_NULL;
    if (!aligned16(targets) || !aligned16(logprob) || !aligned16(entropy) ||
        (top != 0 && (!aligned16(top_ids) || !aligned16(top_logprobs))))
        return QP_ERR_ALIGN;
    if (logits_format != QP_LOGITS_BF16 && logits_format != QP_LOGITS_F32)
        return QP_ERR_FORMAT;
    if (!logits_shape(rows, vocab))
        return QP_ERR_SHAPE;
    if (top > QP_LOGPROBS_MAX_TOP || top > vocab)
        return QP_ERR_RANGE;
    if (workspace_bytes < qp::token_logprobs_work(rows, vocab, top))
        return QP_ERR_SCRATCH;
    return done(qp::launch_token_logprobs({logits, targets, logprob, entropy, top_ids, top_logprobs, workspace,
                                           rows, vocab, top, logits_format == QP_LOGITS_F32},
                                          S(stream)));
}

} // extern "C"
