/*
 * qproj_decoder.h -- what a decoder's step runs between and after the
 * projections of qproj.h and qproj_layer.h, in the same library: the norms and
 * rotary positions of queries and keys with the paged key/value cache they
 * fill, attention over that cache, and the log probabilities at the end.
 *
 * The conventions of qproj.h hold (device pointers to dense row-major memory,
 * 16-byte alignment, caller-owned buffers and scratch, no allocation, no
 * synchronisation, work enqueued on `stream`, host-side checks that enqueue
 * nothing).  What a call writes overlaps nothing else that it is given.  What
 * the host cannot see (slots, page numbers, lengths, tokens) is checked on the
 * GPU: a value that fits no buffer is skipped as stated at the operator and
 * never leads outside one.
 */
#ifndef QPROJ_DECODER_H
#define QPROJ_DECODER_H

#include "qproj.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The paged cache: K and V as [pages, kv_heads, page_size, d] each,
 *   QP_KV_BF16     BF16, no scales (the pointers are not used, may be NULL);
 *   QP_KV_FP8_ROW  E4M3 with F32 scales [pages, kv_heads, page_size], one for
 *                  each position and head (scale = amax/448, one IEEE division
 *                  of the F32 value by it, round to nearest even, a zero row
 *                  as scale 0 and +0 codes).
 * page_size is a power of two from 16 to 4096, d a multiple of 16 up to 256,
 * kv_heads at most 65535, pages * page_size < 2^31, a page (kv_heads *
 * page_size * d) below 2^31 elements; K and V as a whole may be larger than
 * that. */
enum qp_kv_format { QP_KV_BF16 = 0, QP_KV_FP8_ROW = 1 };

/* Which entries of a head one rotation turns: i and i + rot/2, or 2i and 2i+1. */
enum qp_rope_layout { QP_ROPE_HALF = 0, QP_ROPE_INTERLEAVED = 1 };

/* How rotary frequencies follow from base^(-2i/rot) for contexts `factor`
 * times as long as the model's `original` one (r = the turns that pair i makes
 * over `original` positions):
 *   QP_ROPE_PLAIN       as they are;
 *   QP_ROPE_LINEAR      divided by factor (positions pressed together);
 *   QP_ROPE_BASE        base * factor^(rot/(rot-2)) in the place of base;
 *   QP_ROPE_WAVELENGTH  divided by factor where r < low, kept where r > high,
 *                       and between them the mix of both, linear in r;
 *   QP_ROPE_RAMP        kept up to the pair that makes `high` turns (its index
 *                       rounded down, at least 0), divided by factor from the
 *                       pair that makes `low` on (rounded up, at most rot - 1:
 *                       it may lie behind the last pair, rot/2 - 1), and between
 *                       them the mix of both, linear in the pair's index. */
enum qp_rope_scaling {
    QP_ROPE_PLAIN = 0,
    QP_ROPE_LINEAR = 1,
    QP_ROPE_BASE = 2,
    QP_ROPE_WAVELENGTH = 3,
    QP_ROPE_RAMP = 4
};

/* Fills inv_freq [rot/2], a HOST array, computed in 64 bits and rounded once.
 * rot even, from 2 (QP_ROPE_BASE: 4) to QP_ROPE_MAX_ROT, base > 1, factor >= 1,
 * and for the last two 0 < low < high and original >= 1, else QP_ERR_RANGE
 * (QP_ERR_SHAPE for rot, QP_ERR_FORMAT for an unknown scaling).  Launches
 * nothing. */
#define QP_ROPE_MAX_ROT 256
int rope_inv_freq(float *inv_freq, uint32_t rot, double base, int scaling, double factor,
                  double low, double high, uint32_t original);

/* ------------------------------------------------------------------------
 * Norms of queries and keys, rotary positions, and the cache's new entries, in
 * one pass over the q/k/v product's output.
 *   qkv [t, (q_heads + 2 kv_heads) d] BF16: a token's query heads, then its key
 *   heads, then its value heads.  For each query and key head x:
 *     y = x / sqrt(mean(x^2) + eps) * weight        (no norm: y = x)
 *     the first rot entries of y turned in pairs (a, b), c and s being cos and
 *     sin of position * inv_freq[i], times rope_scale:
 *       (a, b) -> (a c - b s, b c + a s);  the others as they are
 *   all in F32 and rounded once: queries to q_out [t, q_heads, d] BF16, keys and
 *   values (these untouched) to the cache at slot = page * page_size + offset.
 * q_norm, k_norm [d] BF16, both or neither (NULL: no norm, eps unused);
 * positions [t], slots [t] int32; inv_freq [rot/2] F32 (NULL where rot is 0).
 * The product position * inv_freq is taken in 64 bits, so that far positions
 * lose nothing.  A slot outside 0..pages*page_size-1 (padding: -1) writes
 * nothing to the cache.  Two tokens with one slot: which of them each 16 bytes
 * of the entry hold is unspecified.  A token's outputs depend on it alone.
 * Refusals: zero extents, d, page_size, t * (q_heads + 2 kv_heads) * d >= 2^31,
 * rot odd or larger than d: QP_ERR_SHAPE; unknown format or layout:
 * QP_ERR_FORMAT; eps (with norms) not finite or below F32's smallest normal
 * number, 2^-126, or rope_scale not finite: QP_ERR_RANGE; one of q_norm and k_norm alone: QP_ERR_NULL.
 * q_heads need not be a multiple of kv_heads here.
 * ---------------------------------------------------------------------- */
int qk_norm_rope_cache(const uint16_t *qkv, const uint16_t *q_norm, const uint16_t *k_norm,
                       float eps, const int32_t *positions, const float *inv_freq,
                       float rope_scale, int layout, uint32_t rot, const int32_t *slots,
                       int kv_format, void *k_cache, void *v_cache, float *k_scale,
                       float *v_scale, uint16_t *q_out, uint32_t t, uint32_t q_heads,
                       uint32_t kv_heads, uint32_t d, uint32_t pages, uint32_t page_size,
                       void *stream);

/* ------------------------------------------------------------------------
 * Attention of new tokens over the paged cache, for decode (one token a
 * sequence), verify batches, chunks of a prompt and whole prompts alike.
 *   q, out [t, q_heads, d] BF16; query head h reads kv head
 *   h / (q_heads / kv_heads).
 *   Sequence s has the rows q_start[s] .. q_start[s+1]-1 of q (q_start
 *   [seqs+1]) and kv_len[s] positions in the cache, its new tokens (which the
 *   cache already holds) the last of them; position p lies in page
 *   page_table[s, p / page_size] (page_table [seqs, table_width]) at offset
 *   p % page_size.  All int32.
 *   The row of position p attends to positions 0..p or, with a window w > 0, to
 *   max(0, p-w+1)..p:
 *     out = bf16( sum_j v_j e^(scale q.k_j - m) / sum_j e^(scale q.k_j - m) ).
 * A row with nothing to attend to (p < 0, where kv_len is less than the
 * sequence's rows; or holes only) gives zeros.  Rows that belong to no sequence
 * are left as they were.  max_q is the most rows of a sequence (a bound; it and
 * the sizes choose the kernel).
 * Scores, maxima, sums and outputs are F32; the probabilities (with an E4M3
 * cache times V's scale) that the matrix cores multiply with V are rounded to
 * BF16, by up to 2^-8, or, where few rows meet a BF16 cache, to two such numbers,
 * by up to 2^-16; their sum is of the unrounded ones.  The sum over the line may
 * be 2^9 times the formula's before it is divided: V of 2^92 and more may
 * overflow it.  An E4M3 cache's scales of V count as the nearest number of 0 to
 * 3.4e38 (NaN as 0).
 * A score of -inf has probability 0 (a row of nothing else gives zeros as well),
 * one of +inf or NaN makes the row NaN.  NaN or an infinity in V makes that
 * element of the rows that attend to it NaN or an infinity (which of them is
 * unspecified).  What the cache holds at a position that a row does not attend
 * to, NaN and infinities included, has no influence on that row.
 * No atomics: the same call gives the same bits; another batch may change a
 * row's last bits.
 * A page number outside 0..pages-1 is a hole: none of its positions is
 * attended to.  A sequence whose numbers do not fit (q_start below 0, falling or
 * past t, more than max_q rows, kv_len below 0 or past table_width *
 * page_size) is left out: its rows are left as they were.  A row that two
 * sequences have (where q_start falls between them) holds either's result.
 * workspace: caller-owned scratch of paged_attention_workspace(...) bytes (fewer
 * is QP_ERR_SCRATCH; enough for a max_q is enough for a smaller one), contents
 * before and after unspecified, not shared by calls that may overlap.
 * Refusals: zero extents, q_heads not a multiple of kv_heads, d, page_size,
 * t * q_heads * d, pages * page_size or seqs * table_width of 2^31 or more,
 * table_width * page_size of 2^27 or more, seqs * table_width * page_size of
 * 2^38 or more: QP_ERR_SHAPE; max_q outside 1..t, scale not positive and
 * finite, also times log2(e): QP_ERR_RANGE; unknown format: QP_ERR_FORMAT.
 * ---------------------------------------------------------------------- */
uint64_t paged_attention_workspace(uint32_t t, uint32_t seqs, uint32_t max_q, uint32_t q_heads,
                                   uint32_t kv_heads, uint32_t d);
int paged_attention(const uint16_t *q, int kv_format, const void *k_cache, const void *v_cache,
                    const float *k_scale, const float *v_scale, const int32_t *page_table,
                    const int32_t *q_start, const int32_t *kv_len, float scale, uint32_t window,
                    void *workspace, uint64_t workspace_bytes, uint16_t *out, uint32_t t,
                    uint32_t seqs, uint32_t max_q, uint32_t q_heads, uint32_t kv_heads,
                    uint32_t d, uint32_t pages, uint32_t page_size, uint32_t table_width,
                    void *stream);

/* ------------------------------------------------------------------------
 * Log probabilities of given tokens, entropy and the most probable tokens of
 * rows of logits, in one pass over them.
 *   logits [rows, vocab], BF16 or F32; targets [rows] int32;
 *   logprob [rows] = x[target] - lse(x);  entropy [rows] = -sum p ln p;
 *   top_ids, top_logprobs [rows, top]: the `top` largest logits, largest first,
 *   of equal ones the lowest token first, as tokens and as log probabilities.
 * targets and logprob are both given or both NULL, entropy may be NULL, and
 * with top = 0 the last two are not used; something has to be asked for.
 * A logit of -inf has probability 0 and adds nothing to the entropy; a row of
 * nothing else has logprobs of -inf and entropy 0.  A target outside
 * 0..vocab-1 gives 0.  Sums are F32; how many workgroups a row has follows from
 * rows and vocab, so that a row's last bits may be others in another batch.  The
 * same call gives the same bits.  A row that holds NaN or +inf gives unspecified
 * numbers and tokens within 0..vocab-1.
 * workspace: token_logprobs_workspace(rows, vocab, top) bytes (fewer is
 * QP_ERR_SCRATCH), not shared by calls that may overlap.
 * Refusals: rows or vocab 0, rows >= 2^24, rows * vocab >= 2^31: QP_ERR_SHAPE;
 * top above QP_LOGPROBS_MAX_TOP or vocab: QP_ERR_RANGE; unknown format:
 * QP_ERR_FORMAT.
 * ---------------------------------------------------------------------- */
enum qp_logits_format { QP_LOGITS_BF16 = 0, QP_LOGITS_F32 = 1 };
#define QP_LOGPROBS_MAX_TOP 32
uint64_t token_logprobs_workspace(uint32_t rows, uint32_t vocab, uint32_t top);
int token_logprobs(const void *logits, int logits_format, const int32_t *targets, float *logprob,
                   float *entropy, int32_t *top_ids, float *top_logprobs, void *workspace,
                   uint64_t workspace_bytes, uint32_t rows, uint32_t vocab, uint32_t top,
                   void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QPROJ_DECODER_H */
