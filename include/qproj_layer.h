/*
 * qproj_layer.h -- the operators around the projections of qproj.h, in the
 * same library (libqproj.so): the norm and the activation that feed a
 * quantized product, the block-scaled FP8 product itself, and a whole
 * mixture-of-experts layer for decode.
 *
 * The conventions of qproj.h hold: device pointers to dense row-major memory,
 * BF16 as uint16_t bits, E4M3 as uint8_t, 16-byte alignment, caller-owned
 * buffers and scratch, no allocation, no synchronisation, work enqueued on
 * `stream`, host-side checks that return a QP_ERR_* code and enqueue nothing.
 * Inputs holding NaN or Inf give unspecified (but in-bounds) results, except
 * where an operator names them.
 */
#ifndef QPROJ_LAYER_H
#define QPROJ_LAYER_H

#include "qproj.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activation formats, each the operand of products of the library:
 *   QP_ACT_FP8_ROW      E4M3 [rows,k], F32 scale [rows]: fp8_gemm_rowscale;
 *   QP_ACT_FP8_BLOCK128 E4M3 [rows,k], F32 scale [rows, ceil(k/128)] (the last
 *                       block is shorter where 128 does not divide k):
 *                       fp8_gemm_blockscale;
 *   QP_ACT_INT8_BLOCK32 int8 [rows,k], F32 scale [rows, k/32]:
 *                       int8_gemm_blockscaled;
 *   QP_ACT_BF16         BF16 [rows,k], no scale (the pointer is not used and
 *                       may be NULL): the GEMVs, moe_fp8_blockscale.
 * Rounding as in qproj.h: scale = amax/448 (127), one IEEE division of the
 * F32 value by the stored scale, round to nearest even, a zero scale encoded
 * as scale 0 with +0 codes; BF16 rounded to nearest even. */
enum qp_act_format {
    QP_ACT_FP8_ROW = 0,
    QP_ACT_FP8_BLOCK128 = 1,
    QP_ACT_INT8_BLOCK32 = 2,
    QP_ACT_BF16 = 16
};

/* Longest row of the two operators below. */
#define QP_LAYER_MAX_K (1u << 18)

/* ------------------------------------------------------------------------
 * Residual addition, RMS norm and quantizer in one pass:
 *   h = bf16(x + residual)                       (written to residual_out)
 *   y = h * (1 / sqrt(mean(h^2) + eps)) * weight      in F32, never stored
 *   q, scale = y in the form `fmt`.
 *   x [rows,k], residual [rows,k] and weight [k] BF16; q [rows,k];
 *   residual_out [rows,k] BF16.
 * residual and residual_out are both given or both NULL (then h = x);
 * residual_out may be residual itself (the residual stream updated in place)
 * and must not overlap anything else.  The norm reads the residual as it is
 * kept, so the result equals the three steps run apart.  Sums are F32; a
 * row's outputs depend on that row alone, bit for bit, whatever `rows` is.
 * 1 <= rows, 1 <= k <= QP_LAYER_MAX_K, k % 16 == 0 (% 32 for int8), else
 * QP_ERR_SHAPE; eps positive and finite, else QP_ERR_RANGE; an unknown fmt is
 * QP_ERR_FORMAT; one of the residual pointers alone is QP_ERR_NULL.
 * ---------------------------------------------------------------------- */
int rmsnorm_residual_quant(const uint16_t *x, const uint16_t *residual,
                           const uint16_t *weight, float eps, int fmt, void *q,
                           float *scale, uint16_t *residual_out, uint32_t rows,
                           uint32_t k, void *stream);

/* ------------------------------------------------------------------------
 * Gated activation and quantizer in one pass:
 *   y = silu(gate) * up,  silu(g) = g / (1 + exp(-g))      in F32 (so silu is
 *   0 where exp(-g) passes F32's range, for gates below -88.7)
 *   q, scale = y in the form `fmt`.
 *   gate_up [rows, 2k] BF16: a row's k gate values, then its k up values (the
 *   output of one product with the gate and up weights stacked);
 *   q [rows,k].  Sizes and errors as above, and rows * 2k < 2^31.
 * ---------------------------------------------------------------------- */
int silu_mul_quant(const uint16_t *gate_up, int fmt, void *q, float *scale,
                   uint32_t rows, uint32_t k, void *stream);

/* ------------------------------------------------------------------------
 * Block-scaled FP8 GEMM, the product of a QP_ACT_FP8_BLOCK128 operand and a
 * block-scaled weight (the weight of fp8_gemv_blockscale, without a requant):
 *   C[i,j] = bf16( sum_b a_scale[i,b] * block_scale[j/128,b] * P_b[i,j] ),
 *   P_b[i,j] = sum of e4m3(a[i,t]) * e4m3(w[j,t]) over the K block b.
 *   a [m,k] E4M3, a_scale [m, ceil(k/128)] F32, w [n,k] E4M3,
 *   block_scale [ceil(n/128), ceil(k/128)] F32 (the last blocks are smaller
 *   where 128 does not divide n or k), out [m,n] BF16.  Requires k % 16 == 0;
 *   any m and n (else QP_ERR_SHAPE).
 * Each P_b is formed by FP8 MFMAs (which keep 13 bits below the largest of 8
 * neighbouring products and add the groups of 8 in F32), the scaled blocks are
 * added in F32, and BF16 rounding happens once.  Any m is served, from one row on.  The order in
 * which the blocks are added follows m, n and k, so a row's last bits may differ
 * between batch sizes.  A NaN in a row of A or W (or in a scale) stays in the
 * outputs of that row (of the rows that the scale is for).
 * ---------------------------------------------------------------------- */
int fp8_gemm_blockscale(const uint8_t *a, const float *a_scale, const uint8_t *w,
                        const float *block_scale, uint16_t *out, uint32_t m,
                        uint32_t n, uint32_t k, void *stream);

/* The kernel that fp8_gemm_blockscale runs for a shape on the current device
 * (256 compute units where there is none): one of the values below, or
 * QP_ERR_SHAPE.  QP_BLOCKSCALE_KSPLIT is a base, to which are added the rows
 * of A in 16s and, times 8, the rows of W in 16s that a workgroup takes, and 64
 * where W is read past the caches.  Informative: for tests and profiles. */
enum qp_blockscale_kernel {
    QP_BLOCKSCALE_TILES_128 = 1,          /* 128 x 128 tiles                       */
    QP_BLOCKSCALE_TILES_256 = 2,          /* 256 x 256 tiles                       */
    QP_BLOCKSCALE_TILES_256_QUARTERS = 3, /* the same, the last as 128 x 128 ones  */
    QP_BLOCKSCALE_KSPLIT = 256            /* small tiles, K split over the waves   */
};
int fp8_gemm_blockscale_kernel(uint32_t m, uint32_t n, uint32_t k);

/* ------------------------------------------------------------------------
 * A mixture-of-experts layer for the few tokens of a decode or verify step,
 * in two launches.
 *   x [t,h] BF16; router_logits [t,e] F32;
 *   w13 [e, 2i, h] E4M3: each expert's i gate rows, then its i up rows;
 *   s13 [e, 2i/128, h/128] F32, one scale per 128 x 128 block;
 *   w2 [e, h, i] E4M3, s2 [e, h/128, i/128] F32; out [t,h] BF16.
 *   p = softmax(logits of the token); its topk largest are kept (of equal
 *   logits the lowest expert) and, with renormalize, divided by their sum;
 *   out = bf16( sum over them of p_e * W2_e (silu(W1_e x) * (W3_e x)) ).
 * An expert whose logit is -inf is never chosen; a token with fewer than
 * topk others takes those, one with none gets a row of zeros.  Sums are F32
 * in a fixed order (no atomics); between the two launches an activation is
 * held to 2^-17 of itself.  Which tokens share a batch may change the order
 * of a token's sum.  Only the chosen experts' weights are read, w13 once for
 * every four (where t*topk >= 3*e, eight) tokens of an expert and w2 once for
 * every two (four).
 * 1 <= t <= QP_MOE_MAX_T, 1 <= topk <= min(e, QP_MOE_MAX_TOPK) (else
 * QP_ERR_RANGE); e <= QP_MOE_MAX_E, h and i multiples of 128, 2*i*h < 2^31
 * (the limit is per expert: all of them together may be larger) and
 * 4*t*topk*i < 2^31, else QP_ERR_SHAPE.  workspace: caller-owned scratch of
 * moe_fp8_blockscale_workspace(t, topk, i) <= 4*t*topk*i + 65536 bytes (fewer
 * is QP_ERR_SCRATCH), its contents before and after the call unspecified.
 * ---------------------------------------------------------------------- */
#define QP_MOE_MAX_T 16
#define QP_MOE_MAX_TOPK 16
#define QP_MOE_MAX_E 512
uint64_t moe_fp8_blockscale_workspace(uint32_t t, uint32_t topk, uint32_t i);
int moe_fp8_blockscale(const uint16_t *x, const float *router_logits,
                       const uint8_t *w13, const float *s13, const uint8_t *w2,
                       const float *s2, void *workspace, uint64_t workspace_bytes,
                       uint16_t *out, uint32_t t, uint32_t e, uint32_t topk,
                       uint32_t h, uint32_t i, int renormalize, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QPROJ_LAYER_H */
