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

/* 8-bit activation formats, each the operand of one GEMM of the library:
 *   QP_ACT_FP8_ROW      E4M3 [rows,k], F32 scale [rows]: fp8_gemm_rowscale;
 *   QP_ACT_FP8_BLOCK128 E4M3 [rows,k], F32 scale [rows, ceil(k/128)] (the last
 *                       block is shorter where 128 does not divide k):
 *                       fp8_gemm_blockscale;
 *   QP_ACT_INT8_BLOCK32 int8 [rows,k], F32 scale [rows, k/32]:
 *                       int8_gemm_blockscaled.
 * Rounding as in qproj.h: scale = amax/448 (127), one IEEE division of the
 * F32 value by the stored scale, round to nearest even, a zero scale encoded
 * as scale 0 with +0 codes. */
enum qp_act_format {
    QP_ACT_FP8_ROW = 0,
    QP_ACT_FP8_BLOCK128 = 1,
    QP_ACT_INT8_BLOCK32 = 2
};

/* Longest row of the two quantizing operators below. */
#define QP_LAYER_MAX_K (1u << 18)

/* ------------------------------------------------------------------------
 * Residual addition, RMS norm and 8-bit quantizer in one pass:
 *   h = bf16(x + residual)                       (written to residual_out)
 *   y = h * (1 / sqrt(mean(h^2) + eps)) * weight      in F32, never stored
 *   q, scale = y quantized per `fmt`.
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
 * Gated activation and 8-bit quantizer in one pass:
 *   y = silu(gate) * up,  silu(g) = g / (1 + exp(-g))      in F32
 *   q, scale = y quantized per `fmt`.
 *   gate_up [rows, 2k] BF16: a row's k gate values, then its k up values (the
 *   output of one product with the gate and up weights stacked);
 *   q [rows,k].  Sizes and errors as above, and rows * 2k < 2^31.
 * ---------------------------------------------------------------------- */
int silu_mul_quant(const uint16_t *gate_up, int fmt, void *q, float *scale,
                   uint32_t rows, uint32_t k, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QPROJ_LAYER_H */
