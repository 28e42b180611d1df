// capi_layer.hip -- the extern "C" boundary of the operators declared in
// include/qproj_layer.h.  As in capi.hip, every argument is checked on the
// host before anything is enqueued; nothing allocates or synchronises.
#include <cmath>

#include "capi_check.hpp"
#include "../../include/qproj_layer.h"

using namespace qp::capi;

namespace {

// fmt known, 1 <= k <= QP_LAYER_MAX_K in whole 16-byte chunks (int8: whole
// blocks), and rows * wide elements (the widest tensor) below 2^31.
int check_act(int fmt, uint32_t rows, uint32_t k, uint64_t wide)
{
    if (fmt != QP_ACT_FP8_ROW && fmt != QP_ACT_FP8_BLOCK128 && fmt != QP_ACT_INT8_BLOCK32 && fmt != QP_ACT_BF16)
        return QP_ERR_FORMAT;
    if (rows == 0 || k == 0 || k > QP_LAYER_MAX_K || k % (fmt == QP_ACT_INT8_BLOCK32 ? 32 : 16) != 0 ||
        !fits(rows, wide))
        return QP_ERR_SHAPE;
    return QP_OK;
}

bool blockscale_shape(uint32_t m, uint32_t n, uint32_t k)
{
    return m != 0 && n != 0 && k != 0 && k % 16 == 0 && fits(m, k) && fits(n, k) && fits(m, n);
}

} // namespace

extern "C" {

int rmsnorm_residual_quant(const uint16_t *x, const uint16_t *residual, const uint16_t *weight,
                           float eps, int fmt, void *q, float *scale, uint16_t *residual_out,
                           uint32_t rows, uint32_t k, void *stream)
{
    if (int e = check_ptrs({x, weight, q, fmt == QP_ACT_BF16 ? q : scale}))
        return e;
    if ((residual == nullptr) != (residual_out == nullptr))
        return QP_ERR_NULL;
    if (!aligned16(residual) || !aligned16(residual_out))
        return QP_ERR_ALIGN;
    if (int e = check_act(fmt, rows, k, k))
        return e;
    if (!(eps > 0.0f) || !std::isfinite(eps))
        return QP_ERR_RANGE;
    return done(qp::launch_rmsnorm_residual_quant(x, residual, weight, eps, fmt, q, scale,
                                                  residual_out, rows, k, S(stream)));
}

int silu_mul_quant(const uint16_t *gate_up, int fmt, void *q, float *scale, uint32_t rows,
                   uint32_t k, void *stream)
{
    if (int e = check_ptrs({gate_up, q, fmt == QP_ACT_BF16 ? q : scale}))
        return e;
    if (int e = check_act(fmt, rows, k, 2 * (uint64_t)k))
        return e;
    return done(qp::launch_silu_mul_quant(gate_up, fmt, q, scale, rows, k, S(stream)));
}

int fp8_gemm_blockscale(const uint8_t *a, const float *a_scale, const uint8_t *w,
                        const float *block_scale, uint16_t *out, uint32_t m, uint32_t n,
                        uint32_t k, void *stream)
{
    if (int e = check_ptrs({a, a_scale, w, block_scale, out}))
        return e;
    if (!blockscale_shape(m, n, k))
        return QP_ERR_SHAPE;
    return done(qp::launch_fp8_gemm_blockscale(a, a_scale, w, block_scale, out, m, n, k, S(stream)));
}

int fp8_gemm_blockscale_kernel(uint32_t m, uint32_t n, uint32_t k)
{
    return blockscale_shape(m, n, k) ? qp::fp8_gemm_blockscale_kernel(m, n, k) : QP_ERR_SHAPE;
}

uint64_t moe_fp8_blockscale_workspace(uint32_t t, uint32_t topk, uint32_t i)
{
    return qp::moe_fp8_workspace(t, topk, i);
}

int moe_fp8_blockscale(const uint16_t *x, const float *router_logits, const uint8_t *w13,
                       const float *s13, const uint8_t *w2, const float *s2, void *workspace,
                       uint64_t workspace_bytes, uint16_t *out, uint32_t t, uint32_t e,
                       uint32_t topk, uint32_t h, uint32_t i, int renormalize, void *stream)
{
    if (int err = check_ptrs({x, router_logits, w13, s13, w2, s2, workspace, out}))
        return err;
    if (t < 1 || t > QP_MOE_MAX_T || topk < 1 || topk > QP_MOE_MAX_TOPK || topk > e)
        return QP_ERR_RANGE;
    if (e > QP_MOE_MAX_E || h == 0 || i == 0 || h % 128 != 0 || i % 128 != 0 ||
        !fits(2 * (uint64_t)i, h) || !fits(2 * (uint64_t)t, h) || !fits(4 * (uint64_t)t * topk, i))
        return QP_ERR_SHAPE;
    if (workspace_bytes < qp::moe_fp8_workspace(t, topk, i))
        return QP_ERR_SCRATCH;
    return done(qp::launch_moe_fp8(x, router_logits, w13, s13, w2, s2, workspace, out, t, e, topk, h,
                                   i, renormalize != 0, S(stream)));
}

} // extern "C"
