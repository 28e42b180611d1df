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
    if (fmt != QP_ACT_FP8_ROW && fmt != QP_ACT_FP8_BLOCK128 && fmt != QP_ACT_INT8_BLOCK32)
        return QP_ERR_FORMAT;
    if (rows == 0 || k == 0 || k > QP_LAYER_MAX_K || k % (fmt == QP_ACT_INT8_BLOCK32 ? 32 : 16) != 0 ||
        !fits(rows, wide))
        return QP_ERR_SHAPE;
    return QP_OK;
}

} // namespace

extern "C" {

int rmsnorm_residual_quant(const uint16_t *x, const uint16_t *residual, const uint16_t *weight,
                           float eps, int fmt, void *q, float *scale, uint16_t *residual_out,
                           uint32_t rows, uint32_t k, void *stream)
{
    if (int e = check_ptrs({x, weight, q, scale}))
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
    if (int e = check_ptrs({gate_up, q, scale}))
        return e;
    if (int e = check_act(fmt, rows, k, 2 * (uint64_t)k))
        return e;
    return done(qp::launch_silu_mul_quant(gate_up, fmt, q, scale, rows, k, S(stream)));
}

} // extern "C"
