// capi_check.hpp -- argument checks shared by the extern "C" entry points.
#pragma once

#include <initializer_list>

#include "qp_launch.hpp"
#include "../../include/qproj.h"

namespace qp {
namespace capi {

constexpr uint64_t MAX_ELEMS = (1ull << 31) - 1;   // every tensor < 2^31 elements

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int check_ptrs(std::initializer_list<const void *> ps)
{
    for (const void *p : ps)
        if (!p)
            return QP_ERR_NULL;
    for (const void *p : ps)
        if (!aligned16(p))
            return QP_ERR_ALIGN;
    return QP_OK;
}

inline bool fits(uint64_t rows, uint64_t cols) { return rows * cols <= MAX_ELEMS; }

inline int done(hipError_t e) { return e == hipSuccess ? QP_OK : QP_ERR_HIP; }

inline hipStream_t S(void *s) { return reinterpret_cast<hipStream_t>(s); }

} // namespace capi
} // namespace qp
