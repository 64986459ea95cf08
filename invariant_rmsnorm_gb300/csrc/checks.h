// Argument checks shared by the C-ABI layers. All run on the host, before any
// launch, and return a status of rmsnorm.h.
#pragma once

#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace rmsn {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int check_shape(int64_t T, int64_t D) {
    if (T < 0 || T >= (int64_t(1) << 31)) return RMSN_EINVAL;
    if (D < 8 || D > kMaxD || (D % 8) != 0) return RMSN_EUNSUPPORTED;
    return RMSN_OK;
}

// An activation matrix [T][ld] of 16-bit values (required = must be non-null).
inline int check_act(const void* p, int64_t ld, int64_t D) {
    if (p == nullptr) return RMSN_EINVAL;
    if (ld < D || ld > (int64_t(1) << 40)) return RMSN_EINVAL;
    if (!aligned16(p) || (ld % 8) != 0) return RMSN_EALIGN;
    return RMSN_OK;
}

inline int check_vec(const void* p) {
    if (p == nullptr) return RMSN_EINVAL;
    if (!aligned16(p)) return RMSN_EALIGN;
    return RMSN_OK;
}

inline int check_eps(float eps) { return (std::isfinite(eps) && eps >= 0.0f) ? RMSN_OK : RMSN_EINVAL; }

#define RMSN_TRY(expr)                  \
    do {                                \
        const int _st = (expr);         \
        if (_st != RMSN_OK) return _st; \
    } while (0)

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? RMSN_OK : RMSN_ECUDA; }

// Variant flags of an activation dtype argument (RMSN_EINVAL if unknown).
inline int dtype_flags(int dtype, int* flags) {
    if (dtype == RMSN_DTYPE_BF16) { *flags = 0; return RMSN_OK; }
    if (dtype == RMSN_DTYPE_F16) { *flags = kFlagF16; return RMSN_OK; }
    return RMSN_EINVAL;
}

}  // namespace rmsn
