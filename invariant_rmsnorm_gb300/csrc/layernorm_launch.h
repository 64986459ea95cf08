// Internal launch interface of LayerNorm between its C-ABI layer (layernorm.cu)
// and the translation units with its kernels. Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rmsn {

struct LnFwdArgs {
    const uint16_t* x; int64_t ldx;
    const float* w;
    const float* b;  // null: no bias
    uint16_t* y; int64_t ldy;
    float* mean;
    float* rstd;
    int64_t T; int D; float eps; int zc;
    float inv_d_pow2;  // 1/D if D is a power of two, else 0
};

struct LnBwdArgs {
    const uint16_t* g; int64_t ldg;
    const uint16_t* x; int64_t ldx;
    const float* w;
    const float* mean;
    const float* rstd;
    uint16_t* dx; int64_t lddx;
    float* partials;  // [chunks][D] of dw, then [chunks][D] of db if it is asked for
    int64_t T; int D; int zc;
    int chunk;         // rows of a partial row: a CTA's
    float inv_d_pow2;
};

cudaError_t launch_ln_fwd(const LnFwdArgs& a, cudaStream_t s);
cudaError_t launch_ln_fwd_f16(const LnFwdArgs& a, cudaStream_t s);
cudaError_t launch_ln_bwd(const LnBwdArgs& a, unsigned chunks, bool bias, cudaStream_t s);
cudaError_t launch_ln_bwd_f16(const LnBwdArgs& a, unsigned chunks, bool bias, cudaStream_t s);
cudaError_t layernorm_read_error(unsigned* flags, bool clear);
cudaError_t layernorm_f16_read_error(unsigned* flags, bool clear);

}  // namespace rmsn
