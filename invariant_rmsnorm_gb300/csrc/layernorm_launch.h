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
    float rcp_d;  // 1/D rounded to fp32
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
    float rcp_d;
};

// Launch shapes of the backward, by D: vectors a lane or thread, ...
// (group kernels: rows a turn, turns in flight, CTAs an SM)
#ifndef LN_B1
#define LN_B1 1, 2, 3, 3
#endif
#ifndef LN_B1_CTAS
#define LN_B1_CTAS 3
#endif
#ifndef LN_B2
#define LN_B2 2, 1, 3, 2
#endif
#ifndef LN_B2_CTAS
#define LN_B2_CTAS 2
#endif
// (CTA kernels: threads at most, CTAs an SM for the register bound, rows an iteration; warps an SM)
#ifndef LN_BW1
#define LN_BW1 1, 256, 3, 2
#endif
#ifndef LN_BW1_WARPS
#define LN_BW1_WARPS 24
#endif
#ifndef LN_BW2
#define LN_BW2 2, 256, 2, 1
#endif
#ifndef LN_BW2_WARPS
#define LN_BW2_WARPS 16
#endif
#ifndef LN_BW2_VPT
#define LN_BW2_VPT 2
#endif
#ifndef LN_BW4
#define LN_BW4 2, 512, 1, 1
#endif
#ifndef LN_BW4_WARPS
#define LN_BW4_WARPS 16
#endif
#ifndef LN_BW4_VPT
#define LN_BW4_VPT 2
#endif
#ifndef LN_BW_RING
#define LN_BW_RING 144  // KB an SM
#endif

struct LnShape {
    int64_t per_sm;  // CTAs an SM
    int64_t step;    // rows that a CTA takes at a time
};

inline LnShape ln_shape(int64_t D) {
    const int64_t NV = D / 8;
    if (NV <= 64) {  // a group of lanes a row
        int64_t G = 1;
        while (G < 32 && G < NV) G *= 2;
        return {NV <= 32 ? LN_B1_CTAS : LN_B2_CTAS, 256 / G};
    }
    auto ctas = [&](int64_t vpt, int64_t warps) { return warps / (((NV + vpt - 1) / vpt + 31) / 32); };
    if (NV <= 256) return {ctas(1, LN_BW1_WARPS), 1};
    if (NV <= 512) return {ctas(LN_BW2_VPT, LN_BW2_WARPS), 1};
    if (NV <= 1024) return {ctas(LN_BW4_VPT, LN_BW4_WARPS), 1};
    return {1, 1};
}

cudaError_t launch_ln_fwd(const LnFwdArgs& a, cudaStream_t s);
cudaError_t launch_ln_fwd_f16(const LnFwdArgs& a, cudaStream_t s);
cudaError_t launch_ln_bwd(const LnBwdArgs& a, unsigned chunks, bool bias, cudaStream_t s);
cudaError_t launch_ln_bwd_f16(const LnBwdArgs& a, unsigned chunks, bool bias, cudaStream_t s);
cudaError_t layernorm_read_error(unsigned* flags, bool clear);
cudaError_t layernorm_f16_read_error(unsigned* flags, bool clear);

}  // namespace rmsn
