// Internal launch interface of LayerNorm between its C-ABI layer (layernorm.cu)
// and the translation units with its kernels. Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

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

// The backward's launch shape, by D alone: it decides the weight gradients' chunks.
constexpr int64_t kLnCtaRowFrom = 128;  // 16-byte vectors a row from which a CTA takes a row (D >= 1024)

constexpr int64_t kLnTeamsTo = 512;      // and up to which a CTA of several teams takes a row a team (D <= 4096)

struct LnShape {
    int64_t per_sm;  // CTAs an SM
    int64_t step;    // rows that a CTA takes at a time
};

inline LnShape ln_shape(int64_t D) {
    const int64_t NV = D / 8;
    if (NV < kLnCtaRowFrom) {
        // Groups of 256-thread CTAs, two an SM: two vectors a lane, or three where
        // that halves the lanes (or a warp is not enough for two), else four.
        auto lanes = [&](int64_t v) {
            int64_t G = 1;
            while (G * v < NV) G *= 2;
            return G;
        };
        int64_t G = NV == 1 ? 1 : lanes(2);
        if (NV > 8 && lanes(3) < G) G = lanes(3);
        return {2, 256 / std::min<int64_t>(G, 32)};
    }
    // Two vectors a thread. One CTA of 16 warps an SM, in teams of a row's warps; a row
    // of more warps is a CTA's alone, two an SM at 10 warps, else one.
    const int64_t warps = ((NV + 1) / 2 + 31) / 32;
    if (NV <= kLnTeamsTo) return {1, 16 / warps};
    return {NV <= 640 ? 20 / warps : 1, 1};
}

cudaError_t launch_ln_fwd(const LnFwdArgs& a, cudaStream_t s);
cudaError_t launch_ln_fwd_f16(const LnFwdArgs& a, cudaStream_t s);
cudaError_t launch_ln_bwd(const LnBwdArgs& a, unsigned chunks, bool bias, cudaStream_t s);
cudaError_t launch_ln_bwd_f16(const LnBwdArgs& a, unsigned chunks, bool bias, cudaStream_t s);
cudaError_t layernorm_read_error(unsigned* flags, bool clear);
cudaError_t layernorm_f16_read_error(unsigned* flags, bool clear);

}  // namespace rmsn
