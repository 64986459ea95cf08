// Internal launch interface of the rotary kernels between their C-ABI layer
// (rope.cu) and the translation units with the kernels. Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "rope.h"

namespace rmsn {

constexpr int kMaxHeadD = 512;

enum RopeMode : int { kTurn = 0, kNormTurn = 1, kNormTurnBwd = 2 };

// A [T][H][D] tensor by its strides in elements.
struct HeadsIn { const uint16_t* p; int64_t token, head; };
struct HeadsOut { uint16_t* p; int64_t token, head; };

struct RopeArgs {
    HeadsIn in[2];       // q, k (forward) / gq, gk (backward)
    HeadsIn x[2];        // q, k of the forward (norm backward)
    HeadsOut out[2];
    const float* w[2];   // norm weights
    float* rstd[2];      // written by the forward, read by the backward
    float* partials;     // norm backward: [chunks][D] of dwq, then of dwk
    const double* inv_freq;
    const void* pos;     // null: the token's index
    int64_t T;
    int H[2];
    int D, R, layout, pos64, back, zc;
    float scale, eps;
    float rcp_d;         // 1/D rounded to fp32
};

// How heads lie in warps: G lanes a head, NU units of two 16-byte vectors a
// lane. A function of D alone, so a row's reduction tree is too (with R and the
// layout, which say which vectors make a unit).
struct RopeShape { int lgG, NU; };

inline RopeShape rope_shape(int D, bool bwd) {
    const int U = (D / 8 + 1) / 2;
    int lg = 0;
    while ((1 << lg) < U) ++lg;
    RopeShape s{lg, 1};
    if (!bwd) {  // more values a lane where that leaves no more lanes idle
        for (int nu = 2; nu <= 3; ++nu) {
            int l = 0;
            while ((nu << l) < U) ++l;
            if (U > 2 && (nu << l) <= (s.NU << s.lgG)) s = {l, nu};
        }
    }
    return s;
}

// Warps' turns of a token: 32 / G heads a turn.
inline int64_t rope_turns_of(int64_t H, const RopeShape& s) { return (H + (32 >> s.lgG) - 1) / (32 >> s.lgG); }

constexpr int kRopeThreads = 256;

// CTAs of the norm backward, each with one partial row of dwq and of dwk: two an
// SM of a GPU of 152, fewer where there are fewer turns of warps. A function of
// T, Hq, Hk and D alone.
inline int64_t rope_bwd_ctas(int64_t T, int64_t Hq, int64_t Hk, int64_t D) {
    const RopeShape s = rope_shape(static_cast<int>(D), true);
    const int64_t turns = T * std::max(rope_turns_of(Hq, s), rope_turns_of(Hk, s));
    return std::max<int64_t>(1, std::min<int64_t>(304, (turns + kRopeThreads / 32 - 1) / (kRopeThreads / 32)));
}

cudaError_t launch_rope(RopeMode mode, const RopeArgs& a, cudaStream_t s);
cudaError_t launch_rope_f16(RopeMode mode, const RopeArgs& a, cudaStream_t s);

}  // namespace rmsn
