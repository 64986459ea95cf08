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
    float* partials;     // norm backward: a row of D a CTA, dwq's, then dwk's
    const double* inv_freq;
    const void* pos;     // null: the token's index
    const uint8_t* axis; // several axes: that of every pair (null: one position a token)
    int axes;
    int64_t pos_axis, pos_token;  // strides of pos [axes][T], several axes alone
    int64_t T;
    int H[2];
    int D, R, layout, pos64, back, zc;
    float scale, eps;
    int ctas_q;          // norm backward: CTAs whose turns are q's
    float rcp_d;         // 1/D rounded to fp32
    bool dense[3][2];    // [in | x | out]: a token's heads lie side by side and are copied whole
    uint32_t row_bytes[2];  // of a head's row to copy: all of it, or in place what is turned
};

constexpr int kRopeThreads = 256;
// Turns of several tokens from one for every warp of a CTA an SM on, of a GPU of
// 152: the order of the weight gradients' sums is the same on every GPU.
constexpr int64_t kRopeManyFrom = 152 * (kRopeThreads / 32);

// log2 of the lanes a head: the smallest power of two that holds its units of two
// times eight values. Where R is no multiple of 16 the halves' last unit is cut
// short, and the rest of a head that is normalised has units of its own, of whole
// vectors counted from the row's end: what they leave is taken two values a lane,
// or needs twice the lanes. A function of D, R and the layout alone, so a row's
// reduction tree is too.
inline int rope_lanes_log2(int D, int R, bool any_halves, bool norm) {
    const int units = (D / 8 + 1) / 2;
    int lg = 2;
    while ((1 << lg) < units) ++lg;
    if (any_halves && norm) {
        const int vectors = std::min((D - R) / 8, 2 * ((1 << lg) - (R / 2 + 7) / 8));
        if (D - R - 8 * vectors > 2 << lg) ++lg;
    }
    return lg;
}

// CTAs of the norm backward, each with a partial row of dwq or of dwk: two an SM
// of a GPU of 152, fewer where there are few heads. A function of T, Hq, Hk
// and D alone.
inline int64_t rope_bwd_ctas(int64_t T, int64_t Hq, int64_t Hk, int64_t D) {
    const int64_t values = T * (Hq + Hk) * D;  // of a warp's turn: about 1024
    return std::max<int64_t>(Hk > 0 ? 2 : 1, std::min<int64_t>(304, (values + 8191) / 8192));
}

// The kernels by mode and format, each in a translation unit of its own.
cudaError_t launch_rope_turn(const RopeArgs& a, int* ctas_q, cudaStream_t s);
cudaError_t launch_rope_norm(const RopeArgs& a, int* ctas_q, cudaStream_t s);
cudaError_t launch_rope_norm_bwd(const RopeArgs& a, int* ctas_q, cudaStream_t s);
cudaError_t launch_rope_turn_f16(const RopeArgs& a, int* ctas_q, cudaStream_t s);
cudaError_t launch_rope_norm_f16(const RopeArgs& a, int* ctas_q, cudaStream_t s);
cudaError_t launch_rope_norm_bwd_f16(const RopeArgs& a, int* ctas_q, cudaStream_t s);
// The same with positions of several axes.
cudaError_t launch_rope_axes_turn(const RopeArgs& a, int* ctas_q, cudaStream_t s);
cudaError_t launch_rope_axes_norm(const RopeArgs& a, int* ctas_q, cudaStream_t s);
cudaError_t launch_rope_axes_norm_bwd(const RopeArgs& a, int* ctas_q, cudaStream_t s);
cudaError_t launch_rope_axes_turn_f16(const RopeArgs& a, int* ctas_q, cudaStream_t s);
cudaError_t launch_rope_axes_norm_f16(const RopeArgs& a, int* ctas_q, cudaStream_t s);
cudaError_t launch_rope_axes_norm_bwd_f16(const RopeArgs& a, int* ctas_q, cudaStream_t s);
cudaError_t rope_axes_turn_read_error(unsigned* flags, bool clear);
cudaError_t rope_axes_norm_read_error(unsigned* flags, bool clear);
cudaError_t rope_axes_norm_bwd_read_error(unsigned* flags, bool clear);
cudaError_t rope_axes_turn_f16_read_error(unsigned* flags, bool clear);
cudaError_t rope_axes_norm_f16_read_error(unsigned* flags, bool clear);
cudaError_t rope_axes_norm_bwd_f16_read_error(unsigned* flags, bool clear);
cudaError_t rope_turn_read_error(unsigned* flags, bool clear);
cudaError_t rope_norm_read_error(unsigned* flags, bool clear);
cudaError_t rope_norm_bwd_read_error(unsigned* flags, bool clear);
cudaError_t rope_turn_f16_read_error(unsigned* flags, bool clear);
cudaError_t rope_norm_f16_read_error(unsigned* flags, bool clear);
cudaError_t rope_norm_bwd_f16_read_error(unsigned* flags, bool clear);

}  // namespace rmsn
