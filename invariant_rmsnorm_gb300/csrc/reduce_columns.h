// Second pass of two weight gradients at once: columns of two stacks of partial
// rows, summed in a fixed order.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rmsn {

// out0[j] = sum over c of partials[c][j], and out1[j] (unless null) the same over
// the n rows of D values that follow the first n.
cudaError_t launch_reduce_columns(const float* partials, int64_t n, int D, float* out0, float* out1,
                                  cudaStream_t s);

}  // namespace rmsn
