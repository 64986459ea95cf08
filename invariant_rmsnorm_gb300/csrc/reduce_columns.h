// Second pass of two weight gradients at once: columns of two stacks of partial
// rows, summed in a fixed order.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rmsn {

// n partial rows and the row that their sum goes to (null: nothing to do).
struct PartialRows {
    const float* p;
    int64_t n;
    float* out;
};

cudaError_t launch_reduce_columns(const PartialRows& first, const PartialRows& second, int D, cudaStream_t s);

}  // namespace rmsn
