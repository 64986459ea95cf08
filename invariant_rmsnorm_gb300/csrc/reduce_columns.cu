// Weight-gradient pass 2 of the operators with two weights (LayerNorm's w and b,
// the head norms of q and k).
//
// The chunk axis is cut into kReduceWarps ranges of ceil(n / kReduceWarps)
// chunks; each range is added in ascending order and the ranges' totals in
// range order: a tree fixed by n alone, no atomics. A CTA owns 8 adjacent
// columns of one of the two outputs (blockIdx.y); thread (range w, column k).
#include "reduce_columns.h"

#include "common.cuh"

namespace rmsn {

namespace {
constexpr int kCols = 8;     // columns of a CTA: one 32-byte sector of each partial row
constexpr int kUnroll = 16;  // loads in flight a thread
}

__global__ void __launch_bounds__(kReduceWarps * kCols)
reduce_columns_kernel(const float* __restrict__ partials, int64_t n, int D, float* __restrict__ out0,
                      float* __restrict__ out1) {
    __shared__ float tot[kReduceWarps][kCols];
    pdl_wait();
    const int k = threadIdx.x % kCols, w = threadIdx.x / kCols;
    const int col = blockIdx.x * kCols + k;  // D is a multiple of 8
    const int64_t per = (n + kReduceWarps - 1) / kReduceWarps;
    const int64_t c0 = w * per, c1 = min(c0 + per, n);
    const float* p = partials + (static_cast<int64_t>(blockIdx.y) * n) * D + col;
    float acc = 0.0f;
    for (int64_t c = c0; c < c1; c += kUnroll) {  // all of a batch in flight, a place without a chunk adds zero
        float v[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) v[i] = c + i < c1 ? __ldcg(p + (c + i) * D) : 0.0f;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) acc = fadd(acc, v[i]);
    }
    pdl_release();
    tot[w][k] = acc;
    __syncthreads();
    if (w == 0) {
        float s = tot[0][k];
#pragma unroll
        for (int r = 1; r < kReduceWarps; ++r) s = fadd(s, tot[r][k]);
        (blockIdx.y == 0 ? out0 : out1)[col] = s;
    }
}

cudaError_t launch_reduce_columns(const float* partials, int64_t n, int D, float* out0, float* out1,
                                  cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(D / kCols), out1 != nullptr ? 2u : 1u);
    cfg.blockDim = dim3(kReduceWarps * kCols);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = RMSN_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, reduce_columns_kernel, partials, n, D, out0, out1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rmsn
