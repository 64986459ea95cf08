// Weight-gradient pass 2 of the operators with two weights (LayerNorm's w and b,
// the head norms of q and k).
//
// The chunk axis is cut into kReduceWarps ranges of ceil(n / kReduceWarps)
// chunks; each range is added in ascending order and the ranges' totals in
// range order: a tree fixed by n alone, no atomics. A CTA owns 8 adjacent columns,
// a 32-byte sector of each partial row, of one of the two outputs (blockIdx.y);
// thread (range w, column k).
// Few columns (FEW): bound by latency, so a thread's loads are all in flight, 16
// at a time (2.9 us at 128 columns of 304 chunks; loads in turn 3.9). Many: by
// the loads' rate, and 16 registers of loads a thread measured slower (LayerNorm
// backward of 8192 x 16384 131 us; with them, or with 32 columns a CTA, 142). There
// the loads are streaming ones: such partial rows lie in L2 at high priority, and
// an ordinary load leaves them there in the way of what comes next (145 us).
#include "reduce_columns.h"

#include "common.cuh"
#include "kernels.h"

namespace rmsn {

namespace {
constexpr int kCols = 8;
constexpr int kUnroll = 16;  // FEW: loads in flight a thread
}

template <bool FEW>
__global__ void __launch_bounds__(kReduceWarps * kCols)
reduce_columns_kernel(const PartialRows first, const PartialRows second, int D) {
    __shared__ float tot[kReduceWarps][kCols];
    pdl_wait();
    const PartialRows& a = blockIdx.y ? second : first;
    const int k = threadIdx.x % kCols, w = threadIdx.x / kCols;
    const int col = blockIdx.x * kCols + k;  // D is a multiple of 8
    const int64_t per = (a.n + kReduceWarps - 1) / kReduceWarps;
    const int64_t c0 = w * per, c1 = min(c0 + per, a.n);
    const float* p = a.p + col;
    float acc = 0.0f;
    if constexpr (FEW) {
        for (int64_t c = c0; c < c1; c += kUnroll) {  // a place without a chunk adds zero
            float v[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) v[i] = c + i < c1 ? __ldcg(p + (c + i) * D) : 0.0f;
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) acc = fadd(acc, v[i]);
        }
    } else {
#pragma unroll 4
        for (int64_t c = c0; c < c1; ++c) acc = fadd(acc, __ldcs(p + c * D));
    }
    pdl_release();
    tot[w][k] = acc;
    __syncthreads();
    if (w == 0) {
        float s = tot[0][k];
#pragma unroll
        for (int r = 1; r < kReduceWarps; ++r) s = fadd(s, tot[r][k]);
        a.out[col] = s;
    }
}

cudaError_t launch_reduce_columns(const PartialRows& first, const PartialRows& second, int D, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(D / kCols), second.out != nullptr ? 2u : 1u);
    cfg.blockDim = dim3(kReduceWarps * kCols);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = RMSN_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool few = static_cast<int>(cfg.gridDim.x * cfg.gridDim.y) <= 2 * sm_count();
    const cudaError_t e = few ? cudaLaunchKernelEx(&cfg, reduce_columns_kernel<true>, first, second, D)
                              : cudaLaunchKernelEx(&cfg, reduce_columns_kernel<false>, first, second, D);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rmsn
