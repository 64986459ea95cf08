// Weight-gradient pass 2 of the operators with two weights (LayerNorm's w and b,
// the head norms of q and k).
//
// The chunk axis is cut into kRanges ranges of ceil(n / kRanges) chunks. Each is
// added in ascending order, then every kParts-th range's total, then the parts: a
// tree fixed by n alone, no atomics. A CTA owns 8 adjacent columns, a 32-byte
// sector of each partial row, of one of the two outputs (blockIdx.y); a thread
// adds 4 of them over one range.
//
// Bound by the latency of a range's loads, so the ranges are short. Of the counts
// that calls have (at most 304 up to 2^27 values) 128 ranges measured best or equal
// (whole backwards of LayerNorm; 128, 64, 32 and 16 ranges): 8192 x 1024, 147
// partial rows, 14.5, 14.8, 15.2 and 16.0 us; 4099 x 5000, 293 rows, 28.4, 28.3,
// 29.0 and 30.4; 262144 x 128, 304 rows, 36.4, 36.6, 37.2 and 39.2. Where there are
// fewer rows than ranges the last ranges are empty. The loads are streaming ones:
// LayerNorm's partial rows lie in L2 at high priority, and an ordinary load leaves
// them there in the way of what comes next (8192 x 16384 by 3 %).
#include "reduce_columns.h"

#include "common.cuh"
#include "kernels.h"

namespace rmsn {

namespace {
constexpr int kCols = 8, kQuads = kCols / 4;
constexpr int kRanges = 128;  // of the chunk axis
constexpr int kParts = 8;     // of the ranges, added side by side
}  // namespace

__global__ void __launch_bounds__(kRanges * kQuads)
reduce_columns_kernel(const PartialRows first, const PartialRows second, int D) {
    __shared__ float4 range[kRanges][kQuads];
    __shared__ float part[kParts][kCols];
    pdl_wait();
    const PartialRows& a = blockIdx.y ? second : first;
    const int q = threadIdx.x % kQuads, r = threadIdx.x / kQuads;
    const int64_t per = (a.n + kRanges - 1) / kRanges;
    const int64_t c0 = min(r * per, a.n), c1 = min(c0 + per, a.n);
    const float* p = a.p + c0 * D + blockIdx.x * kCols + 4 * q;  // D is a multiple of 8
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
    for (int64_t c = c0; c < c1; ++c, p += D) {
        const float4 u = __ldcs(reinterpret_cast<const float4*>(p));
        v = make_float4(fadd(v.x, u.x), fadd(v.y, u.y), fadd(v.z, u.z), fadd(v.w, u.w));
    }
    pdl_release();
    range[r][q] = v;
    __syncthreads();
    const int col = threadIdx.x % kCols, s = threadIdx.x / kCols;
    if (s < kParts) {
        const float* t = reinterpret_cast<const float*>(range) + col;
        float sum = t[s * kCols];
#pragma unroll
        for (int i = s + kParts; i < kRanges; i += kParts) sum = fadd(sum, t[i * kCols]);
        part[s][col] = sum;
    }
    __syncthreads();
    if (s == 0) {
        float sum = part[0][col];
#pragma unroll
        for (int i = 1; i < kParts; ++i) sum = fadd(sum, part[i][col]);
        a.out[blockIdx.x * kCols + col] = sum;
    }
}

cudaError_t launch_reduce_columns(const PartialRows& first, const PartialRows& second, int D, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(D / kCols), second.out != nullptr ? 2u : 1u);
    cfg.blockDim = dim3(kRanges * kQuads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = RMSN_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, reduce_columns_kernel, first, second, D);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rmsn
