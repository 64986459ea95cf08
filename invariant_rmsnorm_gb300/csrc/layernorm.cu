// LayerNorm forward and backward: kernels and C-ABI entry points.
//
// Forward, per row: mu = sum x / D, then the variance from the deviations
// x - mu (a second pass over the row, so a large mean cancels nothing), then
// y = ((x - mu) r) w_eff + b. Backward, per row, with n = (x - mu) r:
// dx = r (g w_eff - mean(g w_eff) - n mean(g w_eff n)); the columns' sums
// dw = sum g n and db = sum g go in two passes as in reduce.cu.
#include <algorithm>

#include "checks.h"
#include "common.cuh"
#include "kernels.h"
#include "layernorm.h"
#include "reduce_columns.h"

namespace rmsn {
namespace {

struct LnFwdArgs {
    const uint16_t* x; int64_t ldx;
    const float* w;
    const float* b;  // null: no bias
    uint16_t* y; int64_t ldy;
    float* mean;
    float* rstd;
    int64_t T; int D; float eps; int zc;
};

struct LnBwdArgs {
    const uint16_t* g; int64_t ldg;
    const uint16_t* x; int64_t ldx;
    const float* w;
    const float* mean;
    const float* rstd;
    uint16_t* dx; int64_t lddx;
    float* partials;  // [chunks][D] of dw, then [chunks][D] of db if it is asked for
    int64_t T; int D; int zc; int chunk; int bias;
};

constexpr int kLnThreads = 256;

// Sum over the CTA, the same bits in every thread: warp butterflies, then the
// warps' totals in warp order.
__device__ float cta_sum(float v, float* red) {
    v = group_sum<32>(v);
    __syncthreads();  // red may still be read from the sum before
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = red[0];
    for (int i = 1; i < kLnThreads / 32; ++i) t = fadd(t, red[i]);
    return t;
}

__device__ __forceinline__ void load8(const float* p, float (&o)[8]) {
    const float4 lo = __ldg(reinterpret_cast<const float4*>(p));
    const float4 hi = __ldg(reinterpret_cast<const float4*>(p) + 1);
    o[0] = lo.x; o[1] = lo.y; o[2] = lo.z; o[3] = lo.w;
    o[4] = hi.x; o[5] = hi.y; o[6] = hi.z; o[7] = hi.w;
}

__device__ __forceinline__ void weights8(const float* w, int zc, int v, float (&o)[8]) {
    load8(w + 8 * v, o);
    if (zc)
        for (int e = 0; e < 8; ++e) o[e] = fadd(o[e], 1.0f);
}

// One CTA a row, the row read three times (the second and third from cache).
template <bool F16>
__global__ void __launch_bounds__(kLnThreads) ln_fwd_kernel(const LnFwdArgs a) {
    __shared__ float red[kLnThreads / 32];
    pdl_wait();
    const int NV = a.D >> 3;
    const float d = static_cast<float>(a.D);
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        const uint4* x = reinterpret_cast<const uint4*>(a.x + row * a.ldx);
        float f[8], s = 0.0f, ss = 0.0f;
        for (int v = threadIdx.x; v < NV; v += kLnThreads) {
            unpack_act<F16>(x[v], f);
            for (int e = 0; e < 8; ++e) s = fadd(s, f[e]);
        }
        const float mu = __fdiv_rn(cta_sum(s, red), d);
        for (int v = threadIdx.x; v < NV; v += kLnThreads) {
            unpack_act<F16>(x[v], f);
            for (int e = 0; e < 8; ++e) {
                const float c = fsub(f[e], mu);
                ss = fadd(ss, fmul(c, c));
            }
        }
        const float r = rsqrtf(fadd(__fdiv_rn(cta_sum(ss, red), d), a.eps));
        if (threadIdx.x == 0) {
            a.mean[row] = mu;
            a.rstd[row] = r;
        }
        uint4* y = reinterpret_cast<uint4*>(a.y + row * a.ldy);
        for (int v = threadIdx.x; v < NV; v += kLnThreads) {
            float w[8], b[8] = {};
            unpack_act<F16>(x[v], f);
            weights8(a.w, a.zc, v, w);
            if (a.b != nullptr) load8(a.b + 8 * v, b);
            for (int e = 0; e < 8; ++e) f[e] = fadd(fmul(fmul(fsub(f[e], mu), r), w[e]), b[e]);
            y[v] = pack_act<F16>(f);
        }
    }
    pdl_release();
}

// One CTA a chunk of rows. Thread t owns the columns of the vectors t, t + 256,
// ...: it adds their rows in ascending order in shared memory that no other
// thread touches.
template <bool F16>
__global__ void __launch_bounds__(kLnThreads) ln_bwd_kernel(const LnBwdArgs a) {
    extern __shared__ __align__(16) float acc[];  // [2][D]: dw, db
    __shared__ float red[kLnThreads / 32];
    const int NV = a.D >> 3;
    const float d = static_cast<float>(a.D);
    float* accw = acc;
    float* accb = acc + a.D;
    for (int v = threadIdx.x; v < NV; v += kLnThreads)
        for (int e = 0; e < 8; ++e) accw[8 * v + e] = accb[8 * v + e] = 0.0f;
    pdl_wait();
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
    const int64_t row1 = min(row0 + a.chunk, a.T);
    for (int64_t row = row0; row < row1; ++row) {
        const uint4* g = reinterpret_cast<const uint4*>(a.g + row * a.ldg);
        const uint4* x = reinterpret_cast<const uint4*>(a.x + row * a.ldx);
        const float mu = a.mean[row], r = a.rstd[row];
        float gf[8], f[8], w[8], s1 = 0.0f, s2 = 0.0f;
        for (int v = threadIdx.x; v < NV; v += kLnThreads) {
            unpack_act<F16>(g[v], gf);
            unpack_act<F16>(x[v], f);
            weights8(a.w, a.zc, v, w);
            for (int e = 0; e < 8; ++e) {
                const float n = fmul(fsub(f[e], mu), r), gw = fmul(gf[e], w[e]);
                s1 = fadd(s1, gw);
                s2 = fadd(s2, fmul(gw, n));
                accw[8 * v + e] = fadd(accw[8 * v + e], fmul(gf[e], n));
                accb[8 * v + e] = fadd(accb[8 * v + e], gf[e]);
            }
        }
        const float c1 = __fdiv_rn(cta_sum(s1, red), d), c2 = __fdiv_rn(cta_sum(s2, red), d);
        uint4* dx = reinterpret_cast<uint4*>(a.dx + row * a.lddx);
        for (int v = threadIdx.x; v < NV; v += kLnThreads) {
            unpack_act<F16>(g[v], gf);
            unpack_act<F16>(x[v], f);
            weights8(a.w, a.zc, v, w);
            for (int e = 0; e < 8; ++e) {
                const float n = fmul(fsub(f[e], mu), r), gw = fmul(gf[e], w[e]);
                f[e] = fmul(r, fsub(fsub(gw, c1), fmul(n, c2)));
            }
            dx[v] = pack_act<F16>(f);
        }
    }
    float* pw = a.partials + static_cast<int64_t>(blockIdx.x) * a.D;
    float* pb = pw + static_cast<int64_t>(gridDim.x) * a.D;
    for (int v = threadIdx.x; v < NV; v += kLnThreads)
        for (int e = 0; e < 8; ++e) {
            pw[8 * v + e] = accw[8 * v + e];
            if (a.bias) pb[8 * v + e] = accb[8 * v + e];
        }
    pdl_release();
}

// Rows of a weight-gradient chunk: a function of T and D alone.
constexpr int64_t kLnChunks = 304;
int64_t ln_chunk_rows(int64_t T, int64_t) { return std::max<int64_t>(1, (T + kLnChunks - 1) / kLnChunks); }
int64_t ln_chunks(int64_t T, int64_t D) {
    const int64_t c = ln_chunk_rows(T, D);
    return (T + c - 1) / c;
}

size_t ws_need(int64_t T, int64_t D) { return static_cast<size_t>(ln_chunks(T, D)) * static_cast<size_t>(D) * 8u; }

}  // namespace
}  // namespace rmsn

using namespace rmsn;

extern "C" {

int layernorm_fwd(const rmsn_act16* x, int64_t ldx, const float* w, const float* b, rmsn_act16* y, int64_t ldy,
                  float* mean, float* rstd, int64_t T, int64_t D, float eps, int zero_centered_gamma, int dtype,
                  rmsn_stream stream) {
    int flags = 0;
    RMSN_TRY(dtype_flags(dtype, &flags));
    RMSN_TRY(check_shape(T, D));
    if (T == 0) return RMSN_OK;
    RMSN_TRY(check_act(x, ldx, D));
    RMSN_TRY(check_act(y, ldy, D));
    RMSN_TRY(check_vec(w));
    if (b) RMSN_TRY(check_vec(b));
    RMSN_TRY(check_vec(mean));
    RMSN_TRY(check_vec(rstd));
    RMSN_TRY(check_eps(eps));
    LnFwdArgs a{x, ldx, w, b, y, ldy, mean, rstd, T, static_cast<int>(D), eps, zero_centered_gamma ? 1 : 0};
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(T, int64_t(sm_count()) * 8));
    return cuda_status(flags ? launch_kernel(ln_fwd_kernel<true>, grid, kLnThreads, 0, stream, a)
                             : launch_kernel(ln_fwd_kernel<false>, grid, kLnThreads, 0, stream, a));
}

size_t layernorm_bwd_workspace_bytes(int64_t T, int64_t D) {
    if (check_shape(T, D) != RMSN_OK || T == 0) return 0;
    return ws_need(T, D);
}

size_t layernorm_bwd_workspace_bytes_max(int64_t T_max, int64_t D) {
    if (check_shape(T_max, D) != RMSN_OK || T_max <= 0) return 0;
    return static_cast<size_t>(std::min<int64_t>(T_max, kLnChunks)) * static_cast<size_t>(D) * 8u;
}

int layernorm_bwd(const rmsn_act16* g, int64_t ldg, const rmsn_act16* x, int64_t ldx, const float* w,
                  const float* mean, const float* rstd, rmsn_act16* dx, int64_t lddx, float* dw, float* db, void* ws,
                  size_t ws_bytes, int64_t T, int64_t D, int zero_centered_gamma, int dtype, rmsn_stream stream) {
    int flags = 0;
    RMSN_TRY(dtype_flags(dtype, &flags));
    RMSN_TRY(check_shape(T, D));
    RMSN_TRY(check_vec(dw));
    if (db) RMSN_TRY(check_vec(db));
    if (T == 0) {  // the sums over no rows
        cudaError_t e = cudaMemsetAsync(dw, 0, static_cast<size_t>(D) * 4u, stream);
        if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, static_cast<size_t>(D) * 4u, stream);
        return cuda_status(e);
    }
    RMSN_TRY(check_act(g, ldg, D));
    RMSN_TRY(check_act(x, ldx, D));
    RMSN_TRY(check_act(dx, lddx, D));
    RMSN_TRY(check_vec(w));
    RMSN_TRY(check_vec(mean));
    RMSN_TRY(check_vec(rstd));
    if (ws == nullptr || ws_bytes < ws_need(T, D)) return RMSN_EWORKSPACE;
    if (!aligned16(ws)) return RMSN_EALIGN;
    const int64_t n = ln_chunks(T, D);
    LnBwdArgs a{g, ldg, x, ldx, w, mean, rstd, dx, lddx, static_cast<float*>(ws), T, static_cast<int>(D),
                zero_centered_gamma ? 1 : 0, static_cast<int>(ln_chunk_rows(T, D)), db != nullptr};
    const size_t smem = static_cast<size_t>(D) * 8u;
    const void* kern = flags ? reinterpret_cast<const void*>(ln_bwd_kernel<true>)
                             : reinterpret_cast<const void*>(ln_bwd_kernel<false>);
    if (ensure_smem_attr(kern, static_cast<int>(smem)) != cudaSuccess) return RMSN_ECUDA;
    cudaError_t e = flags ? launch_kernel(ln_bwd_kernel<true>, static_cast<unsigned>(n), kLnThreads, smem, stream, a)
                          : launch_kernel(ln_bwd_kernel<false>, static_cast<unsigned>(n), kLnThreads, smem, stream, a);
    if (e == cudaSuccess) e = launch_reduce_columns(a.partials, n, a.D, dw, db, stream);
    return cuda_status(e);
}

}  // extern "C"
