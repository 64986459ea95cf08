// LayerNorm kernels and their launchers, included by the translation units that
// instantiate them (layernorm.cu: bf16 activations; layernorm_f16.cu: fp16).
//
// Mathematics, per row: mu = sum x / D; var = sum (x - mu)^2 / D, from the
// deviations themselves, so a mean far from zero cancels nothing;
// y = ((x - mu) r) w + b. Backward, with c = x - mu and gw = g w:
//   dx = r gw - r c1 - c (r^2 c2'),  c1 = sum gw / D,  c2' = r sum(gw c) / D
// (n = c r is never formed there), dw = sum_t g (c r), db = sum_t g.
//
// All kernels are bound by HBM: 4 D bytes a row forward, 6 D backward. Two forms:
//   * Rows of up to 512 (backward) or 2048 values (forward): a group of G lanes,
//     at most a warp, holds a row in registers, straight from global loads, with
//     several rows a group in flight; no barrier, no shared memory. G and the
//     vectors a lane follow from D alone.
//   * Wider rows: a CTA a row. Rows come through a ring of bulk (TMA) copies to
//     shared memory; thread t owns the 16-byte vectors t, t + NT, ...; a row's
//     sums go by warp butterflies and one barrier, warps added in warp order. The
//     barrier also tells thread 0 that the stage is read, so it refills it: there
//     is no producer warp, and 512 threads keep 128 registers each (a 17th warp
//     would cut them to 96).
// Either way a row's tree depends on D alone. Weight gradients are summed in
// registers by the threads that own the columns, one partial row a CTA; pass 2
// is reduce_columns.cu.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "layernorm.h"
#include "layernorm_launch.h"

namespace rmsn {
namespace {

// Device error word of the including translation unit.
__device__ unsigned int g_ln_error;

cudaError_t read_ln_error_word(unsigned* flags, bool clear) {
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_ln_error, sizeof(v));
    if (e != cudaSuccess) return e;
    *flags |= v;
    if (clear && v) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_ln_error, &zero, sizeof(zero));
    }
    return e;
}

__device__ __forceinline__ float fma1(float a, float b, float c) { return __fmaf_rn(a, b, c); }

__device__ __forceinline__ void load8(const float* p, float (&o)[8]) {
    const float4 lo = __ldg(reinterpret_cast<const float4*>(p));
    const float4 hi = __ldg(reinterpret_cast<const float4*>(p) + 1);
    o[0] = lo.x; o[1] = lo.y; o[2] = lo.z; o[3] = lo.w;
    o[4] = hi.x; o[5] = hi.y; o[6] = hi.z; o[7] = hi.w;
}

// Effective weights of vector v.
__device__ __forceinline__ void ln_weights8(const float* w, int zc, int v, float (&o)[8]) {
    load8(w + 8 * v, o);
    if (zc) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fadd(o[e], 1.0f);
    }
}

__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }

// ---------------------------------------------------------------------------
// A group of G lanes a row (V vectors a lane: v = k G + l)
// ---------------------------------------------------------------------------
constexpr int kLnRowThreads = 256;

template <bool F16, int G, int V, int NR>
__global__ void __launch_bounds__(kLnRowThreads) ln_rows_fwd_kernel(const LnFwdArgs a) {
    constexpr int P = kLnRowThreads / G;
    const int NV = a.D >> 3;
    const int gr = threadIdx.x / G, l = threadIdx.x % G;
    pdl_wait();
    float w[V][8], b[V][8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int v = k * G + l;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[k][e] = b[k][e] = 0.0f;
        if (v < NV) {
            ln_weights8(a.w, a.zc, v, w[k]);
            if (a.b != nullptr) load8(a.b + 8 * v, b[k]);
        }
    }
    const int64_t nblocks = (a.T + P * NR - 1) / (P * NR);
    for (int64_t blk = blockIdx.x; blk < nblocks; blk += gridDim.x) {
        const int64_t row0 = blk * (P * NR) + gr;
        uint4 xv[NR][V];
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                xv[i][k] = make_uint4(0, 0, 0, 0);
                if (row0 + i * P < a.T && k * G + l < NV)
                    xv[i][k] = ld_stream(a.x + (row0 + i * P) * a.ldx + 8 * (k * G + l));
            }
        float s[NR], q[NR], mu[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            s[i] = 0.0f;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float f[8];
                unpack_act<F16>(xv[i][k], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[i] = fadd(s[i], f[e]);  // zeros beyond the row
            }
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) mu[i] = div_by_d(group_sum<G>(s[i]), a.D, a.inv_d_pow2);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            q[i] = 0.0f;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float f[8];
                unpack_act<F16>(xv[i][k], f);
                if (k * G + l < NV) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float c = fsub(f[e], mu[i]);
                        q[i] = fma1(c, c, q[i]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) q[i] = group_sum<G>(q[i]);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int64_t row = row0 + i * P;
            if (row < a.T) {
                const float r = rsqrtf(fadd(div_by_d(q[i], a.D, a.inv_d_pow2), a.eps));
                if (l == 0) {
                    a.mean[row] = mu[i];
                    a.rstd[row] = r;
                }
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    if (k * G + l < NV) {
                        float f[8];
                        unpack_act<F16>(xv[i][k], f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = fma1(fmul(fsub(f[e], mu[i]), r), w[k][e], b[k][e]);
                        st_global_cs(a.y + row * a.ldy + 8 * (k * G + l), pack_act<F16>(f));
                    }
                }
            }
        }
    }
    pdl_release();
}

// One CTA a chunk of rows; the group gr of a CTA takes the rows gr, gr + P, ...
// of the chunk in ascending order, and the groups' sums are added in group order.
template <bool F16, int G, int V, int NR, bool BIAS>
__global__ void __launch_bounds__(kLnRowThreads, V == 1 ? 3 : 2) ln_rows_bwd_kernel(const LnBwdArgs a) {
    constexpr int P = kLnRowThreads / G;
    extern __shared__ __align__(16) float comb[];  // [P][D]
    const int NV = a.D >> 3;
    const int gr = threadIdx.x / G, l = threadIdx.x % G;
    pdl_wait();
    float w[V][8], aw[V][8], ab[V][8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[k][e] = aw[k][e] = ab[k][e] = 0.0f;
        if (k * G + l < NV) ln_weights8(a.w, a.zc, k * G + l, w[k]);
    }
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
    const int64_t c1 = min(c0 + a.chunk, a.T);
    for (int64_t row0 = c0 + gr; row0 - gr < c1; row0 += P * NR) {  // every lane takes every turn: the sums are the warp's
        uint4 gv[NR][V], xv[NR][V];
        float mu[NR], r[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int64_t row = row0 + i * P;
            mu[i] = r[i] = 0.0f;
            if (row < c1) {
                mu[i] = __ldg(a.mean + row);
                r[i] = __ldg(a.rstd + row);
            }
#pragma unroll
            for (int k = 0; k < V; ++k) {
                gv[i][k] = xv[i][k] = make_uint4(0, 0, 0, 0);
                if (row < c1 && k * G + l < NV) {
                    gv[i][k] = ld_stream(a.g + row * a.ldg + 8 * (k * G + l));
                    xv[i][k] = ld_stream(a.x + row * a.ldx + 8 * (k * G + l));
                }
            }
        }
        float s1[NR], s2[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            s1[i] = s2[i] = 0.0f;
            if (row0 + i * P < c1) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    float g[8], f[8];
                    unpack_act<F16>(gv[i][k], g);
                    unpack_act<F16>(xv[i][k], f);
                    if (k * G + l < NV) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float c = fsub(f[e], mu[i]), gw = fmul(g[e], w[k][e]);
                            s1[i] = fadd(s1[i], gw);
                            s2[i] = fma1(gw, c, s2[i]);
                            aw[k][e] = fma1(g[e], fmul(c, r[i]), aw[k][e]);
                            if (BIAS) ab[k][e] = fadd(ab[k][e], g[e]);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            s1[i] = group_sum<G>(s1[i]);
            s2[i] = group_sum<G>(s2[i]);
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int64_t row = row0 + i * P;
            if (row < c1) {
                const float rc1 = fmul(r[i], div_by_d(s1[i], a.D, a.inv_d_pow2));
                const float m = -fmul(fmul(r[i], r[i]), div_by_d(fmul(s2[i], r[i]), a.D, a.inv_d_pow2));
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    if (k * G + l < NV) {
                        float g[8], f[8];
                        unpack_act<F16>(gv[i][k], g);
                        unpack_act<F16>(xv[i][k], f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float c = fsub(f[e], mu[i]), gw = fmul(g[e], w[k][e]);
                            f[e] = fma1(gw, r[i], fma1(c, m, -rc1));
                        }
                        st_global_cs(a.dx + row * a.lddx + 8 * (k * G + l), pack_act<F16>(f));
                    }
                }
            }
        }
    }
    // The groups' sums: dw, then db through the same shared memory.
#pragma unroll
    for (int part = 0; part < (BIAS ? 2 : 1); ++part) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (k * G + l < NV) {
                float4* o = reinterpret_cast<float4*>(comb + gr * a.D + 8 * (k * G + l));
                const float(&s)[8] = part ? ab[k] : aw[k];
                o[0] = make_float4(s[0], s[1], s[2], s[3]);
                o[1] = make_float4(s[4], s[5], s[6], s[7]);
            }
        }
        __syncthreads();
        float* out = a.partials + (static_cast<int64_t>(part) * gridDim.x + blockIdx.x) * a.D;
        for (int col = threadIdx.x; col < a.D; col += kLnRowThreads) {
            float t = comb[col];
            for (int p = 1; p < P; ++p) t = fadd(t, comb[p * a.D + col]);
            out[col] = t;
        }
    }
    pdl_release();
}

// ---------------------------------------------------------------------------
// A CTA a row
// ---------------------------------------------------------------------------

// K values a lane (1, 2 or 4) summed over the warp: lane l ends with the total
// of value l / (32 / K). Each halving of the values costs one exchange of half
// of them, so K sums take K - 1 + log2(32 / K) shuffles instead of 5 K.
template <int K>
__device__ __forceinline__ float warp_sums(float (&v)[K], int lane) {
    int o = 16;
#pragma unroll
    for (int n = K; n > 1; n /= 2, o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = up ? v[i + n / 2] : v[i], give = up ? v[i] : v[i + n / 2];
            v[i] = fadd(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
    }
    float t = v[0];
#pragma unroll
    for (int p = 16 / K; p > 0; p >>= 1) t = fadd(t, __shfl_xor_sync(0xffffffffu, t, p));
    return t;
}

// The warps' totals of one value in warp order; the places beyond the last warp
// hold zeros.
template <int NWMAX>
__device__ __forceinline__ float warps_total(const float* red) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < NWMAX; i += 4) {
        const float4 q = *reinterpret_cast<const float4*>(red + i);
        t = fadd(fadd(fadd(fadd(t, q.x), q.y), q.z), q.w);
    }
    return t;
}

// A copy of iteration i's stage timed out: thread 0 waits (bounded) for the
// copies still in flight, up to iteration `last`, and raises the flag.
__device__ void ln_abort(uint64_t* full, int S, int i, int last) {
    for (int j = i; j <= last; ++j) (void)mbar_wait(&full[j % S], static_cast<uint32_t>((j / S) & 1));
    atomicOr(&g_ln_error, kErrWaitTimeout);
}

// Forward: rows cta, cta + grid, ..., R an iteration. Stage: [R][D] 16-bit.
template <bool F16, int VPT, int MAXT, int R>
__global__ void __launch_bounds__(MAXT) ln_wide_fwd_kernel(const LnFwdArgs a, const int S) {
    constexpr int NW = MAXT / 32;
    extern __shared__ __align__(128) unsigned char smem[];
    const int NV = a.D >> 3, nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t row_bytes = static_cast<uint32_t>(a.D) * 2u;
    const uint32_t stage_bytes = R * row_bytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(S) * stage_bytes);
    float* red = reinterpret_cast<float*>(full + ((S + 1) & ~1));  // [2][R][NW]
    const int64_t cta = blockIdx.x, G = gridDim.x;
    const int n_my = static_cast<int>((a.T - 1 - cta) / G + 1);  // grid <= T
    const int n_it = (n_my + R - 1) / R;
    if (tid == 0) {
        for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
        fence_mbar_init();
    }
    for (int i = tid; i < 2 * R * NW; i += nt) red[i] = 0.0f;
    __syncthreads();
    pdl_wait();

    const uint64_t pol = policy_evict_first();
    auto issue = [&](int i) {
        const int s = i % S, nvalid = min(n_my - i * R, R);
        mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(nvalid) * row_bytes);
        for (int r = 0; r < nvalid; ++r)
            bulk_g2s(smem + static_cast<size_t>(s) * stage_bytes + r * row_bytes,
                     a.x + (cta + static_cast<int64_t>(i * R + r) * G) * a.ldx, row_bytes, &full[s], pol);
    };
    if (tid == 0)
        for (int i = 0; i < min(S, n_it); ++i) issue(i);

    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < n_it; ++i) {
        const bool ok = mbar_wait(&full[s], ph);
        const unsigned char* st = smem + static_cast<size_t>(s) * stage_bytes;
        const int nvalid = min(n_my - i * R, R);
        uint4 xv[R][VPT];
        float sum[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sum[r] = 0.0f;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                xv[r][j] = make_uint4(0, 0, 0, 0);
                if (r < nvalid && j * nt + tid < NV) xv[r][j] = ld_shared_v4(st + r * row_bytes + 16 * (j * nt + tid));
                float f[8];
                unpack_act<F16>(xv[r][j], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[r] = fadd(sum[r], f[e]);
            }
        }
        {
            const float t = warp_sums<R>(sum, lane);
            if (lane % (32 / R) == 0) red[(lane / (32 / R)) * NW + warp] = t;
        }
        if (!__syncthreads_and(ok ? 1 : 0)) {
            if (tid == 0) ln_abort(full, S, i, min(i + S, n_it) - 1);
            return;
        }
        if (tid == 0 && i + S < n_it) {  // every thread has the stage in registers
            fence_proxy_async_smem();
            issue(i + S);
        }
        if (++s == S) {
            s = 0;
            ph ^= 1u;
        }
        float mu[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mu[r] = div_by_d(warps_total<NW>(red + r * NW), a.D, a.inv_d_pow2);
            sum[r] = 0.0f;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if (j * nt + tid < NV) {
                    float f[8];
                    unpack_act<F16>(xv[r][j], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float c = fsub(f[e], mu[r]);
                        sum[r] = fma1(c, c, sum[r]);
                    }
                }
            }
        }
        {
            const float t = warp_sums<R>(sum, lane);
            if (lane % (32 / R) == 0) red[(R + lane / (32 / R)) * NW + warp] = t;
        }
        __syncthreads();
        float rr[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            rr[r] = rsqrtf(fadd(div_by_d(warps_total<NW>(red + (R + r) * NW), a.D, a.inv_d_pow2), a.eps));
            if (tid == 0 && r < nvalid) {
                const int64_t row = cta + static_cast<int64_t>(i * R + r) * G;
                a.mean[row] = mu[r];
                a.rstd[row] = rr[r];
            }
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = j * nt + tid;
            if (v < NV) {
                float w[8], b[8];
                ln_weights8(a.w, a.zc, v, w);
                if (a.b != nullptr) {
                    load8(a.b + 8 * v, b);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) b[e] = 0.0f;
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (r < nvalid) {
                        float f[8];
                        unpack_act<F16>(xv[r][j], f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = fma1(fmul(fsub(f[e], mu[r]), rr[r]), w[e], b[e]);
                        st_global_cs(a.y + (cta + static_cast<int64_t>(i * R + r) * G) * a.ldy + 8 * v, pack_act<F16>(f));
                    }
                }
            }
        }
    }
    pdl_release();
}

// Backward: one CTA a chunk of rows, R an iteration. Stage: [R][g | x][D]
// 16-bit. HOLD: the operands are read from the stage again after the reduction
// instead of being kept in registers, and the stage is refilled an iteration later.
template <bool F16, int VPT, int MAXT, int MINB, int R, bool BIAS, bool HOLD>
__global__ void __launch_bounds__(MAXT, MINB) ln_wide_bwd_kernel(const LnBwdArgs a, const int S) {
    constexpr int NW = MAXT / 32;
    extern __shared__ __align__(128) unsigned char smem[];
    const int NV = a.D >> 3, nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t row_bytes = static_cast<uint32_t>(a.D) * 2u;
    const uint32_t stage_bytes = 2 * R * row_bytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(S) * stage_bytes);
    float* red = reinterpret_cast<float*>(full + ((S + 1) & ~1));  // [2][2 R][NW]
    float2* stat = reinterpret_cast<float2*>(red + 4 * R * NW);    // [chunk]: mean, rstd
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
    const int n_my = static_cast<int>(min(static_cast<int64_t>(a.chunk), a.T - row0));
    const int n_it = (n_my + R - 1) / R;
    if (tid == 0) {
        for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
        fence_mbar_init();
    }
    for (int i = tid; i < 4 * R * NW; i += nt) red[i] = 0.0f;
    __syncthreads();
    pdl_wait();

    const uint64_t pol = policy_evict_first();
    auto issue = [&](int i) {
        const int s = i % S, nvalid = min(n_my - i * R, R);
        mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(nvalid) * 2u * row_bytes);
        for (int r = 0; r < nvalid; ++r) {
            unsigned char* dst = smem + static_cast<size_t>(s) * stage_bytes + r * 2 * row_bytes;
            const int64_t row = row0 + i * R + r;
            bulk_g2s(dst, a.g + row * a.ldg, row_bytes, &full[s], pol);
            bulk_g2s(dst + row_bytes, a.x + row * a.ldx, row_bytes, &full[s], pol);
        }
    };
    if (tid == 0)
        for (int i = 0; i < min(S, n_it); ++i) issue(i);
    for (int i = tid; i < n_my; i += nt) stat[i] = make_float2(__ldg(a.mean + row0 + i), __ldg(a.rstd + row0 + i));
    float aw[VPT][8], ab[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) aw[j][e] = ab[j][e] = 0.0f;
    __syncthreads();

    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < n_it; ++i) {
        const bool ok = mbar_wait(&full[s], ph);
        const unsigned char* st = smem + static_cast<size_t>(s) * stage_bytes;
        const int nvalid = min(n_my - i * R, R);
        uint4 gv[R][VPT], xv[R][VPT];
        float sum[2 * R];
        float2 mr[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sum[2 * r] = sum[2 * r + 1] = 0.0f;
            if (r < nvalid) {
                mr[r] = stat[i * R + r];
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int v = j * nt + tid;
                    if (v < NV) {
                        gv[r][j] = ld_shared_v4(st + r * 2 * row_bytes + 16 * v);
                        xv[r][j] = ld_shared_v4(st + r * 2 * row_bytes + row_bytes + 16 * v);
                        float g[8], f[8], w[8];
                        unpack_act<F16>(gv[r][j], g);
                        unpack_act<F16>(xv[r][j], f);
                        ln_weights8(a.w, a.zc, v, w);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float c = fsub(f[e], mr[r].x), gw = fmul(g[e], w[e]);
                            sum[2 * r] = fadd(sum[2 * r], gw);
                            sum[2 * r + 1] = fma1(gw, c, sum[2 * r + 1]);
                            aw[j][e] = fma1(g[e], fmul(c, mr[r].y), aw[j][e]);
                            if (BIAS) ab[j][e] = fadd(ab[j][e], g[e]);
                        }
                    }
                }
            }
        }
        float* rb = red + (i & 1) * 2 * R * NW;
        {
            const float t = warp_sums<2 * R>(sum, lane);
            if (lane % (16 / R) == 0) rb[(lane / (16 / R)) * NW + warp] = t;
        }
        if (!__syncthreads_and(ok ? 1 : 0)) {
            if (tid == 0) ln_abort(full, S, i, min(i + S - (HOLD ? 1 : 0), n_it) - 1);
            return;
        }
        // Free now: this iteration's stage, or with HOLD the one before it.
        const int next = HOLD ? i - 1 + S : i + S;
        if (tid == 0 && next < n_it && next >= S) {
            fence_proxy_async_smem();
            issue(next);
        }
        if (++s == S) {
            s = 0;
            ph ^= 1u;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r < nvalid) {
                const float rs = mr[r].y;
                const float rc1 = fmul(rs, div_by_d(warps_total<NW>(rb + 2 * r * NW), a.D, a.inv_d_pow2));
                const float m = -fmul(fmul(rs, rs), div_by_d(fmul(warps_total<NW>(rb + (2 * r + 1) * NW), rs), a.D, a.inv_d_pow2));
                uint16_t* dx = a.dx + (row0 + i * R + r) * a.lddx;
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int v = j * nt + tid;
                    if (v < NV) {
                        if (HOLD) {
                            gv[r][j] = ld_shared_v4(st + r * 2 * row_bytes + 16 * v);
                            xv[r][j] = ld_shared_v4(st + r * 2 * row_bytes + row_bytes + 16 * v);
                        }
                        float g[8], f[8], w[8];
                        unpack_act<F16>(gv[r][j], g);
                        unpack_act<F16>(xv[r][j], f);
                        ln_weights8(a.w, a.zc, v, w);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float c = fsub(f[e], mr[r].x), gw = fmul(g[e], w[e]);
                            f[e] = fma1(gw, rs, fma1(c, m, -rc1));
                        }
                        st_global_cs(dx + 8 * v, pack_act<F16>(f));
                    }
                }
            }
        }
    }
    // The chunk's partial rows, read again by pass 2 at once: kept in L2.
    const uint64_t keep = policy_evict_last();
    float* pw = a.partials + static_cast<int64_t>(blockIdx.x) * a.D;
    float* pb = pw + static_cast<int64_t>(gridDim.x) * a.D;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = j * nt + tid;
        if (v < NV) {
            st_global_f4_hint(pw + 8 * v, aw[j][0], aw[j][1], aw[j][2], aw[j][3], keep);
            st_global_f4_hint(pw + 8 * v + 4, aw[j][4], aw[j][5], aw[j][6], aw[j][7], keep);
            if (BIAS) {
                st_global_f4_hint(pb + 8 * v, ab[j][0], ab[j][1], ab[j][2], ab[j][3], keep);
                st_global_f4_hint(pb + 8 * v + 4, ab[j][4], ab[j][5], ab[j][6], ab[j][7], keep);
            }
        }
    }
    pdl_release();
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
constexpr size_t kLnMaxSmem = 227 * 1024;

template <bool F16, int G, int V, int NR>
cudaError_t rows_fwd(const LnFwdArgs& a, cudaStream_t st) {
    constexpr int rows = kLnRowThreads / G * NR;
    const void* kern = reinterpret_cast<const void*>(ln_rows_fwd_kernel<F16, G, V, NR>);
    const int occ = ctas_per_sm(kern, kLnRowThreads, 0);
    if (occ < 1) return cudaErrorInvalidConfiguration;
    const int64_t grid = std::min<int64_t>((a.T + rows - 1) / rows, static_cast<int64_t>(sm_count()) * occ);
    return launch_kernel(ln_rows_fwd_kernel<F16, G, V, NR>, static_cast<unsigned>(grid), kLnRowThreads, 0, st, a);
}

template <bool F16, int VPT, int MAXT, int R>
cudaError_t wide_fwd(const LnFwdArgs& a, size_t ring, int most, cudaStream_t st) {
    const int NV = a.D / 8;
    const int threads = ((NV + VPT - 1) / VPT + 31) / 32 * 32;
    const size_t stage = static_cast<size_t>(R) * a.D * 2;
    const size_t fixed = 2 * R * (MAXT / 32) * 4 + 16;
    const int S = static_cast<int>(std::min<size_t>(std::max<size_t>(ring / stage, 2), 16));
    const size_t smem = S * (stage + 8) + fixed;
    if (smem > kLnMaxSmem) return cudaErrorInvalidConfiguration;
    const void* kern = reinterpret_cast<const void*>(ln_wide_fwd_kernel<F16, VPT, MAXT, R>);
    cudaError_t e = ensure_smem_attr(kern, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int occ = std::min(ctas_per_sm(kern, threads, static_cast<int>(smem)), most);
    if (occ < 1) return cudaErrorInvalidConfiguration;
    const int64_t grid = std::min<int64_t>(a.T, static_cast<int64_t>(sm_count()) * occ);
    return launch_kernel(ln_wide_fwd_kernel<F16, VPT, MAXT, R>, static_cast<unsigned>(grid), threads, smem, st, a, S);
}

template <bool F16>
cudaError_t ln_fwd_dispatch(const LnFwdArgs& a, cudaStream_t st) {
    const int NV = a.D / 8;
    if (NV <= 1) return rows_fwd<F16, 1, 1, 4>(a, st);
    if (NV <= 2) return rows_fwd<F16, 2, 1, 4>(a, st);
    if (NV <= 4) return rows_fwd<F16, 4, 1, 4>(a, st);
    if (NV <= 8) return rows_fwd<F16, 8, 1, 4>(a, st);
    if (NV <= 16) return rows_fwd<F16, 16, 1, 4>(a, st);
    if (NV <= 32) return rows_fwd<F16, 32, 1, 4>(a, st);
    if (NV <= 64) return rows_fwd<F16, 32, 2, 2>(a, st);
    if (NV <= 128) return rows_fwd<F16, 32, 4, 1>(a, st);
    if (NV <= 256) return wide_fwd<F16, 1, 256, 4>(a, 64 * 1024, 3, st);
    if (NV <= 512) return wide_fwd<F16, 2, 256, 4>(a, 96 * 1024, 3, st);
    if (NV <= 1024) return wide_fwd<F16, 4, 256, 2>(a, 96 * 1024, 2, st);
    return wide_fwd<F16, 4, 512, 2>(a, 192 * 1024, 1, st);
}

template <bool F16, int G, int V, int NR, bool BIAS>
cudaError_t rows_bwd(const LnBwdArgs& a, unsigned grid, cudaStream_t st) {
    const size_t smem = static_cast<size_t>(kLnRowThreads / G) * a.D * 4;
    return launch_kernel(ln_rows_bwd_kernel<F16, G, V, NR, BIAS>, grid, kLnRowThreads, smem, st, a);
}

template <bool F16, int VPT, int MAXT, int MINB, int R, bool BIAS, bool HOLD>
cudaError_t wide_bwd(const LnBwdArgs& a, unsigned grid, size_t ring, cudaStream_t st) {
    const int NV = a.D / 8;
    const int threads = ((NV + VPT - 1) / VPT + 31) / 32 * 32;
    const size_t stage = static_cast<size_t>(2) * R * a.D * 2;
    const size_t fixed = 4 * R * (MAXT / 32) * 4 + 8 * static_cast<size_t>(a.chunk) + 16;
    int S = static_cast<int>(std::min<size_t>(std::max<size_t>(ring / stage, HOLD ? 3 : 2), 16));
    const size_t smem = S * (stage + 8) + fixed;
    if (smem > kLnMaxSmem) return cudaErrorInvalidConfiguration;
    const void* kern = reinterpret_cast<const void*>(ln_wide_bwd_kernel<F16, VPT, MAXT, MINB, R, BIAS, HOLD>);
    cudaError_t e = ensure_smem_attr(kern, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_kernel(ln_wide_bwd_kernel<F16, VPT, MAXT, MINB, R, BIAS, HOLD>, grid, threads, smem, st, a, S);
}

template <bool F16, bool BIAS>
cudaError_t ln_bwd_dispatch(const LnBwdArgs& a, unsigned grid, cudaStream_t st) {
    const int NV = a.D / 8;
    if (NV <= 1) return rows_bwd<F16, 1, 1, 2, BIAS>(a, grid, st);
    if (NV <= 2) return rows_bwd<F16, 2, 1, 2, BIAS>(a, grid, st);
    if (NV <= 4) return rows_bwd<F16, 4, 1, 2, BIAS>(a, grid, st);
    if (NV <= 8) return rows_bwd<F16, 8, 1, 2, BIAS>(a, grid, st);
    if (NV <= 16) return rows_bwd<F16, 16, 1, 2, BIAS>(a, grid, st);
    if (NV <= 32) return rows_bwd<F16, 32, 1, 2, BIAS>(a, grid, st);
    if (NV <= 64) return rows_bwd<F16, 32, 2, 1, BIAS>(a, grid, st);
    if (NV <= 256) return wide_bwd<F16, 1, 256, 3, 2, BIAS, false>(a, grid, 48 * 1024, st);
    if (NV <= 512) return wide_bwd<F16, 2, 256, 2, 1, BIAS, false>(a, grid, 64 * 1024, st);
    if (NV <= 1024) return wide_bwd<F16, 2, 512, 1, 1, BIAS, false>(a, grid, 128 * 1024, st);
    return wide_bwd<F16, 4, 512, 1, 1, BIAS, true>(a, grid, 192 * 1024, st);
}

}  // namespace
}  // namespace rmsn
