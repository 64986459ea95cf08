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

// Pairs of fp32 operations in one instruction, each half rounded as the scalar
// operation is: half the issue slots. Every product that feeds a sum is an
// explicit fused multiply-add, so nothing is left for ptxas to contract.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// Eight values as four pairs.
struct Oct { float2 p[4]; };

__device__ __forceinline__ Oct oct_zero() {
    Oct o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.p[i] = make_float2(0.0f, 0.0f);
    return o;
}

template <bool F16>
__device__ __forceinline__ Oct oct_unpack(const uint4 v) {
    float f[8];
    unpack_act<F16>(v, f);
    Oct o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.p[i] = pair(f, 2 * i);
    return o;
}

template <bool F16>
__device__ __forceinline__ uint4 oct_pack(const Oct& o) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = o.p[i].x;
        f[2 * i + 1] = o.p[i].y;
    }
    return pack_act<F16>(f);
}

__device__ __forceinline__ Oct oct_of(float4 lo, float4 hi) {
    Oct o;
    o.p[0] = make_float2(lo.x, lo.y); o.p[1] = make_float2(lo.z, lo.w);
    o.p[2] = make_float2(hi.x, hi.y); o.p[3] = make_float2(hi.z, hi.w);
    return o;
}

__device__ __forceinline__ Oct load_oct(const float* p) {
    return oct_of(__ldg(reinterpret_cast<const float4*>(p)), __ldg(reinterpret_cast<const float4*>(p) + 1));
}

// Effective weights of vector v.
__device__ __forceinline__ Oct ln_weights(const float* w, int zc, int v) {
    Oct o = load_oct(w + 8 * v);
    if (zc) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o.p[i] = fadd2(o.p[i], both(1.0f));
    }
    return o;
}

__device__ __forceinline__ Oct ln_bias(const float* b, int v) { return b != nullptr ? load_oct(b + 8 * v) : oct_zero(); }

__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }

// s / D through the fp32 reciprocal of D, its remainder taken back once: the
// correctly rounded quotient (the mean of a constant row is that constant), in
// three instructions in a division's place. An infinite sum stays infinite.
__device__ __forceinline__ float over_d(float s, float d, float rcp_d) {
    const float q = fmul(s, rcp_d);
    const float e = __fmaf_rn(__fmaf_rn(-q, d, s), rcp_d, q);
    return fabsf(q) < __int_as_float(0x7f800000) ? e : q;
}

// Parts of a lane's sums, even and odd elements apart.
__device__ __forceinline__ float2 oct_sum(float2 s, const Oct& o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fadd2(s, o.p[i]);
    return s;
}
// o - mu in place; the squares' sum is added to q.
__device__ __forceinline__ float2 oct_centre(Oct& o, float mu, float2 q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o.p[i] = fadd2(o.p[i], both(-mu));
        q = fma2(o.p[i], o.p[i], q);
    }
    return q;
}
// (c r) w + b
__device__ __forceinline__ Oct oct_affine(const Oct& c, float r, const Oct& w, const Oct& b) {
    Oct o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.p[i] = fma2(fmul2(c.p[i], both(r)), w.p[i], b.p[i]);
    return o;
}
// The backward's first half for eight values: x becomes c = x - mu and g becomes
// gw = g w, their sums (s1: gw, s2: gw c) and the weight gradients grow.
template <bool BIAS>
__device__ __forceinline__ void oct_grad(Oct& g, Oct& x, const Oct& w, float mu, float r, float2& s1, float2& s2,
                                         Oct& aw, Oct& ab) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x.p[i] = fadd2(x.p[i], both(-mu));
        aw.p[i] = fma2(g.p[i], fmul2(x.p[i], both(r)), aw.p[i]);
        if (BIAS) ab.p[i] = fadd2(ab.p[i], g.p[i]);
        s1 = fma2(g.p[i], w.p[i], s1);
        g.p[i] = fmul2(g.p[i], w.p[i]);
        s2 = fma2(g.p[i], x.p[i], s2);
    }
}
// r gw + (m c - r c1)
__device__ __forceinline__ Oct oct_dx(const Oct& gw, const Oct& c, float r, float m, float rc1) {
    Oct o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.p[i] = fma2(gw.p[i], both(r), fma2(c.p[i], both(m), both(-rc1)));
    return o;
}

// ---------------------------------------------------------------------------
// A group of G lanes a row (V vectors a lane: v = k G + l)
// ---------------------------------------------------------------------------
constexpr int kLnRowThreads = 256;

// Every lane keeps its own ring of S turns in flight: it copies its vectors to
// its own slots of shared memory (cp.async, past L1) and reads them back itself,
// so a wait for its own copies is all the synchronisation there is, and data in
// flight costs no registers. Slot layout [turn][vector][thread]: conflict-free.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// w_eff and b of a row in shared memory as [w low | w high | b low | b high][NV]
// float4 (the halves of a vector's eight): conflict-free reads.
__device__ __forceinline__ void stage_weights(float4* wb, const float* w, const float* b, int zc, int NV) {
    for (int v = threadIdx.x; v < NV; v += blockDim.x) {
        const Oct x = ln_weights(w, zc, v);
        wb[v] = make_float4(x.p[0].x, x.p[0].y, x.p[1].x, x.p[1].y);
        wb[NV + v] = make_float4(x.p[2].x, x.p[2].y, x.p[3].x, x.p[3].y);
        if (b != nullptr) {
            const Oct y = load_oct(b + 8 * v);
            wb[2 * NV + v] = make_float4(y.p[0].x, y.p[0].y, y.p[1].x, y.p[1].y);
            wb[3 * NV + v] = make_float4(y.p[2].x, y.p[2].y, y.p[3].x, y.p[3].y);
        }
    }
}
__device__ __forceinline__ Oct staged_weights(const float4* wb, int NV, int v) { return oct_of(wb[v], wb[NV + v]); }
__device__ __forceinline__ Oct staged_bias(const float4* wb, bool bias, int NV, int v) {
    return bias ? oct_of(wb[2 * NV + v], wb[3 * NV + v]) : oct_zero();
}

// Weights in registers at one vector a lane, else in shared memory, read once
// for the NR rows of a turn.
template <bool F16, int G, int V, int NR, int S, int MINB>
__global__ void __launch_bounds__(kLnRowThreads, MINB) ln_rows_fwd_kernel(const LnFwdArgs a) {
    constexpr int P = kLnRowThreads / G;
    extern __shared__ __align__(16) uint4 ring[];  // [S][NR][V][threads], then V > 1: the weights
    const int NV = a.D >> 3;
    const int gr = threadIdx.x / G, l = threadIdx.x % G;
    const bool bias = a.b != nullptr;
    float4* wb = reinterpret_cast<float4*>(ring + S * NR * V * kLnRowThreads);
    pdl_wait();
    const int64_t nblocks = (a.T + P * NR - 1) / (P * NR);
    auto fetch = [&](int64_t blk, int s) {
        if (blk < nblocks) {
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int64_t row = blk * (P * NR) + gr + i * P;
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (row < a.T && k * G + l < NV)
                        cp_async16(ring + ((s * NR + i) * V + k) * kLnRowThreads + threadIdx.x, a.x + row * a.ldx + 8 * (k * G + l));
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) fetch(blockIdx.x + static_cast<int64_t>(s) * gridDim.x, s);
    Oct w1 = oct_zero(), b1 = oct_zero();
    if constexpr (V == 1) {
        if (l < NV) {
            w1 = ln_weights(a.w, a.zc, l);
            b1 = ln_bias(a.b, l);
        }
    } else {
        stage_weights(wb, a.w, a.b, a.zc, NV);
        __syncthreads();
    }
    const float d = static_cast<float>(a.D);
    int s = 0;
    for (int64_t blk = blockIdx.x; blk < nblocks; blk += gridDim.x) {
        const int64_t row0 = blk * (P * NR) + gr;
        cp_async_wait<S - 2>();
        Oct c[NR][V];
        float mu[NR], r[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                uint4 xv = make_uint4(0, 0, 0, 0);  // zeros beyond the row
                if (row0 + i * P < a.T && k * G + l < NV) xv = ring[((s * NR + i) * V + k) * kLnRowThreads + threadIdx.x];
                c[i][k] = oct_unpack<F16>(xv);
                sum = oct_sum(sum, c[i][k]);
            }
            mu[i] = fadd(sum.x, sum.y);
        }
        // The slots of the turn before are free: every value of them is used.
        fetch(blk + static_cast<int64_t>(S - 1) * gridDim.x, s == 0 ? S - 1 : s - 1);
        if (++s == S) s = 0;
#pragma unroll
        for (int i = 0; i < NR; ++i) mu[i] = over_d(group_sum<G>(mu[i]), d, a.rcp_d);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            float2 q = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (k * G + l < NV) q = oct_centre(c[i][k], mu[i], q);
            r[i] = fadd(q.x, q.y);
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) r[i] = rsqrtf(fadd(fmul(group_sum<G>(r[i]), a.rcp_d), a.eps));
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int v = k * G + l;
            if (v < NV) {
                Oct w = w1, b = b1;
                if constexpr (V > 1) {
                    w = staged_weights(wb, NV, v);
                    b = staged_bias(wb, bias, NV, v);
                }
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const int64_t row = row0 + i * P;
                    if (row < a.T) st_global_cs(a.y + row * a.ldy + 8 * v, oct_pack<F16>(oct_affine(c[i][k], r[i], w, b)));
                }
            }
        }
        if (l == 0) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
                if (row0 + i * P < a.T) {
                    a.mean[row0 + i * P] = mu[i];
                    a.rstd[row0 + i * P] = r[i];
                }
        }
    }
    cp_async_wait<0>();
    pdl_release();
}

// One CTA a chunk of rows; the group gr of a CTA takes the rows gr, gr + P, ...
// of the chunk in ascending order, and the groups' sums are added in group order.
template <bool F16, int G, int V, int NR, int S, int MINB, bool BIAS>
__global__ void __launch_bounds__(kLnRowThreads, MINB) ln_rows_bwd_kernel(const LnBwdArgs a) {
    constexpr int P = kLnRowThreads / G;
    extern __shared__ __align__(16) uint4 ring[];  // [S][NR][g | x][V][threads]; at the end [P][D] sums
    const int NV = a.D >> 3;
    const int gr = threadIdx.x / G, l = threadIdx.x % G;
    pdl_wait();
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
    const int n_rows = static_cast<int>(min(static_cast<int64_t>(a.chunk), a.T - c0));
    auto slot = [&](int s, int i, int op, int k) { return ring + (((s * NR + i) * 2 + op) * V + k) * kLnRowThreads + threadIdx.x; };
    auto fetch = [&](int at, int s) {  // the turn whose first row is c0 + at
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int rel = at + gr + i * P;
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (rel < n_rows && k * G + l < NV) {
                    cp_async16(slot(s, i, 0, k), a.g + (c0 + rel) * a.ldg + 8 * (k * G + l));
                    cp_async16(slot(s, i, 1, k), a.x + (c0 + rel) * a.ldx + 8 * (k * G + l));
                }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) fetch(s * P * NR, s);
    float mu1[NR], r1[NR];  // the next turn's statistics
    auto stats = [&](int at) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int rel = at + gr + i * P;
            mu1[i] = r1[i] = 0.0f;
            if (rel < n_rows) {
                mu1[i] = __ldg(a.mean + c0 + rel);
                r1[i] = __ldg(a.rstd + c0 + rel);
            }
        }
    };
    stats(0);
    Oct w[V], aw[V], ab[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        w[k] = aw[k] = ab[k] = oct_zero();
        if (k * G + l < NV) w[k] = ln_weights(a.w, a.zc, k * G + l);
    }
    int s = 0;
    for (int at = 0; at < n_rows; at += P * NR) {  // every lane takes every turn: the sums are the warp's
        cp_async_wait<S - 2>();
        Oct g[NR][V], c[NR][V];
        float s1[NR], s2[NR], mu[NR], r[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            mu[i] = mu1[i];
            r[i] = r1[i];
        }
        stats(at + P * NR);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            float2 p1 = make_float2(0.0f, 0.0f), p2 = p1;
            if (at + gr + i * P < n_rows) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    if (k * G + l < NV) {
                        g[i][k] = oct_unpack<F16>(*slot(s, i, 0, k));
                        c[i][k] = oct_unpack<F16>(*slot(s, i, 1, k));
                        oct_grad<BIAS>(g[i][k], c[i][k], w[k], mu[i], r[i], p1, p2, aw[k], ab[k]);
                    }
                }
            }
            s1[i] = fadd(p1.x, p1.y);
            s2[i] = fadd(p2.x, p2.y);
        }
        fetch(at + (S - 1) * P * NR, s == 0 ? S - 1 : s - 1);
        if (++s == S) s = 0;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            s1[i] = group_sum<G>(s1[i]);
            s2[i] = group_sum<G>(s2[i]);
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int rel = at + gr + i * P;
            if (rel < n_rows) {
                const float rc1 = fmul(r[i], fmul(s1[i], a.rcp_d));
                const float m = -fmul(fmul(r[i], r[i]), fmul(fmul(s2[i], r[i]), a.rcp_d));
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (k * G + l < NV)
                        st_global_cs(a.dx + (c0 + rel) * a.lddx + 8 * (k * G + l),
                                     oct_pack<F16>(oct_dx(g[i][k], c[i][k], r[i], m, rc1)));
            }
        }
    }
    cp_async_wait<0>();
    // The groups' sums: dw, then db through the same shared memory.
    float* comb = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int part = 0; part < (BIAS ? 2 : 1); ++part) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (k * G + l < NV) {
                float4* o = reinterpret_cast<float4*>(comb + gr * a.D + 8 * (k * G + l));
                const Oct& t = part ? ab[k] : aw[k];
                o[0] = make_float4(t.p[0].x, t.p[0].y, t.p[1].x, t.p[1].y);
                o[1] = make_float4(t.p[2].x, t.p[2].y, t.p[3].x, t.p[3].y);
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
template <bool F16, int VPT, int MAXT, int MINB, int R>
__global__ void __launch_bounds__(MAXT, MINB) ln_wide_fwd_kernel(const LnFwdArgs a, const int S) {
    constexpr int NW = MAXT / 32;
    extern __shared__ __align__(128) unsigned char smem[];
    const int NV = a.D >> 3, nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t row_bytes = static_cast<uint32_t>(a.D) * 2u;
    const uint32_t stage_bytes = R * row_bytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(S) * stage_bytes);
    float* red = reinterpret_cast<float*>(full + ((S + 1) & ~1));  // [2][R][NW]
    float4* wb = reinterpret_cast<float4*>(red + 2 * R * NW);      // weights (and bias)
    const bool bias = a.b != nullptr;
    const int64_t cta = blockIdx.x, G = gridDim.x;
    const float d = static_cast<float>(a.D);
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
    stage_weights(wb, a.w, a.b, a.zc, NV);  // seen by every thread after the first barrier below

    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < n_it; ++i) {
        const bool ok = mbar_wait(&full[s], ph);
        const unsigned char* st = smem + static_cast<size_t>(s) * stage_bytes;
        const int nvalid = min(n_my - i * R, R);
        Oct c[R][VPT];
        float sum[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 p = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                uint4 xv = make_uint4(0, 0, 0, 0);
                if (r < nvalid && j * nt + tid < NV) xv = ld_shared_v4(st + r * row_bytes + 16 * (j * nt + tid));
                c[r][j] = oct_unpack<F16>(xv);
                p = oct_sum(p, c[r][j]);
            }
            sum[r] = fadd(p.x, p.y);
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
            mu[r] = over_d(warps_total<NW>(red + r * NW), d, a.rcp_d);
            float2 q = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (j * nt + tid < NV) q = oct_centre(c[r][j], mu[r], q);
            sum[r] = fadd(q.x, q.y);
        }
        {
            const float t = warp_sums<R>(sum, lane);
            if (lane % (32 / R) == 0) red[(R + lane / (32 / R)) * NW + warp] = t;
        }
        __syncthreads();
        float rr[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            rr[r] = rsqrtf(fadd(fmul(warps_total<NW>(red + (R + r) * NW), a.rcp_d), a.eps));
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
                const Oct w = staged_weights(wb, NV, v), b = staged_bias(wb, bias, NV, v);
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (r < nvalid)
                        st_global_cs(a.y + (cta + static_cast<int64_t>(i * R + r) * G) * a.ldy + 8 * v,
                                     oct_pack<F16>(oct_affine(c[r][j], rr[r], w, b)));
            }
        }
    }
    pdl_release();
}

// Backward: one CTA a chunk of rows, R an iteration. Stage: [R][g | x][D]
// 16-bit. Between the two halves of a row its c and g w stay in registers; SW
// (the widest rows, whose weight gradients take 64 registers): the packed g and x
// stay instead, and the weights lie in shared memory.
template <bool F16, int VPT, int MAXT, int MINB, int R, bool BIAS, bool SW>
__global__ void __launch_bounds__(MAXT, MINB) ln_wide_bwd_kernel(const LnBwdArgs a, const int S) {
    constexpr int NW = MAXT / 32;
    extern __shared__ __align__(128) unsigned char smem[];
    const int NV = a.D >> 3, nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t row_bytes = static_cast<uint32_t>(a.D) * 2u;
    const uint32_t stage_bytes = 2 * R * row_bytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(S) * stage_bytes);
    float* red = reinterpret_cast<float*>(full + ((S + 1) & ~1));  // [2][2 R][NW]
    float4* wb = reinterpret_cast<float4*>(red + 4 * R * NW);      // SW: the weights
    float2* stat = reinterpret_cast<float2*>(wb + (SW ? 2 * NV : 0));  // [chunk]: mean, rstd
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
    Oct w[VPT], aw[VPT], ab[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        w[j] = aw[j] = ab[j] = oct_zero();
        if (!SW && j * nt + tid < NV) w[j] = ln_weights(a.w, a.zc, j * nt + tid);
    }
    if constexpr (SW) stage_weights(wb, a.w, nullptr, a.zc, NV);
    __syncthreads();

    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < n_it; ++i) {
        const bool ok = mbar_wait(&full[s], ph);
        const unsigned char* st = smem + static_cast<size_t>(s) * stage_bytes;
        const int nvalid = min(n_my - i * R, R);
        Oct g[R][VPT], c[R][VPT];  // gw and x - mu
        uint4 gv[R][VPT], xv[R][VPT];
        float sum[2 * R];
        float2 mr[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 p1 = make_float2(0.0f, 0.0f), p2 = p1;
            if (r < nvalid) {
                mr[r] = stat[i * R + r];
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int v = j * nt + tid;
                    if (v < NV) {
                        gv[r][j] = ld_shared_v4(st + r * 2 * row_bytes + 16 * v);
                        xv[r][j] = ld_shared_v4(st + r * 2 * row_bytes + row_bytes + 16 * v);
                        g[r][j] = oct_unpack<F16>(gv[r][j]);
                        c[r][j] = oct_unpack<F16>(xv[r][j]);
                        oct_grad<BIAS>(g[r][j], c[r][j], SW ? staged_weights(wb, NV, v) : w[j], mr[r].x, mr[r].y, p1, p2,
                                       aw[j], ab[j]);
                    }
                }
            }
            sum[2 * r] = fadd(p1.x, p1.y);
            sum[2 * r + 1] = fadd(p2.x, p2.y);
        }
        float* rb = red + (i & 1) * 2 * R * NW;
        {
            const float t = warp_sums<2 * R>(sum, lane);
            if (lane % (16 / R) == 0) rb[(lane / (16 / R)) * NW + warp] = t;
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
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r < nvalid) {
                const float rs = mr[r].y;
                const float rc1 = fmul(rs, fmul(warps_total<NW>(rb + 2 * r * NW), a.rcp_d));
                const float m = -fmul(fmul(rs, rs), fmul(fmul(warps_total<NW>(rb + (2 * r + 1) * NW), rs), a.rcp_d));
                uint16_t* dx = a.dx + (row0 + i * R + r) * a.lddx;
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int v = j * nt + tid;
                    if (v < NV) {
                        if constexpr (SW) {
                            const Oct wv = staged_weights(wb, NV, v);
                            g[r][j] = oct_unpack<F16>(gv[r][j]);
                            c[r][j] = oct_unpack<F16>(xv[r][j]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                g[r][j].p[e] = fmul2(g[r][j].p[e], wv.p[e]);
                                c[r][j].p[e] = fadd2(c[r][j].p[e], both(-mr[r].x));
                            }
                        }
                        st_global_cs(dx + 8 * v, oct_pack<F16>(oct_dx(g[r][j], c[r][j], rs, m, rc1)));
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
            st_global_f4_hint(pw + 8 * v, aw[j].p[0].x, aw[j].p[0].y, aw[j].p[1].x, aw[j].p[1].y, keep);
            st_global_f4_hint(pw + 8 * v + 4, aw[j].p[2].x, aw[j].p[2].y, aw[j].p[3].x, aw[j].p[3].y, keep);
            if (BIAS) {
                st_global_f4_hint(pb + 8 * v, ab[j].p[0].x, ab[j].p[0].y, ab[j].p[1].x, ab[j].p[1].y, keep);
                st_global_f4_hint(pb + 8 * v + 4, ab[j].p[2].x, ab[j].p[2].y, ab[j].p[3].x, ab[j].p[3].y, keep);
            }
        }
    }
    pdl_release();
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
constexpr size_t kLnMaxSmem = 227 * 1024;

template <bool F16, int G, int V, int NR, int S, int MINB>
cudaError_t rows_fwd(const LnFwdArgs& a, cudaStream_t st) {
    constexpr int rows = kLnRowThreads / G * NR;
    const int smem = S * NR * V * kLnRowThreads * 16 + (V > 1 ? a.D * 8 : 0);
    const auto kern = ln_rows_fwd_kernel<F16, G, V, NR, S, MINB>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    const int occ = ctas_per_sm(reinterpret_cast<const void*>(kern), kLnRowThreads, smem);
    if (occ < 1) return cudaErrorInvalidConfiguration;
    const int64_t grid = std::min<int64_t>((a.T + rows - 1) / rows, static_cast<int64_t>(sm_count()) * occ);
    return launch_kernel(kern, static_cast<unsigned>(grid), kLnRowThreads, smem, st, a);
}

template <bool F16, int VPT, int MAXT, int MINB, int R>
cudaError_t wide_fwd(const LnFwdArgs& a, size_t ring, cudaStream_t st) {
    const int NV = a.D / 8;
    const int threads = ((NV + VPT - 1) / VPT + 31) / 32 * 32;
    const size_t stage = static_cast<size_t>(R) * a.D * 2;
    const size_t fixed = 2 * R * (MAXT / 32) * 4 + 16 + static_cast<size_t>(a.D) * (a.b != nullptr ? 8 : 4);
    const int S = static_cast<int>(std::min<size_t>(std::max<size_t>(ring / stage, 2), 16));
    const size_t smem = S * (stage + 8) + fixed;
    if (smem > kLnMaxSmem) return cudaErrorInvalidConfiguration;
    const auto kern = ln_wide_fwd_kernel<F16, VPT, MAXT, MINB, R>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int occ = ctas_per_sm(reinterpret_cast<const void*>(kern), threads, static_cast<int>(smem));
    if (occ < 1) return cudaErrorInvalidConfiguration;
    const int64_t grid = std::min<int64_t>(a.T, static_cast<int64_t>(sm_count()) * occ);
    return launch_kernel(kern, static_cast<unsigned>(grid), threads, smem, st, a, S);
}

// lanes, vectors a lane, rows a turn, turns in flight, CTAs an SM
#ifndef LN_F1
#define LN_F1 1, 2, 4, 4
#endif
#ifndef LN_FNARROW
#define LN_FNARROW(n) rows_fwd<F16, n, LN_F1>(a, st)
#endif
#ifndef LN_F2
#define LN_F2 2, 2, 3, 4
#endif
#ifndef LN_F4
#define LN_F4 4, 1, 3, 3
#endif
#ifndef LN_F8
#define LN_F8 8, 1, 2, 2
#endif
// vectors a thread, threads, CTAs an SM, rows an iteration; ring KB
#ifndef LN_W2
#define LN_W2 2, 256, 2, 4
#endif
#ifndef LN_W2_RING
#define LN_W2_RING 64
#endif
#ifndef LN_W4
#define LN_W4 2, 512, 1, 2
#endif
#ifndef LN_W4_RING
#define LN_W4_RING 128
#endif
#ifndef LN_W8
#define LN_W8 2, 1024, 1, 1
#endif
#ifndef LN_W8_RING
#define LN_W8_RING 64
#endif

template <bool F16>
cudaError_t ln_fwd_dispatch(const LnFwdArgs& a, cudaStream_t st) {
    const int NV = a.D / 8;
    if (NV <= 1) return LN_FNARROW(1);
    if (NV <= 2) return LN_FNARROW(2);
    if (NV <= 4) return LN_FNARROW(4);
    if (NV <= 8) return LN_FNARROW(8);
    if (NV <= 16) return LN_FNARROW(16);
    if (NV <= 32) return LN_FNARROW(32);
    if (NV <= 64) return rows_fwd<F16, 32, LN_F2>(a, st);
    if (NV <= 128) return rows_fwd<F16, 32, LN_F4>(a, st);
    if (NV <= 256) return rows_fwd<F16, 32, LN_F8>(a, st);
    if (NV <= 512) return wide_fwd<F16, LN_W2>(a, LN_W2_RING * 1024, st);
    if (NV <= 1024) return wide_fwd<F16, LN_W4>(a, LN_W4_RING * 1024, st);
    return wide_fwd<F16, LN_W8>(a, LN_W8_RING * 1024, st);
}

template <bool F16, int G, int V, int NR, int S, int MINB, bool BIAS>
cudaError_t rows_bwd(const LnBwdArgs& a, unsigned grid, cudaStream_t st) {
    const int smem = std::max(S * NR * 2 * V * kLnRowThreads * 16, kLnRowThreads / G * a.D * 4);
    const auto kern = ln_rows_bwd_kernel<F16, G, V, NR, S, MINB, BIAS>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, grid, kLnRowThreads, smem, st, a);
}

template <bool F16, int VPT, int MAXT, int MINB, int R, bool BIAS, bool SW>
cudaError_t wide_bwd(const LnBwdArgs& a, unsigned grid, size_t ring, cudaStream_t st) {
    const int NV = a.D / 8;
    const int threads = ((NV + VPT - 1) / VPT + 31) / 32 * 32;
    const size_t stage = static_cast<size_t>(2) * R * a.D * 2;
    const size_t fixed = 4 * R * (MAXT / 32) * 4 + 8 * static_cast<size_t>(a.chunk) + 16 + (SW ? static_cast<size_t>(a.D) * 4 : 0);
    const int S = static_cast<int>(std::min<size_t>(std::max<size_t>(ring / stage, 2), 16));
    const size_t smem = S * (stage + 8) + fixed;
    if (smem > kLnMaxSmem) return cudaErrorInvalidConfiguration;
    const auto kern = ln_wide_bwd_kernel<F16, VPT, MAXT, MINB, R, BIAS, SW>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, grid, threads, smem, st, a, S);
}

template <bool F16, bool BIAS>
cudaError_t ln_bwd_dispatch(const LnBwdArgs& a, unsigned grid, cudaStream_t st) {
    const int NV = a.D / 8;
    if (NV <= 1) return rows_bwd<F16, 1, LN_B1, BIAS>(a, grid, st);
    if (NV <= 2) return rows_bwd<F16, 2, LN_B1, BIAS>(a, grid, st);
    if (NV <= 4) return rows_bwd<F16, 4, LN_B1, BIAS>(a, grid, st);
    if (NV <= 8) return rows_bwd<F16, 8, LN_B1, BIAS>(a, grid, st);
    if (NV <= 16) return rows_bwd<F16, 16, LN_B1, BIAS>(a, grid, st);
    if (NV <= 32) return rows_bwd<F16, 32, LN_B1, BIAS>(a, grid, st);
    if (NV <= 64) return rows_bwd<F16, 32, LN_B2, BIAS>(a, grid, st);
    const size_t ring = LN_BW_RING * 1024 / ln_shape(a.D).per_sm;
    if (NV <= 256) return wide_bwd<F16, LN_BW1, BIAS, false>(a, grid, ring, st);
    if (NV <= 512) return wide_bwd<F16, LN_BW2, BIAS, false>(a, grid, ring, st);
    if (NV <= 1024) return wide_bwd<F16, LN_BW4, BIAS, false>(a, grid, ring, st);
    return wide_bwd<F16, 4, 512, 1, 1, BIAS, true>(a, grid, 128 * 1024, st);
}

}  // namespace
}  // namespace rmsn
