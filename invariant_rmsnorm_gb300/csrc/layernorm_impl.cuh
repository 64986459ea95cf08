// LayerNorm kernels and their launchers, included by the translation units that
// instantiate them (layernorm.cu: bf16 activations; layernorm_f16.cu: fp16).
//
// Mathematics, per row: mu = sum x / D; var = sum (x - mu)^2 / D, from the
// deviations themselves, so a mean far from zero cancels nothing;
// y = ((x - mu) r) w + b. Backward, with c = x - mu and gw = g w:
//   dx = r gw - r c1 - c (r^2 c2'),  c1 = sum gw / D,  c2' = r sum(gw c) / D
// (n = c r is never formed there), dw = sum_t g (c r), db = sum_t g.
//
// All kernels are bound by HBM: 4 D bytes a row forward, 6 D backward. Three forms:
//   * Groups (rows of up to 512 values, backward 1016): a group of G lanes, at most
//     a warp, holds a row, up to four vectors of 8 values a lane, fed by rings of
//     asynchronous copies that each lane keeps for itself. Sums are butterflies in
//     the group; no barrier.
//   * Teams (forward, wider rows): 1 to 8 warps a row, up to 8 vectors a thread in
//     registers. A row's two sums meet at its team's own barrier.
//   * CTA rows (backward, wider rows): a CTA, or a team of its warps, a row from a
//     ring of bulk (TMA) copies; thread t owns the 16-byte vectors t, t + NT, ... and
//     their columns' weight gradients; warps' sums are added in warp order after one
//     barrier, which also tells thread 0 that the stage is read, so it refills it:
//     there is no producer warp, and 512 threads keep 128 registers each (a 17th warp
//     would cut them to 96).
// Either way a row's tree depends on D alone. The arithmetic is issued in pairs
// (f32x2): at one operation a value the group kernels spent 19 issue slots a value
// and stood at 64 % of the copy rate at D = 128. Weight gradients are summed by the
// threads that own the columns, one partial row a CTA; pass 2 is reduce_columns.cu.
#pragma once

#include <algorithm>

#include "f32x2.cuh"
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

__device__ __forceinline__ Oct ln_bias(const float* b, int v) { return b != nullptr ? load_oct(b + 8 * v) : oct_zero(); }

__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }

// s / D through the fp32 reciprocal of D, its remainder taken back once (the last
// step of Markstein's division): the correctly rounded quotient, so the mean of a
// constant row is that constant, in three instructions in a division's place. His
// theorem asks for a first quotient within one step, which s times the reciprocal
// need not be; compared with the division over every significand of s and every D
// that the calls take, it is right in all 8.6e9 cases (without the correction in
// 73 %). An infinite sum stays infinite.
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

// w_eff and b of a row in shared memory as [w low | w high | b low | b high][NV]
// float4 (the halves of a vector's eight): conflict-free reads.
__device__ __forceinline__ void stage_weights(float4* wb, const float* w, const float* b, int zc, int NV) {
    for (int v = threadIdx.x; v < NV; v += blockDim.x) {
        const Oct x = oct_weights(w, zc, v);
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

// Every lane keeps its own ring of S turns in flight: it copies its vectors to
// its own slots of shared memory (cp.async, past L1) and reads them back itself,
// so a wait for its own copies is all the synchronisation there is, and data in
// flight costs no registers. Slot layout [turn][vector][thread]: conflict-free.
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
            w1 = oct_weights(a.w, a.zc, l);
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
// HOLD (three or four vectors a lane, whose weight gradients take 48 or 64
// registers): the weights lie in shared memory, and after the row's sums g and x
// are read again from the lane's slots, which are refilled a turn later.
template <bool F16, int G, int V, int NR, int S, int MINB, bool HOLD, bool BIAS>
__global__ void __launch_bounds__(kLnRowThreads, MINB) ln_rows_bwd_kernel(const LnBwdArgs a) {
    constexpr int P = kLnRowThreads / G;
    extern __shared__ __align__(16) uint4 ring[];  // [S][NR][g | x][V][threads], HOLD: the weights; at the end [P][D] sums
    float4* wb = reinterpret_cast<float4*>(ring + S * NR * 2 * V * kLnRowThreads);
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
        if (!HOLD && k * G + l < NV) w[k] = oct_weights(a.w, a.zc, k * G + l);
    }
    if constexpr (HOLD) {
        stage_weights(wb, a.w, nullptr, a.zc, NV);
        __syncthreads();
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
                        oct_grad<BIAS>(g[i][k], c[i][k], HOLD ? staged_weights(wb, NV, k * G + l) : w[k], mu[i], r[i], p1, p2, aw[k], ab[k]);
                    }
                }
            }
            s1[i] = fadd(p1.x, p1.y);
            s2[i] = fadd(p2.x, p2.y);
        }
        if constexpr (!HOLD) fetch(at + (S - 1) * P * NR, s == 0 ? S - 1 : s - 1);
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
                    if (k * G + l < NV) {
                        if constexpr (HOLD) {
                            const Oct wv = staged_weights(wb, NV, k * G + l);
                            g[i][k] = oct_unpack<F16>(*slot(s, i, 0, k));
                            c[i][k] = oct_unpack<F16>(*slot(s, i, 1, k));
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                g[i][k].p[e] = fmul2(g[i][k].p[e], wv.p[e]);
                                c[i][k].p[e] = fadd2(c[i][k].p[e], both(-mu[i]));
                            }
                        }
                        st_global_cs(a.dx + (c0 + rel) * a.lddx + 8 * (k * G + l),
                                     oct_pack<F16>(oct_dx(g[i][k], c[i][k], r[i], m, rc1)));
                    }
            }
        }
        if constexpr (HOLD) fetch(at + (S - 1) * P * NR, s == 0 ? S - 1 : s - 1);
        if (++s == S) s = 0;
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
// A CTA, or a team of its warps, a row
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

// Places for the warps' totals of one value: whole float4s.
__host__ __device__ constexpr int warp_places(int threads) { return (threads / 32 + 3) / 4 * 4; }

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

// Forward: a team of TW warps a row, V vectors a thread, in registers; the CTA's
// teams take rows of their own and share the weights in shared memory. A row's
// two sums meet at the team's own named barrier, so one team's wait is another's
// work. PRE: the next row's loads are issued as soon as this row is unpacked and
// stay in registers until its turn.
template <int TW>
__device__ __forceinline__ float team_sum(float v, float* red, int warp, int lane, int bar) {
    v = group_sum<32>(v);
    if constexpr (TW > 1) {
        if (lane == 0) red[warp] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(TW * 32) : "memory");
        v = red[0];
#pragma unroll
        for (int i = 1; i < TW; ++i) v = fadd(v, red[i]);
    }
    return v;
}

template <bool F16, int TW, int V, bool PRE, int THREADS, int MINB>
__global__ void __launch_bounds__(THREADS, MINB) ln_team_fwd_kernel(const LnFwdArgs a) {
    constexpr int NT = TW * 32, TEAMS = THREADS / NT;
    extern __shared__ __align__(16) float4 wb[];  // the weights, then the teams' sums
    const int NV = a.D >> 3;
    const int team = threadIdx.x / NT, t = threadIdx.x % NT, lane = t & 31, warp = t >> 5;
    const bool bias = a.b != nullptr;
    float* red = reinterpret_cast<float*>(wb + (bias ? 4 : 2) * NV) + team * 2 * TW;  // [teams][2][TW]
    pdl_wait();
    const int64_t step = static_cast<int64_t>(gridDim.x) * TEAMS;
    int64_t row = static_cast<int64_t>(blockIdx.x) * TEAMS + team;
    uint4 xv[V];
    auto load = [&](int64_t at) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            xv[k] = make_uint4(0, 0, 0, 0);  // zeros beyond the row
            if (k * NT + t < NV && at < a.T) xv[k] = ld_stream(a.x + at * a.ldx + 8 * (k * NT + t));
        }
    };
    if constexpr (PRE) load(row);
    stage_weights(wb, a.w, a.b, a.zc, NV);
    __syncthreads();
    const float d = static_cast<float>(a.D);
    for (; row < a.T; row += step) {
        Oct c[V];
        if constexpr (!PRE) load(row);
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            c[k] = oct_unpack<F16>(xv[k]);
            sum = oct_sum(sum, c[k]);
        }
        if constexpr (PRE) load(row + step);
        const float mu = over_d(team_sum<TW>(fadd(sum.x, sum.y), red, warp, lane, team + 1), d, a.rcp_d);
        float2 q = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k * NT + t < NV) q = oct_centre(c[k], mu, q);
        const float r = rsqrtf(fadd(fmul(team_sum<TW>(fadd(q.x, q.y), red + TW, warp, lane, team + 1), a.rcp_d), a.eps));
        if (t == 0) {
            a.mean[row] = mu;
            a.rstd[row] = r;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int v = k * NT + t;
            if (v < NV)
                st_global_cs(a.y + row * a.ldy + 8 * v,
                             oct_pack<F16>(oct_affine(c[k], r, staged_weights(wb, NV, v), staged_bias(wb, bias, NV, v))));
        }
    }
    pdl_release();
}

// The teams' predicate, true for all of a team's threads if it is for each.
template <bool TEAMS>
__device__ __forceinline__ bool team_and(bool ok, int bar, int threads) {
    if constexpr (!TEAMS) return __syncthreads_and(ok ? 1 : 0);
    int all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 q, %1, 0;\n\tbarrier.cta.red.and.pred p, %2, %3, q;\n\tselp.s32 %0, 1, 0, p;\n\t}"
        : "=r"(all) : "r"(ok ? 1 : 0), "r"(bar), "r"(threads) : "memory");
    return all != 0;
}

// Backward: one CTA a chunk of rows. Stage: [g | x][D] 16-bit. Between the two
// halves of a row its c and g w stay in registers; SW (the widest rows, whose
// weight gradients take 48 or 64 registers): the packed g and x stay instead, and
// the weights lie in shared memory. TEAMS: several teams of nt threads a CTA, each
// with a ring and a barrier of its own, take every so many-th row; their weight
// gradients are added in team order at the end, so that narrow rows leave a partial
// row a CTA and not one a few warps.
template <bool F16, int VPT, int MAXT, int THREADS, int MINB, bool BIAS, bool SW, bool TEAMS>
__global__ void __launch_bounds__(THREADS, MINB) ln_wide_bwd_kernel(const LnBwdArgs a, const int S, const int team_threads) {
    constexpr int NW = warp_places(MAXT);
    extern __shared__ __align__(128) unsigned char smem[];
    const int nt = TEAMS ? team_threads : blockDim.x, teams = TEAMS ? blockDim.x / nt : 1;
    const int team = TEAMS ? threadIdx.x / nt : 0, tid = threadIdx.x - team * nt;
    const int NV = a.D >> 3, lane = tid & 31, warp = tid >> 5;
    const uint32_t row_bytes = static_cast<uint32_t>(a.D) * 2u;
    const uint32_t stage_bytes = 2 * row_bytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(teams) * S * stage_bytes);
    uint64_t* full = bars + team * S;
    float* reds = reinterpret_cast<float*>(bars + ((teams * S + 1) & ~1));  // [teams][2][2][NW]
    float* red = reds + team * 4 * NW;
    unsigned char* ring = smem + static_cast<size_t>(team) * S * stage_bytes;
    float4* wb = reinterpret_cast<float4*>(reds + teams * 4 * NW);     // SW: the weights
    float2* stat = reinterpret_cast<float2*>(wb + (SW ? 2 * NV : 0));  // [chunk]: mean, rstd
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
    const int n_rows = static_cast<int>(min(static_cast<int64_t>(a.chunk), a.T - row0));
    const int n_my = TEAMS ? (n_rows - team + teams - 1) / teams : n_rows;  // rows team, team + teams, ... of the chunk
    if (tid == 0) {
        for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
        fence_mbar_init();
    }
    for (int i = tid; i < 4 * NW; i += nt) red[i] = 0.0f;
    __syncthreads();
    pdl_wait();

    const uint64_t pol = policy_evict_first();
    auto issue = [&](int i) {
        const int s = i % S;
        unsigned char* dst = ring + static_cast<size_t>(s) * stage_bytes;
        const int64_t row = row0 + i * teams + team;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        bulk_g2s(dst, a.g + row * a.ldg, row_bytes, &full[s], pol);
        bulk_g2s(dst + row_bytes, a.x + row * a.ldx, row_bytes, &full[s], pol);
    };
    if (tid == 0)
        for (int i = 0; i < min(S, n_my); ++i) issue(i);
    for (int i = threadIdx.x; i < n_rows; i += blockDim.x) stat[i] = make_float2(__ldg(a.mean + row0 + i), __ldg(a.rstd + row0 + i));
    Oct w[VPT], aw[VPT], ab[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        w[j] = aw[j] = ab[j] = oct_zero();
        if (!SW && j * nt + tid < NV) w[j] = oct_weights(a.w, a.zc, j * nt + tid);
    }
    if constexpr (SW) stage_weights(wb, a.w, nullptr, a.zc, NV);
    __syncthreads();

    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < n_my; ++i) {
        const bool ok = mbar_wait(&full[s], ph);
        const unsigned char* st = ring + static_cast<size_t>(s) * stage_bytes;
        const float2 mr = stat[i * teams + team];
        Oct g[VPT], c[VPT];  // g w and x - mu
        uint4 gv[VPT], xv[VPT];
        float2 p1 = make_float2(0.0f, 0.0f), p2 = p1;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = j * nt + tid;
            if (v < NV) {
                gv[j] = ld_shared_v4(st + 16 * v);
                xv[j] = ld_shared_v4(st + row_bytes + 16 * v);
                g[j] = oct_unpack<F16>(gv[j]);
                c[j] = oct_unpack<F16>(xv[j]);
                oct_grad<BIAS>(g[j], c[j], SW ? staged_weights(wb, NV, v) : w[j], mr.x, mr.y, p1, p2, aw[j], ab[j]);
            }
        }
        float* rb = red + (i & 1) * 2 * NW;
        {
            float sum[2] = {fadd(p1.x, p1.y), fadd(p2.x, p2.y)};
            const float t = warp_sums<2>(sum, lane);
            if ((lane & 15) == 0) rb[(lane >> 4) * NW + warp] = t;
        }
        if (!team_and<TEAMS>(ok, team + 1, nt)) {
            if (tid == 0) ln_abort(full, S, i, min(i + S, n_my) - 1);
            break;
        }
        if (tid == 0 && i + S < n_my) {  // every thread has the stage in registers
            fence_proxy_async_smem();
            issue(i + S);
        }
        if (++s == S) {
            s = 0;
            ph ^= 1u;
        }
        const float rc1 = fmul(mr.y, fmul(warps_total<NW>(rb), a.rcp_d));
        const float m = -fmul(fmul(mr.y, mr.y), fmul(fmul(warps_total<NW>(rb + NW), mr.y), a.rcp_d));
        uint16_t* dx = a.dx + (row0 + i * teams + team) * a.lddx;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = j * nt + tid;
            if (v < NV) {
                if constexpr (SW) {
                    const Oct wv = staged_weights(wb, NV, v);
                    g[j] = oct_unpack<F16>(gv[j]);
                    c[j] = oct_unpack<F16>(xv[j]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        g[j].p[e] = fmul2(g[j].p[e], wv.p[e]);
                        c[j].p[e] = fadd2(c[j].p[e], both(-mr.x));
                    }
                }
                st_global_cs(dx + 8 * v, oct_pack<F16>(oct_dx(g[j], c[j], mr.y, m, rc1)));
            }
        }
    }
    // The chunk's partial rows, read again by pass 2 at once: kept in L2.
    const uint64_t keep = policy_evict_last();
    float* pw = a.partials + static_cast<int64_t>(blockIdx.x) * a.D;
    float* pb = pw + static_cast<int64_t>(gridDim.x) * a.D;
    if constexpr (TEAMS) {  // the teams' sums in team order, dw, then db through the rings' memory
        float* comb = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int part = 0; part < (BIAS ? 2 : 1); ++part) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = j * nt + tid;
                if (v < NV) {
                    float4* o = reinterpret_cast<float4*>(comb + team * a.D + 8 * v);
                    const Oct& t = part ? ab[j] : aw[j];
                    o[0] = make_float4(t.p[0].x, t.p[0].y, t.p[1].x, t.p[1].y);
                    o[1] = make_float4(t.p[2].x, t.p[2].y, t.p[3].x, t.p[3].y);
                }
            }
            __syncthreads();
            for (int q = threadIdx.x; q < a.D / 4; q += blockDim.x) {
                float4 t = reinterpret_cast<const float4*>(comb)[q];
                for (int m = 1; m < teams; ++m) {
                    const float4 u = reinterpret_cast<const float4*>(comb + m * a.D)[q];
                    t = make_float4(fadd(t.x, u.x), fadd(t.y, u.y), fadd(t.z, u.z), fadd(t.w, u.w));
                }
                st_global_f4_hint((part ? pb : pw) + 4 * q, t.x, t.y, t.z, t.w, keep);
            }
        }
        pdl_release();
        return;
    }
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

template <bool F16, int TW, int V, bool PRE, int THREADS, int MINB>
cudaError_t team_fwd(const LnFwdArgs& a, cudaStream_t st) {
    constexpr int teams = THREADS / (TW * 32);
    const int smem = a.D * (a.b != nullptr ? 8 : 4) + teams * 2 * TW * 4;
    const auto kern = ln_team_fwd_kernel<F16, TW, V, PRE, THREADS, MINB>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    const int occ = ctas_per_sm(reinterpret_cast<const void*>(kern), THREADS, smem);
    if (occ < 1) return cudaErrorInvalidConfiguration;
    const int64_t grid = std::min<int64_t>((a.T + teams - 1) / teams, static_cast<int64_t>(sm_count()) * occ);
    return launch_kernel(kern, static_cast<unsigned>(grid), THREADS, smem, st, a);
}

// lanes, vectors a lane, rows a turn, turns in flight, CTAs an SM
// Shapes by width, each the fastest measured: as many vectors a lane as its
// registers hold (fewer lanes a row: fewer shuffles, more loads in flight a lane),
// in steps that leave few lanes idle. Of the copy rate at 256 MB a tensor: D = 128
// 85 % (at 64 MB 90 %, with 16 lanes of one vector 76 %), 2048 95 %, 4096 93 %,
// 5000 92 %, 8192 91 %, 16384 91 %. Rows of 8 vectors a lane on one or two warps
// do without PRE (2048: 95 against 89 %): 16 warps of 4 KB are in flight as it is.
template <bool F16>
cudaError_t ln_fwd_dispatch(const LnFwdArgs& a, cudaStream_t st) {
    const int NV = a.D / 8;
    if (NV <= 1) return rows_fwd<F16, 1, 1, 2, 4, 4>(a, st);
    if (NV <= 2) return rows_fwd<F16, 1, 2, 2, 3, 3>(a, st);
    if (NV <= 4) return rows_fwd<F16, 2, 2, 2, 3, 3>(a, st);
    if (NV <= 8) return rows_fwd<F16, 4, 2, 2, 3, 3>(a, st);
    if (NV <= 12) return rows_fwd<F16, 4, 3, 1, 3, 3>(a, st);
    if (NV <= 16) return rows_fwd<F16, 4, 4, 1, 3, 3>(a, st);
    if (NV <= 24) return rows_fwd<F16, 8, 3, 1, 3, 3>(a, st);
    if (NV <= 32) return rows_fwd<F16, 8, 4, 1, 3, 3>(a, st);
    if (NV <= 48) return rows_fwd<F16, 16, 3, 1, 3, 3>(a, st);
    if (NV <= 64) return rows_fwd<F16, 16, 4, 1, 3, 3>(a, st);
    if (NV <= 96) return team_fwd<F16, 1, 3, true, 256, 3>(a, st);
    if (NV <= 128) return team_fwd<F16, 1, 4, true, 256, 3>(a, st);
    if (NV <= 160) return team_fwd<F16, 1, 5, true, 256, 2>(a, st);
    if (NV <= 192) return team_fwd<F16, 1, 6, true, 256, 2>(a, st);
    if (NV <= 224) return team_fwd<F16, 1, 7, true, 256, 2>(a, st);
    if (NV <= 256) return team_fwd<F16, 1, 8, false, 256, 2>(a, st);
    if (NV <= 320) return team_fwd<F16, 2, 5, true, 256, 2>(a, st);
    if (NV <= 384) return team_fwd<F16, 2, 6, true, 256, 2>(a, st);
    if (NV <= 448) return team_fwd<F16, 2, 7, true, 256, 2>(a, st);
    if (NV <= 512) return team_fwd<F16, 2, 8, false, 256, 2>(a, st);
    if (NV <= 640) return team_fwd<F16, 4, 5, true, 512, 1>(a, st);
    if (NV <= 768) return team_fwd<F16, 4, 6, true, 512, 1>(a, st);
    if (NV <= 896) return team_fwd<F16, 4, 7, true, 512, 1>(a, st);
    if (NV <= 1024) return team_fwd<F16, 4, 8, true, 512, 1>(a, st);
    if (NV <= 1280) return team_fwd<F16, 8, 5, true, 512, 1>(a, st);
    if (NV <= 1536) return team_fwd<F16, 8, 6, true, 512, 1>(a, st);
    if (NV <= 1792) return team_fwd<F16, 8, 7, true, 512, 1>(a, st);
    return team_fwd<F16, 8, 8, true, 512, 1>(a, st);
}

template <bool F16, int G, int V, int NR, int S, int MINB, bool HOLD, bool BIAS>
cudaError_t rows_bwd(const LnBwdArgs& a, unsigned grid, cudaStream_t st) {
    const int smem = std::max(S * NR * 2 * V * kLnRowThreads * 16 + (HOLD ? a.D * 4 : 0), kLnRowThreads / G * a.D * 4);
    const auto kern = ln_rows_bwd_kernel<F16, G, V, NR, S, MINB, HOLD, BIAS>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, grid, kLnRowThreads, smem, st, a);
}

// The ring's stages: as many as bring the copies in flight on an SM (of all its
// CTAs and teams) to 88 KB. More measured slower as well as fewer (32768 x 4096,
// two rows at a time with three stages of 16 KB each 95 % of the copy rate, with
// four 87 %, with two 89 %; 16384 x 8192, one CTA: three of 32 KB 93 %, four 92 %, two 82 %).
constexpr size_t kLnBwdInFlight = 88 * 1024;

template <bool F16, int VPT, int MAXT, int THREADS, int MINB, bool BIAS, bool SW>
cudaError_t wide_bwd(const LnBwdArgs& a, unsigned grid, cudaStream_t st) {
    constexpr bool TEAMS = THREADS > MAXT;
    const int NV = a.D / 8;
    const LnShape shape = ln_shape(a.D);
    const int teams = TEAMS ? static_cast<int>(shape.step) : 1;
    const int threads = ((NV + VPT - 1) / VPT + 31) / 32 * 32;
    const size_t stage = static_cast<size_t>(4) * a.D;
    const size_t fixed = teams * 4 * warp_places(MAXT) * 4 + 8 * static_cast<size_t>(a.chunk) + 16 + (SW ? static_cast<size_t>(a.D) * 4 : 0);
    const size_t all = stage * shape.per_sm * teams;
    const int S = std::max(2, static_cast<int>((kLnBwdInFlight + all - 1) / all));
    const size_t smem = teams * S * (stage + 8) + fixed;
    if (smem > kLnMaxSmem || threads > MAXT || teams * threads > THREADS) return cudaErrorInvalidConfiguration;
    const auto kern = ln_wide_bwd_kernel<F16, VPT, MAXT, THREADS, MINB, BIAS, SW, TEAMS>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, grid, teams * threads, smem, st, a, S, threads);
}

// Shapes by width, each the fastest measured (ln_shape has their CTAs an SM). Of
// the copy rate, both passes, 65536 to 8192 rows: D = 768 87 % (a CTA a row: 80),
// 1024 91, 2048 97, 4096 97, 5000 91, 8192 96, 16384 92; 2^20 rows of 128 or 2^21
// of 64 96, 262144 of them 82 and 71. (4104 to 5120 without a bias spill 8 bytes at
// the 96 registers that two CTAs leave them.)
// Up to 4096 several teams a CTA leave 152 partial rows: a CTA a row, as many warps
// an SM and 304 to 1216 partial rows, 88, 92 and 96 %.
template <bool F16, bool BIAS>
cudaError_t ln_bwd_dispatch(const LnBwdArgs& a, unsigned grid, cudaStream_t st) {
    const int NV = a.D / 8;
    if (NV <= 1) return rows_bwd<F16, 1, 1, 1, 4, 2, false, BIAS>(a, grid, st);
    if (NV <= 2) return rows_bwd<F16, 1, 2, 1, 3, 2, false, BIAS>(a, grid, st);
    if (NV <= 4) return rows_bwd<F16, 2, 2, 1, 3, 2, false, BIAS>(a, grid, st);
    if (NV <= 8) return rows_bwd<F16, 4, 2, 1, 3, 2, false, BIAS>(a, grid, st);
    if (NV <= 12) return rows_bwd<F16, 4, 3, 1, 3, 2, true, BIAS>(a, grid, st);
    if (NV <= 16) return rows_bwd<F16, 8, 2, 1, 3, 2, false, BIAS>(a, grid, st);
    if (NV <= 24) return rows_bwd<F16, 8, 3, 1, 3, 2, true, BIAS>(a, grid, st);
    if (NV <= 32) return rows_bwd<F16, 16, 2, 1, 3, 2, false, BIAS>(a, grid, st);
    if (NV <= 48) return rows_bwd<F16, 16, 3, 1, 3, 2, true, BIAS>(a, grid, st);
    if (NV <= 64) return rows_bwd<F16, 32, 2, 1, 3, 2, false, BIAS>(a, grid, st);
    if (NV <= 96) return rows_bwd<F16, 32, 3, 1, 3, 2, true, BIAS>(a, grid, st);
    if (NV < kLnCtaRowFrom) return rows_bwd<F16, 32, 4, 1, 3, 2, true, BIAS>(a, grid, st);
    if (NV <= kLnTeamsTo) return wide_bwd<F16, 2, 256, 512, 1, BIAS, false>(a, grid, st);
    if (NV <= 640) return wide_bwd<F16, 2, 320, 320, 2, BIAS, false>(a, grid, st);
    if (NV <= 768) return wide_bwd<F16, 2, 384, 384, 1, BIAS, false>(a, grid, st);
    if (NV <= 1024) return wide_bwd<F16, 2, 512, 512, 1, BIAS, false>(a, grid, st);
    if (NV <= 1536) return wide_bwd<F16, 3, 512, 512, 1, BIAS, true>(a, grid, st);
    return wide_bwd<F16, 4, 512, 512, 1, BIAS, true>(a, grid, st);
}

}  // namespace
}  // namespace rmsn
