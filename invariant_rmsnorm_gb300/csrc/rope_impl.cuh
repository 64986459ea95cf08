// Rotary positions and the head norm fused with them: kernels and launchers,
// included by the translation units that instantiate them (rope.cu: bf16
// activations; rope_f16.cu: fp16).
//
// Mathematics, per pair (u, v) of a head and its angle a:
//   turn:            (u c - v s, v c + u s), c = scale cos a, s = scale sin a
//   norm + turn:     r = rsqrt(sum x^2 / D + eps), the turn of (x r) w
//   its backward:    g' = turn of g by -a; gw = g' w;
//                    dx = r gw - x (r^3 / D) sum(gw x);  dw = sum g' (x r)
// The kernels are bound by HBM: 4 D bytes a head forward, 6 D backward; the
// angles (rope_math.cuh) are computed once a token by the warp that has it, a few
// percent of its work.
//
// A warp takes a turn of 32 / G heads of one token at a time, G lanes a head. The
// turns of a launch are split among its warps in contiguous ranges, so a warp
// computes a token's cosines once for all its heads, in its own part of shared
// memory. Every warp keeps a ring of S turns in flight through asynchronous
// copies. Warps never wait for one another; dw is summed in registers and
// joined over the CTA's groups at the end, in group order, one partial row a CTA.
//
// Two kernels, by how pairs lie in 16-byte vectors:
//   * units: each lane holds whole vectors whose pairs are complete (a vector and
//     its partner R/2 values on, or a vector of neighbours), copied and read back
//     by the lane itself. ROPE_HALF with R a multiple of 16, ROPE_INTERLEAVED.
//   * pairs: any other R of ROPE_HALF. A head is copied vector by vector to
//     shared memory and read value by value, lane by lane in order.
#pragma once

#include <algorithm>

#include "f32x2.cuh"
#include "kernels.h"
#include "rope_launch.h"
#include "rope_math.cuh"

namespace rmsn {
namespace {

template <bool F16>
__device__ __forceinline__ float widen(uint16_t v) {
    return F16 ? __half2float(__ushort_as_half(v)) : __uint_as_float(static_cast<uint32_t>(v) << 16);
}
template <bool F16>
__device__ __forceinline__ uint16_t narrow(float v) {
    return F16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

__device__ __forceinline__ long long position(const RopeArgs& a, int64_t t) {
    if (a.pos == nullptr) return t;
    return a.pos64 ? static_cast<const long long*>(a.pos)[t] : static_cast<const int*>(a.pos)[t];
}

// A warp's contiguous range of the turns (t, b): token t, b-th turn of its heads,
// q's first, then k's (a turn has heads of one of them only, so all that depends on
// which is the same for the whole warp). (A warp's own turns fit an int: 2^31 of
// them would be 2^35 bytes a warp.)
struct Turns {
    int left, t, b, nb, nq;
    __device__ __forceinline__ Turns(int64_t T, int nb_, int nq_, int64_t warp, int64_t warps) : nb(nb_), nq(nq_) {
        const int64_t all = T * nb, first = all * warp / warps;
        left = static_cast<int>(all * (warp + 1) / warps - first);
        t = static_cast<int>(first / nb);
        b = static_cast<int>(first - static_cast<int64_t>(t) * nb);
    }
    __device__ __forceinline__ void next() {
        --left;
        if (++b == nb) {
            b = 0;
            ++t;
        }
    }
    __device__ __forceinline__ int tensor() const { return b >= nq; }
    __device__ __forceinline__ int turn_of_tensor() const { return b >= nq ? b - nq : b; }
};

__device__ __forceinline__ float lanes_sum(float v, int G) {  // over aligned groups of G lanes
    for (int o = G >> 1; o > 0; o >>= 1) v = fadd(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// scale (cos, sin) of every pair of a token, by its warp: [cos | sin][hp]
// floats. Backward: of minus the angle.
__device__ __forceinline__ void token_angles(float* cs, int hp, int half, const unsigned long long* F, long long p, float scale,
                                             bool back, int lane) {
    __syncwarp();  // the token before is done with
    for (int i = lane; i < half; i += 32) {
        const float2 c = rope_cos_sin(p, F[i], scale);
        cs[i] = c.x;
        cs[hp + i] = back ? -c.y : c.y;
    }
    __syncwarp();
}

__device__ __forceinline__ Oct oct_at(const float* p) {
    const float4* q = reinterpret_cast<const float4*>(p);
    return oct_of(q[0], q[1]);
}

// (A, B) turned, pair by pair: halves.
__device__ __forceinline__ void turn_halves(Oct& A, Oct& B, const Oct& c, const Oct& s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = A.p[i], v = B.p[i];
        const float2 uc = fmul2(u, c.p[i]);
        A.p[i] = make_float2(__fmaf_rn(-v.x, s.p[i].x, uc.x), __fmaf_rn(-v.y, s.p[i].y, uc.y));
        B.p[i] = fma2(u, s.p[i], fmul2(v, c.p[i]));
    }
}
// The first n of A's neighbours turned (n may pass 4).
__device__ __forceinline__ void turn_neighbours(Oct& A, const float4 c, const float4 s, int n) {
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
    const Oct was = A;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = A.p[i], uc = fmul2(u, both(cc[i]));
        A.p[i] = make_float2(__fmaf_rn(-u.y, ss[i], uc.x), __fmaf_rn(u.x, ss[i], uc.y));
    }
    if (n < 4) {
#pragma unroll
        for (int i = 1; i < 4; ++i)
            if (i >= n) A.p[i] = was.p[i];
    }
}

// ---------------------------------------------------------------------------
// Units: NU of two vectors a lane
// ---------------------------------------------------------------------------
template <int MODE, bool INTER, bool F16, int NU, int S, int MINB>
__global__ void __launch_bounds__(kRopeThreads, MINB) rope_units_kernel(const RopeArgs a, const int lgG) {
    constexpr bool NORM = MODE != kTurn, BWD = MODE == kNormTurnBwd;
    constexpr int OPS = BWD ? 2 : 1;
    extern __shared__ __align__(16) unsigned char smem[];
    const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
    const int D = a.D, NC = D >> 3, half = a.R >> 1, hp = (half + 7) & ~7;
    const int G = 1 << lgG, l = lane & (G - 1), head = lane >> lgG, per = 32 >> lgG;
    uint4* ring = reinterpret_cast<uint4*>(smem);                                   // [S][OPS][2 NU][threads]
    float* ring_r = reinterpret_cast<float*>(ring + S * OPS * 2 * NU * nt);         // BWD: [S][threads]
    float4* wb = reinterpret_cast<float4*>(ring_r + (BWD ? S * nt : 0));            // NORM: [q | k][low | high][NC]
    float* cs = reinterpret_cast<float*>(wb + (NORM ? 4 * NC : 0)) + warp * 2 * hp;  // [warps][cos | sin][hp]
    unsigned long long* F = reinterpret_cast<unsigned long long*>(reinterpret_cast<float*>(wb + (NORM ? 4 * NC : 0)) + nw * 2 * hp);

    // This lane's vectors: unit u = j G + l is a vector and its partner.
    const int NP = INTER ? 0 : half >> 3;               // units of the halves
    const int rest = (NC - 2 * NP + 1) >> 1;            // other units: two vectors `rest` apart
    int c0[NU], c1[NU];
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        const int u = (j << lgG) + l;
        c0[j] = u < NP ? u : u + NP;                     // 2 NP + (u - NP)
        c1[j] = u < NP ? u + NP : c0[j] + rest;
        if (u >= NP + rest) c0[j] = NC;                  // none
        if (c1[j] >= NC) c1[j] = NC;
    }
    pdl_wait();
    for (int i = tid; i < half; i += nt) F[i] = rope_turns(a.inv_freq[i]);
    if constexpr (NORM) {
        for (int i = tid; i < 2 * NC; i += nt) {
            const int s = i >= NC, v = s ? i - NC : i;
            if (a.H[s] > 0) {
                const Oct w = oct_weights(a.w[s], a.zc, v);
                wb[2 * s * NC + v] = make_float4(w.p[0].x, w.p[0].y, w.p[1].x, w.p[1].y);
                wb[(2 * s + 1) * NC + v] = make_float4(w.p[2].x, w.p[2].y, w.p[3].x, w.p[3].y);
            }
        }
    }
    __syncthreads();

    auto slot = [&](int s, int op, int k) { return ring + ((s * OPS + op) * 2 * NU + k) * nt + tid; };
    // Forward: one pass over the turns of q and of k. Backward: q, then k, each with its own weight gradient.
    for (int pass = 0; pass < (BWD ? 2 : 1); ++pass) {
        const int nq = (a.H[0] + per - 1) >> (5 - lgG), nk = (a.H[1] + per - 1) >> (5 - lgG);
        const int nb = BWD ? (pass ? nk : nq) : nq + nk;
        if (nb == 0) continue;
        Turns now(a.T, nb, BWD && pass ? 0 : nq, static_cast<int64_t>(blockIdx.x) * nw + warp, static_cast<int64_t>(gridDim.x) * nw);
        Turns ahead = now;
        int fs = 0;
        auto fetch = [&]() {
            if (ahead.left > 0) {
                const int s = ahead.tensor(), h = ahead.turn_of_tensor() * per + head;
                if (h < a.H[s]) {
                    const uint16_t* p = a.in[s].p + ahead.t * a.in[s].token + h * a.in[s].head;
#pragma unroll
                    for (int j = 0; j < NU; ++j) {
                        if (c0[j] < NC) cp_async16(slot(fs, 0, 2 * j), p + 8 * c0[j]);
                        if (c1[j] < NC) cp_async16(slot(fs, 0, 2 * j + 1), p + 8 * c1[j]);
                    }
                    if constexpr (BWD) {
                        const uint16_t* x = a.x[s].p + ahead.t * a.x[s].token + h * a.x[s].head;
#pragma unroll
                        for (int j = 0; j < NU; ++j) {
                            if (c0[j] < NC) cp_async16(slot(fs, 1, 2 * j), x + 8 * c0[j]);
                            if (c1[j] < NC) cp_async16(slot(fs, 1, 2 * j + 1), x + 8 * c1[j]);
                        }
                        cp_async4(ring_r + fs * nt + tid, a.rstd[s] + static_cast<int64_t>(ahead.t) * a.H[s] + h);
                    }
                }
                ahead.next();
            }
            cp_async_commit();
            fs = fs + 1 == S ? 0 : fs + 1;
        };
#pragma unroll
        for (int i = 0; i < S - 1; ++i) fetch();
        long long p_next = now.left > 0 ? position(a, now.t) : 0;
        Oct acc[NU][2];
        if constexpr (BWD) {
#pragma unroll
            for (int j = 0; j < NU; ++j) acc[j][0] = acc[j][1] = oct_zero();
        }
        int t_angles = -1;
        int cur = 0;
        while (now.left > 0) {
            if (now.t != t_angles) {
                t_angles = now.t;
                token_angles(cs, hp, half, F, p_next, a.scale, BWD || a.back, lane);
                if (t_angles + 1 < a.T) p_next = position(a, t_angles + 1);
            }
            cp_async_wait<S - 2>();
            const int s = now.tensor(), h = now.turn_of_tensor() * per + head;
            const bool have = h < a.H[s];
            const float4* ws = wb + 2 * s * NC;
            Oct o[NU][2], x[NU][2];
            uint4 raw[NU][2];
            float2 sum2 = make_float2(0.0f, 0.0f);
            float r = 0.0f;
            if constexpr (BWD) {
                if (have) r = ring_r[cur * nt + tid];
            }
            auto turn = [&](int j) {
                if constexpr (INTER) {
                    const float4* q = reinterpret_cast<const float4*>(cs);
                    if (4 * c0[j] < half) turn_neighbours(o[j][0], q[c0[j]], q[(hp >> 2) + c0[j]], half - 4 * c0[j]);
                    if (4 * c1[j] < half) turn_neighbours(o[j][1], q[c1[j]], q[(hp >> 2) + c1[j]], half - 4 * c1[j]);
                } else {
                    if (c0[j] < NP) turn_halves(o[j][0], o[j][1], oct_at(cs + 8 * c0[j]), oct_at(cs + hp + 8 * c0[j]));
                }
            };
#pragma unroll
            for (int j = 0; j < NU; ++j) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    raw[j][i] = make_uint4(0, 0, 0, 0);
                    if (have && (i ? c1[j] : c0[j]) < NC) raw[j][i] = *slot(cur, 0, 2 * j + i);
                    o[j][i] = oct_unpack<F16>(raw[j][i]);
                }
                if constexpr (BWD) {
                    turn(j);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int c = i ? c1[j] : c0[j];
                        if (have && c < NC) {
                            x[j][i] = oct_unpack<F16>(*slot(cur, 1, 2 * j + i));
                            const Oct w = oct_of(ws[c], ws[NC + c]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                acc[j][i].p[e] = fma2(o[j][i].p[e], fmul2(x[j][i].p[e], both(r)), acc[j][i].p[e]);
                                o[j][i].p[e] = fmul2(o[j][i].p[e], w.p[e]);
                                sum2 = fma2(o[j][i].p[e], x[j][i].p[e], sum2);
                            }
                        }
                    }
                } else if constexpr (NORM) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum2 = fma2(o[j][i].p[e], o[j][i].p[e], sum2);
                }
            }
            fetch();
            float coef = 0.0f;
            if constexpr (NORM) {
                const float sum = lanes_sum(fadd(sum2.x, sum2.y), G);
                if constexpr (BWD) {
                    coef = -fmul(fmul(fmul(fmul(r, r), r), a.rcp_d), sum);
                } else {
                    r = rsqrtf(fadd(fmul(sum, a.rcp_d), a.eps));
                    if (have && l == 0) a.rstd[s][static_cast<int64_t>(now.t) * a.H[s] + h] = r;
                }
            }
            if (have) {
                uint16_t* out = a.out[s].p + now.t * a.out[s].token + h * a.out[s].head;
                const bool in_place = MODE == kTurn && a.out[s].p == a.in[s].p;
#pragma unroll
                for (int j = 0; j < NU; ++j) {
                    if constexpr (BWD) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int c = i ? c1[j] : c0[j];
                            if (c < NC) {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    o[j][i].p[e] = fma2(o[j][i].p[e], both(r), fmul2(x[j][i].p[e], both(coef)));
                                st_global_cs(out + 8 * c, oct_pack<F16>(o[j][i]));
                            }
                        }
                    } else if constexpr (NORM) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int c = i ? c1[j] : c0[j];
                            if (c < NC) {
                                const Oct w = oct_of(ws[c], ws[NC + c]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[j][i].p[e] = fmul2(fmul2(o[j][i].p[e], both(r)), w.p[e]);
                            }
                        }
                        turn(j);
                        if (c0[j] < NC) st_global_cs(out + 8 * c0[j], oct_pack<F16>(o[j][0]));
                        if (c1[j] < NC) st_global_cs(out + 8 * c1[j], oct_pack<F16>(o[j][1]));
                    } else {
                        turn(j);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int c = i ? c1[j] : c0[j];
                            if (c >= NC) continue;
                            const int n = INTER ? half - 4 * c : c0[j] < NP ? 4 : 0;  // pairs of this vector that are turned
                            if (n > 0) {
                                uint4 q = oct_pack<F16>(o[j][i]);
                                if (INTER && n < 4) {  // the rest of the head keeps its bits
                                    if (n < 2) q.y = raw[j][i].y;
                                    if (n < 3) q.z = raw[j][i].z;
                                    q.w = raw[j][i].w;
                                }
                                st_global_cs(out + 8 * c, q);
                            } else if (!in_place) {
                                st_global_cs(out + 8 * c, raw[j][i]);
                            }
                        }
                    }
                }
            }
            cur = cur + 1 == S ? 0 : cur + 1;
            now.next();
        }
        cp_async_wait<0>();
        if constexpr (BWD) {
            // The groups' sums in group order, through the rings' memory.
            float* part = reinterpret_cast<float*>(smem);  // [groups][D]
            const int groups = nt >> lgG;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NU; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = i ? c1[j] : c0[j];
                    if (c < NC) {
                        float4* q = reinterpret_cast<float4*>(part + (tid >> lgG) * D + 8 * c);
                        const Oct& v = acc[j][i];
                        q[0] = make_float4(v.p[0].x, v.p[0].y, v.p[1].x, v.p[1].y);
                        q[1] = make_float4(v.p[2].x, v.p[2].y, v.p[3].x, v.p[3].y);
                    }
                }
            __syncthreads();
            float* row = a.partials + (static_cast<int64_t>(pass) * gridDim.x + blockIdx.x) * D;
            for (int col = tid; col < D; col += nt) {
                float v = part[col];
                for (int g = 1; g < groups; ++g) v = fadd(v, part[g * D + col]);
                row[col] = v;
            }
            __syncthreads();  // before the next pass fills the rings
        }
    }
    pdl_release();
}

// ---------------------------------------------------------------------------
// Pairs: G lanes a head; lane l has the slots q = l, l + G, ... of D/2. Slot q is
// two values: the pair (q, q + R/2) of the rotation, or from R/2 on two neighbours
// of the rest. NJ slots a lane at most, NV vectors a lane to copy.
// ---------------------------------------------------------------------------
template <int MODE, bool F16, int NJ, int S>
__global__ void __launch_bounds__(kRopeThreads) rope_pairs_kernel(const RopeArgs a, const int lgG) {
    constexpr bool NORM = MODE != kTurn, BWD = MODE == kNormTurnBwd;
    constexpr int OPS = BWD ? 2 : 1;
    extern __shared__ __align__(16) unsigned char smem[];
    const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
    const int D = a.D, NC = D >> 3, half = a.R >> 1, hp = (half + 7) & ~7;
    const int G = 1 << lgG, l = lane & (G - 1), head = lane >> lgG, per = 32 >> lgG;
    const int groups = nt >> lgG, group = tid >> lgG;
    uint16_t* rows = reinterpret_cast<uint16_t*>(smem) + group * D;               // [S][OPS][groups][D]
    const int stride = groups * D;
    float* wsm = reinterpret_cast<float*>(smem + static_cast<size_t>(S) * OPS * stride * 2);  // NORM: [q | k][D]
    float* cs = wsm + (NORM ? 2 * D : 0) + warp * 2 * hp;                           // [warps][cos | sin][hp]
    unsigned long long* F = reinterpret_cast<unsigned long long*>(wsm + (NORM ? 2 * D : 0) + nw * 2 * hp);
    pdl_wait();
    for (int i = tid; i < half; i += nt) F[i] = rope_turns(a.inv_freq[i]);
    if constexpr (NORM) {
        for (int i = tid; i < 2 * D; i += nt) {
            const int s = i >= D;
            if (a.H[s] > 0) {
                const float w = a.w[s][s ? i - D : i];
                wsm[i] = a.zc ? fadd(w, 1.0f) : w;
            }
        }
    }
    __syncthreads();

    for (int pass = 0; pass < (BWD ? 2 : 1); ++pass) {
        const int nq = (a.H[0] + per - 1) >> (5 - lgG), nk = (a.H[1] + per - 1) >> (5 - lgG);
        const int nb = BWD ? (pass ? nk : nq) : nq + nk;
        if (nb == 0) continue;
        Turns now(a.T, nb, BWD && pass ? 0 : nq, static_cast<int64_t>(blockIdx.x) * nw + warp, static_cast<int64_t>(gridDim.x) * nw);
        Turns ahead = now;
        int fs = 0;
        auto fetch = [&]() {
            if (ahead.left > 0) {
                const int s = ahead.tensor(), h = ahead.turn_of_tensor() * per + head;
                if (h < a.H[s]) {
                    const uint16_t* p = a.in[s].p + static_cast<int64_t>(ahead.t) * a.in[s].token + h * a.in[s].head;
                    uint16_t* to = rows + fs * OPS * stride;
                    for (int v = l; v < NC; v += G) cp_async16(to + 8 * v, p + 8 * v);
                    if constexpr (BWD) {
                        const uint16_t* x = a.x[s].p + static_cast<int64_t>(ahead.t) * a.x[s].token + h * a.x[s].head;
                        for (int v = l; v < NC; v += G) cp_async16(to + stride + 8 * v, x + 8 * v);
                    }
                }
                ahead.next();
            }
            cp_async_commit();
            fs = fs + 1 == S ? 0 : fs + 1;
        };
#pragma unroll
        for (int i = 0; i < S - 1; ++i) fetch();
        long long p_next = now.left > 0 ? position(a, now.t) : 0;
        float acc[NJ][2];
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[j][0] = acc[j][1] = 0.0f;
        int t_angles = -1;
        int cur = 0;
        while (now.left > 0) {
            if (now.t != t_angles) {
                t_angles = now.t;
                token_angles(cs, hp, half, F, p_next, a.scale, BWD || a.back, lane);
                if (t_angles + 1 < a.T) p_next = position(a, t_angles + 1);
            }
            const int s = now.tensor(), h = now.turn_of_tensor() * per + head;
            const bool have = h < a.H[s];
            float r = 0.0f, coef = 0.0f, sum = 0.0f;
            if constexpr (BWD) {
                if (have) r = __ldg(a.rstd[s] + static_cast<int64_t>(now.t) * a.H[s] + h);
            }
            cp_async_wait<S - 2>();
            __syncwarp();  // the other lanes' copies too
            uint16_t* ri = rows + cur * OPS * stride;
            const uint16_t* rx = ri + stride;
            const float* w = wsm + s * D;
            float u[NJ][2], x[NJ][2];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int q = l + (j << lgG);
                if (have && 2 * q < D) {
                    const bool turn = q < half;
                    const int i0 = turn ? q : 2 * q, i1 = turn ? q + half : 2 * q + 1;
                    u[j][0] = widen<F16>(ri[i0]);
                    u[j][1] = widen<F16>(ri[i1]);
                    if constexpr (BWD) {
                        x[j][0] = widen<F16>(rx[i0]);
                        x[j][1] = widen<F16>(rx[i1]);
                        if (turn) {
                            const float2 o = rope_turn(u[j][0], u[j][1], make_float2(cs[q], cs[hp + q]));
                            u[j][0] = o.x;
                            u[j][1] = o.y;
                        }
                        acc[j][0] = __fmaf_rn(u[j][0], fmul(x[j][0], r), acc[j][0]);
                        acc[j][1] = __fmaf_rn(u[j][1], fmul(x[j][1], r), acc[j][1]);
                        u[j][0] = fmul(u[j][0], w[i0]);
                        u[j][1] = fmul(u[j][1], w[i1]);
                        sum = __fmaf_rn(u[j][0], x[j][0], sum);
                        sum = __fmaf_rn(u[j][1], x[j][1], sum);
                    } else if constexpr (NORM) {
                        sum = __fmaf_rn(u[j][0], u[j][0], sum);
                        sum = __fmaf_rn(u[j][1], u[j][1], sum);
                    }
                }
            }
            if constexpr (NORM) {
                sum = lanes_sum(sum, G);
                if constexpr (BWD) {
                    coef = -fmul(fmul(fmul(fmul(r, r), r), a.rcp_d), sum);
                } else {
                    r = rsqrtf(fadd(fmul(sum, a.rcp_d), a.eps));
                    if (have && l == 0) a.rstd[s][static_cast<int64_t>(now.t) * a.H[s] + h] = r;
                }
            }
            __syncwarp();  // every lane has its values: the row is overwritten with the results
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int q = l + (j << lgG);
                if (have && 2 * q < D) {
                    const bool turn = q < half;
                    const int i0 = turn ? q : 2 * q, i1 = turn ? q + half : 2 * q + 1;
                    if constexpr (BWD) {
                        u[j][0] = __fmaf_rn(u[j][0], r, fmul(x[j][0], coef));
                        u[j][1] = __fmaf_rn(u[j][1], r, fmul(x[j][1], coef));
                    } else {
                        if constexpr (NORM) {
                            u[j][0] = fmul(fmul(u[j][0], r), w[i0]);
                            u[j][1] = fmul(fmul(u[j][1], r), w[i1]);
                        }
                        if (turn) {
                            const float2 o = rope_turn(u[j][0], u[j][1], make_float2(cs[q], cs[hp + q]));
                            u[j][0] = o.x;
                            u[j][1] = o.y;
                        }
                    }
                    if (NORM || turn) {  // the rest of a rotation alone keeps its bits
                        ri[i0] = narrow<F16>(u[j][0]);
                        ri[i1] = narrow<F16>(u[j][1]);
                    }
                }
            }
            __syncwarp();
            if (have) {
                uint16_t* out = a.out[s].p + static_cast<int64_t>(now.t) * a.out[s].token + h * a.out[s].head;
                const int n = MODE == kTurn && a.out[s].p == a.in[s].p ? (a.R + 7) >> 3 : NC;  // in place: what is turned
                for (int v = l; v < n; v += G) st_global_cs(out + 8 * v, reinterpret_cast<const uint4*>(ri)[v]);
            }
            __syncwarp();  // before the row's slot is filled again
            fetch();
            cur = cur + 1 == S ? 0 : cur + 1;
            now.next();
        }
        cp_async_wait<0>();
        if constexpr (BWD) {
            float* part = reinterpret_cast<float*>(smem);  // [groups][D]
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int q = l + (j << lgG);
                if (2 * q < D) {
                    part[group * D + (q < half ? q : 2 * q)] = acc[j][0];
                    part[group * D + (q < half ? q + half : 2 * q + 1)] = acc[j][1];
                }
            }
            __syncthreads();
            float* row = a.partials + (static_cast<int64_t>(pass) * gridDim.x + blockIdx.x) * D;
            for (int col = tid; col < D; col += nt) {
                float v = part[col];
                for (int g = 1; g < groups; ++g) v = fadd(v, part[g * D + col]);
                row[col] = v;
            }
            __syncthreads();
        }
    }
    pdl_release();
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------

// CTAs of a launch whose order of sums does not matter: all that fit, in smaller
// CTAs where there are few turns of warps, so that they spread over the SMs.
template <typename Kern>
cudaError_t rope_launch_free(Kern kern, const RopeArgs& a, int lgG, int64_t turns, size_t smem_thread, size_t smem_warp,
                             size_t smem_fixed, cudaStream_t st) {
    const int64_t sms = sm_count();
    int threads = kRopeThreads;
    while (threads > 32 && turns * 32 < sms * threads) threads /= 2;
    const int smem = static_cast<int>(smem_thread * threads + smem_warp * (threads / 32) + smem_fixed);
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    const int occ = ctas_per_sm(reinterpret_cast<const void*>(kern), threads, smem);
    if (occ < 1) return cudaErrorInvalidConfiguration;
    const int64_t warps = threads / 32;
    const int64_t grid = std::min<int64_t>((turns + warps - 1) / warps, sms * occ);
    return launch_kernel(kern, static_cast<unsigned>(grid), threads, static_cast<size_t>(smem), st, a, lgG);
}

template <int MODE, bool INTER, bool F16, int NU, int S, int MINB>
cudaError_t rope_units(const RopeArgs& a, int lgG, int64_t turns, cudaStream_t st) {
    constexpr bool NORM = MODE != kTurn, BWD = MODE == kNormTurnBwd;
    const auto kern = rope_units_kernel<MODE, INTER, F16, NU, S, MINB>;
    const int half = a.R / 2, hp = (half + 7) & ~7;
    const size_t thread = static_cast<size_t>(S) * (BWD ? 2 : 1) * 2 * NU * 16 + (BWD ? S * 4 : 0);
    const size_t fixed = (NORM ? static_cast<size_t>(a.D) * 8 : 0) + static_cast<size_t>(half) * 8;
    if constexpr (!BWD) {
        return rope_launch_free(kern, a, lgG, turns, thread, static_cast<size_t>(hp) * 8, fixed, st);
    } else {
        const size_t smem = std::max<size_t>(thread * kRopeThreads + static_cast<size_t>(hp) * 8 * (kRopeThreads / 32) + fixed,
                                             static_cast<size_t>(kRopeThreads >> lgG) * a.D * 4);
        cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        const unsigned grid = static_cast<unsigned>(rope_bwd_ctas(a.T, a.H[0], a.H[1], a.D));
        return launch_kernel(kern, grid, kRopeThreads, smem, st, a, lgG);
    }
}

template <int MODE, bool F16, int NJ, int S>
cudaError_t rope_pairs(const RopeArgs& a, int lgG, int64_t turns, cudaStream_t st) {
    constexpr bool NORM = MODE != kTurn, BWD = MODE == kNormTurnBwd;
    const auto kern = rope_pairs_kernel<MODE, F16, NJ, S>;
    const int half = a.R / 2, hp = (half + 7) & ~7;
    // a head's row for each group of lanes: bytes a thread, of whole warps
    const size_t warp_rows = static_cast<size_t>(S) * (BWD ? 2 : 1) * (32 >> lgG) * a.D * 2;
    const size_t fixed = (NORM ? static_cast<size_t>(a.D) * 8 : 0) + static_cast<size_t>(half) * 8;
    if constexpr (!BWD) {
        return rope_launch_free(kern, a, lgG, turns, 0, warp_rows + static_cast<size_t>(hp) * 8, fixed, st);
    } else {
        const size_t smem = std::max<size_t>((warp_rows + static_cast<size_t>(hp) * 8) * (kRopeThreads / 32) + fixed,
                                             static_cast<size_t>(kRopeThreads >> lgG) * a.D * 4);
        cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        const unsigned grid = static_cast<unsigned>(rope_bwd_ctas(a.T, a.H[0], a.H[1], a.D));
        return launch_kernel(kern, grid, kRopeThreads, smem, st, a, lgG);
    }
}

#ifndef RP_F1
#define RP_F1 1, 3, 4
#endif
#ifndef RP_F2
#define RP_F2 2, 3, 3
#endif
#ifndef RP_F3
#define RP_F3 3, 3, 2
#endif
#ifndef RP_B1
#define RP_B1 1, 3, 2
#endif

template <int MODE, bool INTER, bool F16>
cudaError_t rope_units_of(const RopeArgs& a, cudaStream_t st) {
    const RopeShape s = rope_shape(a.D, MODE == kNormTurnBwd);
    const int64_t turns = a.T * (rope_turns_of(a.H[0], s) + rope_turns_of(a.H[1], s));
    if constexpr (MODE == kNormTurnBwd) {
        return rope_units<MODE, INTER, F16, RP_B1>(a, s.lgG, turns, st);
    } else {
        if (s.NU == 1) return rope_units<MODE, INTER, F16, RP_F1>(a, s.lgG, turns, st);
        if (s.NU == 2) return rope_units<MODE, INTER, F16, RP_F2>(a, s.lgG, turns, st);
        return rope_units<MODE, INTER, F16, RP_F3>(a, s.lgG, turns, st);
    }
}

template <int MODE, bool F16>
cudaError_t rope_dispatch(const RopeArgs& a, cudaStream_t st) {
    if (a.layout == ROPE_INTERLEAVED) return rope_units_of<MODE, true, F16>(a, st);
    if (a.R % 16 == 0) return rope_units_of<MODE, false, F16>(a, st);
    int lg = 0;
    while (lg < 5 && (8 << lg) < a.D) ++lg;  // four slots a lane, eight beyond D = 256
    const RopeShape s{lg, 0};
    const int64_t turns = a.T * (rope_turns_of(a.H[0], s) + rope_turns_of(a.H[1], s));
    return a.D <= 256 ? rope_pairs<MODE, F16, 4, 3>(a, lg, turns, st) : rope_pairs<MODE, F16, 8, 3>(a, lg, turns, st);
}

template <bool F16>
cudaError_t rope_mode(RopeMode mode, const RopeArgs& a, cudaStream_t st) {
    switch (mode) {
        case kTurn: return rope_dispatch<kTurn, F16>(a, st);
        case kNormTurn: return rope_dispatch<kNormTurn, F16>(a, st);
        default: return rope_dispatch<kNormTurnBwd, F16>(a, st);
    }
}

}  // namespace
}  // namespace rmsn
