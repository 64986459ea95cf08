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
// A warp takes a turn of up to NR x 32 / G heads of one token at a time, G lanes a
// head (the smallest power of two that holds its units). The turns of a launch are
// split among its warps in contiguous ranges, so a warp computes a token's cosines
// once for all its heads and keeps those of its lanes' pairs in registers. Rows come
// and go by bulk (TMA) copies between HBM and a ring of S stages in the warp's own
// shared memory: lanes read their values there, overwrite them with the results,
// and one lane sends the stage back. Warps never wait for one another; dw is
// summed in registers and joined over the CTA's groups at the end, in group order,
// one partial row a CTA.
//
// A lane's unit is two times eight values, A and B:
//   * kHalves (ROPE_HALF, R a multiple of 16): a 16-byte vector of the first half
//     and the vector of its partners R/2 values on; beyond the turned part two vectors.
//   * kNeighbours (ROPE_INTERLEAVED): two vectors.
//   * kHalvesAny (ROPE_HALF, any R): as kHalves, but B (and, beyond the turned part,
//     A) lies at any even number of bytes and may be cut short by the half's end.
#pragma once

#include <algorithm>

#include "f32x2.cuh"
#include "kernels.h"
#include "rope_launch.h"
#include "rope_math.cuh"

namespace rmsn {
namespace {

__device__ __forceinline__ long long position(const RopeArgs& a, int64_t t) {
    if (a.pos == nullptr) return t;
    return a.pos64 ? static_cast<const long long*>(a.pos)[t] : static_cast<const int*>(a.pos)[t];
}

// Device error word of the including translation unit.
__device__ unsigned int g_rope_error;

cudaError_t read_rope_error_word(unsigned* flags, bool clear) {
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_rope_error, sizeof(v));
    if (e != cudaSuccess) return e;
    *flags |= v;
    if (clear && v) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(zero));
    }
    return e;
}

// A warp's contiguous range of the turns: token t, heads h .. h + step - 1 of
// tensor s, q's heads first, then k's (a turn has heads of one of them only, so
// all that depends on which is the same for the whole warp). (A warp's own turns
// fit an int: 2^31 of them would be 2^35 bytes a warp.)
struct Turns {
    int left, t, s, h;
    __device__ __forceinline__ Turns(int64_t T, int nq, int nk, int step, int64_t warp, int64_t warps) {
        const int64_t all = T * (nq + nk), first = all * warp / warps;
        left = static_cast<int>(all * (warp + 1) / warps - first);
        t = static_cast<int>(first / (nq + nk));
        const int b = static_cast<int>(first - static_cast<int64_t>(t) * (nq + nk));
        s = b >= nq;
        h = (s ? b - nq : b) * step;
    }
    // Hq, Hk: the heads that the walk covers (0: none of that tensor).
    __device__ __forceinline__ void next(int Hq, int Hk, int step) {
        --left;
        h += step;
        if (h >= (s ? Hk : Hq)) {
            h = 0;
            if (s == 0 && Hk > 0) {
                s = 1;
            } else {
                s = Hq > 0 ? 0 : 1;
                ++t;
            }
        }
    }
};

__device__ __forceinline__ uint4 lds128(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t p) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t p) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(p) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t p, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t p, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(p), "r"(v) : "memory"); }
__device__ __forceinline__ void sts16(uint32_t p, uint32_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(p), "h"(static_cast<uint16_t>(v)) : "memory");
}

template <bool F16>
__device__ __forceinline__ float widen(uint32_t v) {
    return F16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(v))) : __uint_as_float(v << 16);
}
template <bool F16>
__device__ __forceinline__ uint32_t narrow(float v) {
    return F16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Sixteen bytes at any even address, through the words that hold them (n <= 8
// values are wanted; no word without one of them is read).
__device__ __forceinline__ uint4 lds_window(uint32_t p, int n) {
    const bool odd = p & 2u;
    const uint32_t q = p & ~3u;
    uint32_t w[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = 2 * i < n + (odd ? 1 : 0) ? lds32(q + 4 * i) : 0u;
    uint4 v;
    v.x = odd ? __funnelshift_r(w[0], w[1], 16) : w[0];
    v.y = odd ? __funnelshift_r(w[1], w[2], 16) : w[1];
    v.z = odd ? __funnelshift_r(w[2], w[3], 16) : w[2];
    v.w = odd ? __funnelshift_r(w[3], w[4], 16) : w[3];
    return v;
}
// The first n of eight values to any even address.
__device__ __forceinline__ void sts_window(uint32_t p, uint4 v, int n) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if ((p & 2u) == 0 && n == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sts32(p + 4 * i, w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) sts16(p + 2 * i, i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
    }
}

// 1-D bulk copy shared -> global, in the thread's current bulk group.
__device__ __forceinline__ void bulk_s2g(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// All but the N newest of the thread's bulk groups have read their shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

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
__device__ __forceinline__ void turn_neighbours(Oct& A, const float2 (&c)[2], const float2 (&s)[2], int n) {
    const float cc[4] = {c[0].x, c[0].y, c[1].x, c[1].y}, ss[4] = {s[0].x, s[0].y, s[1].x, s[1].y};
    const Oct was = A;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = A.p[i], uc = fmul2(u, both(cc[i]));
        A.p[i] = make_float2(__fmaf_rn(-u.y, ss[i], uc.x), __fmaf_rn(u.x, ss[i], uc.y));
    }
    if (n < 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i >= n) A.p[i] = was.p[i];
    }
}
// Values from place n on become zero.
__device__ __forceinline__ void cut(Oct& A, int n) {
    if (n < 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (2 * i >= n) A.p[i].x = 0.0f;
            if (2 * i + 1 >= n) A.p[i].y = 0.0f;
        }
    }
}

enum RopeKind : int { kHalves = 0, kNeighbours = 1, kHalvesAny = 2 };

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <int MODE, int KIND, bool F16, int NR, int S, int MINB>
__global__ void __launch_bounds__(kRopeThreads, MINB) rope_kernel(const RopeArgs a, const int lgG) {
    constexpr bool NORM = MODE != kTurn, BWD = MODE == kNormTurnBwd;
    constexpr int OPS = BWD ? 2 : 1;
    extern __shared__ __align__(128) unsigned char smem[];
    const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
    const int D = a.D, half = a.R >> 1, hp = (half + 7) & ~7;
    const int l = lane & ((1 << lgG) - 1), head = lane >> lgG, per = 32 >> lgG, step = per * NR;
    const uint32_t pitch = static_cast<uint32_t>(D) * 2u;
    const uint32_t op_bytes = static_cast<uint32_t>(step) * pitch, stage_bytes = OPS * op_bytes;
    // Shared memory: every warp's stages; weights [q | k][D]; every warp's [cos | sin][hp];
    // BWD: every warp's inverse RMS [S][step]; barriers; frequencies.
    float* wsm = reinterpret_cast<float*>(smem + static_cast<size_t>(nw) * S * stage_bytes);
    float* cs = wsm + (NORM ? 2 * D : 0) + warp * 2 * hp;
    float* rs = wsm + (NORM ? 2 * D : 0) + nw * 2 * hp + (BWD ? warp * S * step : 0);
    uint64_t* bars = reinterpret_cast<uint64_t*>(wsm + (NORM ? 2 * D : 0) + nw * 2 * hp + (BWD ? nw * S * step : 0));
    unsigned long long* F = reinterpret_cast<unsigned long long*>(bars + nw * S);
    uint64_t* full = bars + warp * S;
    const uint32_t ring = smem_u32(smem) + warp * S * stage_bytes;

    // This lane's unit: where A and B lie in a row (bytes), how many of their eight
    // values there are, and of what pairs they are.
    const int NC = D >> 3;
    const int NP = KIND == kNeighbours ? 0 : KIND == kHalves ? half >> 3 : (half + 7) >> 3;  // units of the halves
    const bool turned = l < NP;
    int atA, atB, nA = 8, nB = 8;
    if (turned) {
        atA = 8 * l;
        atB = half + 8 * l;
        if constexpr (KIND == kHalvesAny) nA = nB = min(8, half - 8 * l);
    } else if constexpr (KIND == kHalvesAny) {
        atA = a.R + 16 * (l - NP);
        atB = atA + 8;
        nA = max(0, min(8, D - atA));
        nB = max(0, min(8, D - atB));
    } else {
        const int rest = (NC - 2 * NP + 1) >> 1, c = l + NP;  // 2 NP + (l - NP)
        atA = 8 * c;
        atB = 8 * (c + rest);
        if (l >= NP + rest) nA = 0;
        if (nA == 0 || c + rest >= NC) nB = 0;
    }
    // kHalvesAny: a value beyond the units of 32 lanes, if there is one for this lane.
    const int atX = KIND == kHalvesAny && NORM ? a.R + 16 * ((1 << lgG) - NP) + l : D;
    const bool hasX = KIND == kHalvesAny && NORM && atX < D;
    const uint32_t rowA = head * pitch + 2u * atA, rowB = head * pitch + 2u * atB;

    for (int i = tid; i < nw * S; i += nt) mbar_init(&bars[i], 1);
    fence_mbar_init();
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

    const uint64_t pol = policy_evict_first();
    auto load = [&](uint32_t at, int n) -> uint4 {
        if constexpr (KIND == kHalvesAny) return lds_window(at, n);
        return lds128(at);
    };
    auto store = [&](uint32_t at, const Oct& o, int n) {
        const uint4 v = oct_pack<F16>(o);
        if constexpr (KIND == kHalvesAny) sts_window(at, v, n);
        else sts128(at, v);
    };
    uint32_t phase = 0;  // of the stage that comes next
    int cur = 0;
    // Forward: one pass over the turns of q and of k. Backward: q, then k, each with its own weight gradient.
    for (int pass = 0; pass < (BWD ? 2 : 1); ++pass) {
        const int Hq = BWD && pass ? 0 : a.H[0], Hk = BWD && !pass ? 0 : a.H[1];
        const int nq = (Hq + step - 1) / step, nk = (Hk + step - 1) / step;
        if (nq + nk == 0) continue;
        Turns now(a.T, nq, nk, step, static_cast<int64_t>(blockIdx.x) * nw + warp, static_cast<int64_t>(gridDim.x) * nw);
        Turns ahead = now;
        int fs = cur;
        auto fetch = [&]() {
            if (ahead.left > 0) {
                const int s = ahead.s, n = min(step, a.H[s] - ahead.h);
                const uint32_t to = ring + fs * stage_bytes;
                if (lane == 0) {
                    const uint32_t bytes = a.row_bytes[s];
                    mbar_arrive_expect_tx(&full[fs], static_cast<uint32_t>(n) * OPS * bytes);
#pragma unroll
                    for (int op = 0; op < OPS; ++op) {
                        const HeadsIn& in = op ? a.x[s] : a.in[s];
                        const uint16_t* p = in.p + ahead.t * in.token + ahead.h * in.head;
                        // Heads side by side come in one copy.
                        const bool one = in.head == D && bytes == pitch;
                        const int copies = one ? 1 : n;
                        for (int i = 0; i < copies; ++i)
                            bulk_g2s(smem + (to - smem_u32(smem)) + op * op_bytes + i * pitch, p + i * in.head,
                                     one ? n * pitch : bytes, &full[fs], pol);
                    }
                }
                if constexpr (BWD) {
                    for (int i = lane; i < n; i += 32)
                        cp_async4(rs + fs * step + i, a.rstd[s] + static_cast<int64_t>(ahead.t) * a.H[s] + ahead.h + i);
                }
                ahead.next(Hq, Hk, step);
            }
            if constexpr (BWD) cp_async_commit();
            fs = fs + 1 == S ? 0 : fs + 1;
        };
#pragma unroll
        for (int i = 0; i < S - 1; ++i) fetch();
        long long p_next = now.left > 0 ? position(a, now.t) : 0;
        Oct accA = oct_zero(), accB = oct_zero(), wA = oct_zero(), wB = oct_zero();
        float accX = 0.0f, wX = 0.0f;
        float2 c[4], sn[4];  // cos and sin of this lane's pairs
        int t_have = -1, s_have = -1;
        while (now.left > 0) {
            if (now.t != t_have) {
                t_have = now.t;
                token_angles(cs, hp, half, F, p_next, a.scale, BWD || a.back, lane);
                if (t_have + 1 < a.T) p_next = position(a, t_have + 1);
                if constexpr (KIND == kNeighbours) {
                    const float4* q = reinterpret_cast<const float4*>(cs);
                    const int iA = min(atA >> 3, (hp >> 2) - 1), iB = min(atB >> 3, (hp >> 2) - 1);
                    const float4 ca = q[iA], cb = q[iB], sa = q[(hp >> 2) + iA], sb = q[(hp >> 2) + iB];
                    c[0] = make_float2(ca.x, ca.y); c[1] = make_float2(ca.z, ca.w); c[2] = make_float2(cb.x, cb.y); c[3] = make_float2(cb.z, cb.w);
                    sn[0] = make_float2(sa.x, sa.y); sn[1] = make_float2(sa.z, sa.w); sn[2] = make_float2(sb.x, sb.y); sn[3] = make_float2(sb.z, sb.w);
                } else if (turned) {
                    const float2* q = reinterpret_cast<const float2*>(cs + atA);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        c[i] = q[i];
                        sn[i] = q[(hp >> 1) + i];
                    }
                }
            }
            const int s = now.s;
            if (NORM && s != s_have) {
                s_have = s;
                const float* w = wsm + s * D;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (KIND != kHalvesAny) {
                        if (nA > 0) wA.p[i] = reinterpret_cast<const float2*>(w + atA)[i];
                        if (nB > 0) wB.p[i] = reinterpret_cast<const float2*>(w + atB)[i];
                    } else {
                        wA.p[i] = make_float2(2 * i < nA ? w[atA + 2 * i] : 0.0f, 2 * i + 1 < nA ? w[atA + 2 * i + 1] : 0.0f);
                        wB.p[i] = make_float2(2 * i < nB ? w[atB + 2 * i] : 0.0f, 2 * i + 1 < nB ? w[atB + 2 * i + 1] : 0.0f);
                    }
                }
                if (hasX) wX = w[atX];
            }
            if constexpr (BWD) cp_async_wait<S - 2>();
            if (!__all_sync(0xffffffffu, mbar_wait(&full[cur], phase))) {
                // Give up: wait (bounded) for the copies in flight, and leave the turns.
                if (lane == 0) {
                    for (int i = 1, f = cur, ph = phase; i < S; ++i) {
                        if (++f == S) {
                            f = 0;
                            ph ^= 1u;
                        }
                        if (i < now.left) (void)mbar_wait(&full[f], ph);
                    }
                    atomicOr(&g_rope_error, kErrWaitTimeout);
                }
                break;
            }
            __syncwarp();  // BWD: the other lanes' inverse RMS
            const uint32_t st = ring + cur * stage_bytes;
            const int n = min(step, a.H[s] - now.h);
            auto turn = [&](Oct& A, Oct& B) {
                if constexpr (KIND == kNeighbours) {
                    const int tA = half - (atA >> 1), tB = half - (atB >> 1);  // pairs of A and of B that are turned
                    const float2 c0[2] = {c[0], c[1]}, c1[2] = {c[2], c[3]}, s0[2] = {sn[0], sn[1]}, s1[2] = {sn[2], sn[3]};
                    if (tA > 0) turn_neighbours(A, c0, s0, tA);
                    if (tB > 0) turn_neighbours(B, c1, s1, tB);
                } else if (turned) {
                    Oct co, so;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        co.p[i] = c[i];
                        so.p[i] = sn[i];
                    }
                    turn_halves(A, B, co, so);
                }
            };
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                if (i * per >= n) break;  // the same for all lanes
                const bool have = i * per + head < n;
                const uint32_t at = st + i * per * pitch;
                if constexpr (MODE == kTurn) {
                    // What is not turned stays where it is.
                    if constexpr (KIND == kNeighbours) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int n_turn = half - ((k ? atB : atA) >> 1);
                            const uint32_t p = at + (k ? rowB : rowA);
                            if (have && (k ? nB : nA) > 0 && n_turn > 0) {
                                const uint4 raw = lds128(p);
                                Oct A = oct_unpack<F16>(raw);
                                const float2 ck[2] = {c[2 * k], c[2 * k + 1]}, sk[2] = {sn[2 * k], sn[2 * k + 1]};
                                turn_neighbours(A, ck, sk, 4);
                                uint4 v = oct_pack<F16>(A);
                                if (n_turn < 4) {  // the rest of the vector keeps its bits
                                    if (n_turn < 2) v.y = raw.y;
                                    if (n_turn < 3) v.z = raw.z;
                                    v.w = raw.w;
                                }
                                sts128(p, v);
                            }
                        }
                    } else {
                        Oct A, B;
                        if (have && turned) {
                            A = oct_unpack<F16>(load(at + rowA, nA));
                            B = oct_unpack<F16>(load(at + rowB, nB));
                        }
                        if (KIND == kHalvesAny) __syncwarp();  // all are read before any is written
                        if (have && turned) {
                            turn(A, B);
                            store(at + rowA, A, nA);
                            store(at + rowB, B, nB);
                        }
                    }
                } else {
                    Oct A = oct_zero(), B = oct_zero(), xA = oct_zero(), xB = oct_zero();
                    float2 sum2 = make_float2(0.0f, 0.0f);
                    float r = 0.0f, coef = 0.0f, X = 0.0f, xX = 0.0f, sumX = 0.0f;
                    const uint32_t pX = at + head * pitch + 2u * atX;
                    if (have && hasX) X = widen<F16>(lds16(pX));
                    if (have && nA > 0) A = oct_unpack<F16>(load(at + rowA, nA));
                    if (have && nB > 0) B = oct_unpack<F16>(load(at + rowB, nB));
                    if constexpr (KIND == kHalvesAny) {
                        cut(A, nA);
                        cut(B, nB);
                    }
                    if constexpr (BWD) {
                        if (have && nA > 0) xA = oct_unpack<F16>(load(at + op_bytes + rowA, nA));
                        if (have && nB > 0) xB = oct_unpack<F16>(load(at + op_bytes + rowB, nB));
                        if constexpr (KIND == kHalvesAny) {
                            cut(xA, nA);
                            cut(xB, nB);
                        }
                        if (have) r = rs[cur * step + i * per + head];
                        if (have && hasX) {
                            xX = widen<F16>(lds16(pX + op_bytes));
                            accX = __fmaf_rn(X, fmul(xX, r), accX);
                            X = fmul(X, wX);
                            sumX = fmul(X, xX);
                        }
                        turn(A, B);
                        if constexpr (KIND == kHalvesAny) {  // what the cosines beyond the half's end made of zeros
                            cut(A, nA);
                            cut(B, nB);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            accA.p[e] = fma2(A.p[e], fmul2(xA.p[e], both(r)), accA.p[e]);
                            accB.p[e] = fma2(B.p[e], fmul2(xB.p[e], both(r)), accB.p[e]);
                            A.p[e] = fmul2(A.p[e], wA.p[e]);
                            B.p[e] = fmul2(B.p[e], wB.p[e]);
                            sum2 = fma2(A.p[e], xA.p[e], sum2);
                            sum2 = fma2(B.p[e], xB.p[e], sum2);
                        }
                    } else {
                        if (KIND == kHalvesAny) sumX = fmul(X, X);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            sum2 = fma2(A.p[e], A.p[e], sum2);
                            sum2 = fma2(B.p[e], B.p[e], sum2);
                        }
                    }
                    float mine = fadd(sum2.x, sum2.y);
                    if constexpr (KIND == kHalvesAny) mine = fadd(mine, sumX);
                    const float sum = lanes_sum(mine, 1 << lgG);  // every lane of the group has read its values
                    if constexpr (BWD) {
                        coef = -fmul(fmul(fmul(fmul(r, r), r), a.rcp_d), sum);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            A.p[e] = fma2(A.p[e], both(r), fmul2(xA.p[e], both(coef)));
                            B.p[e] = fma2(B.p[e], both(r), fmul2(xB.p[e], both(coef)));
                        }
                    } else {
                        r = rsqrtf(fadd(fmul(sum, a.rcp_d), a.eps));
                        if (have && l == 0) a.rstd[s][static_cast<int64_t>(now.t) * a.H[s] + now.h + i * per + head] = r;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            A.p[e] = fmul2(fmul2(A.p[e], both(r)), wA.p[e]);
                            B.p[e] = fmul2(fmul2(B.p[e], both(r)), wB.p[e]);
                        }
                        turn(A, B);
                    }
                    if (have && nA > 0) store(at + rowA, A, nA);
                    if (have && nB > 0) store(at + rowB, B, nB);
                    if (have && hasX) sts16(pX, narrow<F16>(BWD ? __fmaf_rn(X, r, fmul(xX, coef)) : fmul(fmul(X, r), wX)));
                }
            }
            fence_proxy_async_smem();  // the results, before the copy that sends them and the one that refills the stage
            __syncwarp();
            if (lane == 0) {
                const HeadsOut& o = a.out[s];
                uint16_t* p = o.p + now.t * o.token + now.h * o.head;
                const uint32_t bytes = a.row_bytes[s];
                const bool one = o.head == D && bytes == pitch;
                const int copies = one ? 1 : n;
                for (int i = 0; i < copies; ++i) bulk_s2g(p + i * o.head, st + i * pitch, one ? n * pitch : bytes);
                bulk_commit();
                bulk_wait_read<1>();  // the stage of the turn before is sent: it is filled next
            }
            if (++cur == S) {
                cur = 0;
                phase ^= 1u;
            }
            now.next(Hq, Hk, step);
            fetch();
        }
        if (lane == 0) bulk_wait_all();
        if constexpr (BWD) {
            cp_async_wait<0>();
            // The groups' sums in group order, through the stages' memory.
            float* part = reinterpret_cast<float*>(smem);  // [groups][D]
            const int groups = nt >> lgG, group = tid >> lgG;
            fence_proxy_async_smem();
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (e < nA) part[group * D + atA + e] = e & 1 ? accA.p[e / 2].y : accA.p[e / 2].x;
                if (e < nB) part[group * D + atB + e] = e & 1 ? accB.p[e / 2].y : accB.p[e / 2].x;
            }
            if (hasX) part[group * D + atX] = accX;
            __syncthreads();
            float* row = a.partials + (static_cast<int64_t>(pass) * gridDim.x + blockIdx.x) * D;
            for (int col = tid; col < D; col += nt) {
                float v = part[col];
                for (int g = 1; g < groups; ++g) v = fadd(v, part[g * D + col]);
                row[col] = v;
            }
            fence_proxy_async_smem();
            __syncthreads();  // before the next pass fills the stages
        }
    }
    pdl_release();
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
#ifndef RP_T
#define RP_T 2, 3, 3
#endif
#ifndef RP_F
#define RP_F 2, 3, 3
#endif
#ifndef RP_B
#define RP_B 2, 3, 2
#endif

template <int MODE, int KIND, bool F16, int NR, int S, int MINB>
cudaError_t rope_run_kernel(const RopeArgs& a, cudaStream_t st) {
    constexpr bool NORM = MODE != kTurn, BWD = MODE == kNormTurnBwd;
    const auto kern = rope_kernel<MODE, KIND, F16, NR, S, MINB>;
    const int lgG = rope_lanes_log2(a.D, a.R, KIND == kHalvesAny, NORM);
    const int step = (32 >> lgG) * NR, hp = (a.R / 2 + 7) & ~7;
    const size_t warp_bytes = static_cast<size_t>(S) * (BWD ? 2 : 1) * step * a.D * 2 + hp * 8 + (BWD ? S * step * 4 : 0) + S * 8;
    const size_t fixed = (NORM ? static_cast<size_t>(a.D) * 8 : 0) + static_cast<size_t>(a.R / 2) * 8;
    const int64_t turns = a.T * ((a.H[0] + step - 1) / step + (a.H[1] + step - 1) / step);
    const int64_t sms = sm_count();
    // Threads: few turns spread over the SMs in smaller CTAs. The backward's CTAs
    // are a function of the problem (rope_bwd_ctas).
    int threads = kRopeThreads;
    if (!BWD)
        while (threads > 32 && turns * 32 < sms * threads) threads /= 2;
    size_t smem = warp_bytes * (threads / 32) + fixed;
    if (BWD) smem = std::max(smem, static_cast<size_t>(threads >> lgG) * a.D * 4);
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    int64_t grid = rope_bwd_ctas(a.T, a.H[0], a.H[1], a.D);
    if (!BWD) {
        const int occ = ctas_per_sm(reinterpret_cast<const void*>(kern), threads, static_cast<int>(smem));
        if (occ < 1) return cudaErrorInvalidConfiguration;
        grid = std::min<int64_t>((turns + threads / 32 - 1) / (threads / 32), sms * occ);
    }
    return launch_kernel(kern, static_cast<unsigned>(grid), threads, smem, st, a, lgG);
}

template <int MODE, bool F16>
cudaError_t rope_dispatch(const RopeArgs& a, cudaStream_t st) {
    if constexpr (MODE == kTurn) {
        if (a.layout == ROPE_INTERLEAVED) return rope_run_kernel<MODE, kNeighbours, F16, RP_T>(a, st);
        if (a.R % 16 == 0) return rope_run_kernel<MODE, kHalves, F16, RP_T>(a, st);
        return rope_run_kernel<MODE, kHalvesAny, F16, RP_T>(a, st);
    } else if constexpr (MODE == kNormTurn) {
        if (a.layout == ROPE_INTERLEAVED) return rope_run_kernel<MODE, kNeighbours, F16, RP_F>(a, st);
        if (a.R % 16 == 0) return rope_run_kernel<MODE, kHalves, F16, RP_F>(a, st);
        return rope_run_kernel<MODE, kHalvesAny, F16, RP_F>(a, st);
    } else {
        if (a.layout == ROPE_INTERLEAVED) return rope_run_kernel<MODE, kNeighbours, F16, RP_B>(a, st);
        if (a.R % 16 == 0) return rope_run_kernel<MODE, kHalves, F16, RP_B>(a, st);
        return rope_run_kernel<MODE, kHalvesAny, F16, RP_B>(a, st);
    }
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
