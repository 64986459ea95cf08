// Rotary positions and the head norm fused with them: kernels and launchers,
// included by the translation units that instantiate them (rope_turn, rope_norm and
// rope_norm_bwd: bf16 activations; with _f16: fp16).
//
// Mathematics, per pair (u, v) of a head and its angle a:
//   turn:            (u c - v s, v c + u s), c = scale cos a, s = scale sin a
//   norm + turn:     r = rsqrt(sum x^2 / D + eps), the turn of (x r) w
//   its backward:    g' = turn of g by -a; gw = g' w;
//                    dx = r gw - x r^2 (r sum(gw x) / D);  dw = sum g' (x r)
// The kernels are bound by HBM: 4 D bytes a head forward, 6 D backward; the
// angles (rope_math.cuh) are computed once a token by the warp that has it, a few
// percent of its work.
//
// A warp takes a turn of up to NR x 32 / G heads of one token at a time, G lanes a
// head (the smallest power of two that holds its units); or, where a token has few
// heads (MANY), of up to NR heads each of 32 / G tokens, a token a group of lanes.
// The turns of a launch are split among its warps in contiguous ranges, so a warp
// computes a token's cosines once for all its heads (MANY: every lane those of its
// own pairs) and keeps those of its lanes' pairs in registers. Rows come
// and go by bulk (TMA) copies between HBM and a ring of S stages in the warp's own
// shared memory: lanes read their values there, overwrite them with the results,
// and one lane sends the stage back. Warps never wait for one another; dw is
// summed in registers and joined over the CTA's groups at the end, in group order,
// one partial row a CTA (a CTA has turns of q alone or of k alone).
//
// A lane's unit is two times eight values, A and B:
//   * kHalves (ROPE_HALF, R a multiple of 16): a 16-byte vector of the first half
//     and the vector of its partners R/2 values on; beyond the turned part two vectors.
//   * kNeighbours (ROPE_INTERLEAVED): two vectors.
//   * kHalvesAny (ROPE_HALF, any R): as kHalves, but the turned B lies at any even
//     number of bytes, and both may be cut short by the half's end. Beyond the turned
//     part the vectors are counted from the row's end; what is left between, two
//     values a lane.
//   * kHalves8 (ROPE_HALF, R a multiple of 8): the same in whole steps of 8 bytes.
#pragma once

#include <algorithm>
#include <type_traits>

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
__device__ __forceinline__ void sts128(uint32_t p, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t p, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(p), "r"(v) : "memory"); }
__device__ __forceinline__ void sts16(uint32_t p, uint32_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(p), "h"(static_cast<uint16_t>(v)) : "memory");
}

// Two values of a word.
template <bool F16>
__device__ __forceinline__ float2 widen2(uint32_t v) {
    if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&v));
    else return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <bool F16>
__device__ __forceinline__ uint32_t narrow2(float2 v) {
    uint32_t w;
    if constexpr (F16) *reinterpret_cast<__half2*>(&w) = __floats2half2_rn(v.x, v.y);
    else *reinterpret_cast<__nv_bfloat162*>(&w) = __floats2bfloat162_rn(v.x, v.y);
    return w;
}

// Eight values at any even address, through the words that hold them (the first n
// are wanted; no word without one of them is read).
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

// The first n of eight values to any even address: whole words, and the half words
// at the ends, which may share theirs with another lane's values.
__device__ __forceinline__ void sts_window(uint32_t p, uint4 v, int n) {
    const uint32_t w[5] = {v.x, v.y, v.z, v.w, 0u};
    if ((p & 2u) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (2 * i + 1 < n) sts32(p + 4 * i, w[i]);
            else if (2 * i < n) sts16(p + 4 * i, w[i]);
        }
    } else {
        if (n > 0) sts16(p, w[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // values 2 i + 1 and 2 i + 2
            if (2 * i + 2 < n) sts32(p + 4 * i + 2, __funnelshift_r(w[i], w[i + 1], 16));
            else if (2 * i + 1 < n) sts16(p + 4 * i + 2, w[i] >> 16);
        }
    }
}

// The first n (even) of eight values at an address of whole words, zeros beyond.
__device__ __forceinline__ uint4 lds_words(uint32_t p, int n) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (n > 0) v.x = lds32(p);
    if (n > 2) v.y = lds32(p + 4);
    if (n > 4) v.z = lds32(p + 8);
    if (n > 6) v.w = lds32(p + 12);
    return v;
}
__device__ __forceinline__ void sts_words(uint32_t p, uint4 v, int n) {
    if (n > 0) sts32(p, v.x);
    if (n > 2) sts32(p + 4, v.y);
    if (n > 4) sts32(p + 8, v.z);
    if (n > 6) sts32(p + 12, v.w);
}

// Four (n > 0) or eight (n > 4) values at an address of whole 8 bytes, zeros beyond.
__device__ __forceinline__ uint4 lds_window8(uint32_t p, int n) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (n > 0) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p) : "memory");
    if (n > 4) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.z), "=r"(v.w) : "r"(p + 8) : "memory");
    return v;
}
__device__ __forceinline__ void sts_window8(uint32_t p, uint4 v, int n) {
    if (n > 0) asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(p), "r"(v.x), "r"(v.y) : "memory");
    if (n > 4) asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(p + 8), "r"(v.z), "r"(v.w) : "memory");
}

// 1-D bulk copy shared -> global, in the thread's current bulk group.
__device__ __forceinline__ void bulk_s2g(void* dst, uint32_t src, uint32_t bytes, uint64_t policy) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group.L2::cache_hint [%0], [%1], %2, %3;"
                 ::"l"(dst), "r"(src), "r"(bytes), "l"(policy) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// All but the N newest of the thread's bulk groups have read their shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

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
__device__ __forceinline__ uint4 keep_if(bool k, uint4 v) {
    return make_uint4(k ? v.x : 0u, k ? v.y : 0u, k ? v.z : 0u, k ? v.w : 0u);
}

// The first n of eight 16-bit values, zeros beyond.
__device__ __forceinline__ uint4 first_of(uint4 v, int n) {
    if (n < 8) {
        auto word = [n](uint32_t w, int i) { return 2 * i + 1 < n ? w : 2 * i < n ? w & 0xffffu : 0u; };
        v = make_uint4(word(v.x, 0), word(v.y, 1), word(v.z, 2), word(v.w, 3));
    }
    return v;
}

enum RopeKind : int { kHalves = 0, kNeighbours = 1, kHalvesAny = 2, kHalves8 = 3 };

// ---------------------------------------------------------------------------
// The kernel: 2^LG lanes a head, NR heads a group and turn, RB of them at a time.
// FULL: every lane has a whole unit (D = 16 x 2^LG, no unit cut short).
// MANY: a turn is of a token a group.
// ---------------------------------------------------------------------------
template <int MODE, int KIND, bool F16, int LG, bool FULL, bool MANY, int NR, int RBATCH, int S, int MINB>
__global__ void __launch_bounds__(kRopeThreads, MINB) rope_kernel(const RopeArgs a) {
    constexpr bool NORM = MODE != kTurn, BWD = MODE == kNormTurnBwd;
    constexpr bool ANY = KIND == kHalvesAny || KIND == kHalves8;  // units may be cut short
    constexpr int OPS = BWD ? 2 : 1, per = 32 >> LG, rows = per * NR;
    static_assert(NR % RBATCH == 0 && RBATCH <= 2 && !(FULL && ANY), "whole batches; cut units are not full");
    // A turn's heads: of one token, group g taking the i-th g + i per; or of per tokens, one a group.
    constexpr int tokens = MANY ? per : 1, step = MANY ? NR : rows, spread = MANY ? 1 : per;
    extern __shared__ __align__(128) unsigned char smem[];
    const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
    const int D = FULL ? 16 << LG : a.D, half = a.R >> 1, hp = (half + 7) & ~7;
    const int l = lane & ((1 << LG) - 1), head = lane >> LG;
    const uint32_t pitch = static_cast<uint32_t>(D) * 2u;
    const uint32_t op_bytes = rows * pitch, stage_bytes = OPS * op_bytes;
    // Shared memory: every warp's stages; weights [q | k][D]; every warp's [cos | sin][hp];
    // every warp's inverse RMS [S][rows] (read backward, gathered forward); barriers; frequencies.
    float* wsm = reinterpret_cast<float*>(smem + static_cast<size_t>(nw) * S * stage_bytes);
    float* cs = wsm + (NORM ? 2 * D : 0) + warp * 2 * hp;
    float* rs = wsm + (NORM ? 2 * D : 0) + nw * 2 * hp + (NORM ? warp * S * rows : 0);
    uint64_t* bars = reinterpret_cast<uint64_t*>(wsm + (NORM ? 2 * D : 0) + nw * 2 * hp + (NORM ? nw * S * rows : 0));
    unsigned long long* F = reinterpret_cast<unsigned long long*>(bars + nw * S);
    uint64_t* full = bars + warp * S;
    const uint32_t ring = smem_u32(smem) + warp * S * stage_bytes;

    // This lane's unit: where A and B lie in a row (in values), and how many of
    // their eight values there are.
    const int NC = D >> 3;
    const int NP = KIND == kNeighbours ? 0 : ANY ? (half + 7) >> 3 : half >> 3;  // units of the halves
    const int NV = ANY ? min((D - a.R) >> 3, 2 * ((1 << LG) - NP)) : 0;  // ANY: vectors at the row's end, not turned
    const bool turned = l < NP;
    int atA, atB, nA = 8, nB = 8;
    if (turned) {
        atA = 8 * l;
        atB = half + 8 * l;
        if constexpr (ANY) nA = nB = min(8, half - 8 * l);
    } else if constexpr (ANY) {
        const int c = l - NP, rest = (NV + 1) >> 1;
        atA = D - 8 * (NV - c);
        atB = D - 8 * (NV - rest - c);
        nA = c < rest ? 8 : 0;
        nB = c + rest < NV ? 8 : 0;
    } else {
        const int rest = (NC - 2 * NP + 1) >> 1, c = l + NP;  // 2 NP + (l - NP)
        atA = 8 * c;
        atB = 8 * (c + rest);
        if constexpr (!FULL) {
            if (l >= NP + rest) nA = 0;
            if (nA == 0 || c + rest >= NC) nB = 0;
        }
    }
    if constexpr (!FULL) {  // no address of a unit that is not there
        if (nA == 0) atA = 0;
        if (nB == 0) atB = 0;
    }
    const bool hasA = FULL || nA > 0, hasB = FULL || nB > 0;
    // ANY: two values between the halves and those vectors, if there are any for this lane.
    const int atX = a.R + 2 * l;
    const bool hasX = ANY && NORM && atX < D - 8 * NV;
    const uint32_t rowA = 2u * atA, rowB = 2u * atB, rowX = 2u * atX;
    // kNeighbours: pairs of A and of B that are turned (past 4: all).
    const int tA = hasA ? half - (atA >> 1) : 0, tB = hasB ? half - (atB >> 1) : 0;

    for (int i = tid; i < nw * S; i += nt) mbar_init(&bars[i], 1);
    fence_mbar_init();
    pdl_wait();
    __syncthreads();  // the barriers

    // Rows come and go once: out of L2 first, both ways (stores at the default
    // priority measured 1 to 3 % slower, loads at the ordinary one 0 to 4 %).
    const uint64_t pol = policy_evict_first();
    const bool words = (half & 1) == 0;  // kHalvesAny: B lies at whole words
    auto loadA = [&](uint32_t at) -> uint4 {
        if constexpr (KIND == kHalves8) return lds_window8(at, nA);
        const uint4 v = lds128(at);
        if constexpr (ANY) return NORM ? first_of(v, nA) : v;
        else return FULL ? v : keep_if(hasA, v);
    };
    auto loadB = [&](uint32_t at) -> uint4 {
        if constexpr (KIND == kHalvesAny) {
            if (words) return lds_words(at, nB);
            const uint4 v = lds_window(at, nB);
            return NORM ? first_of(v, nB) : v;
        } else if constexpr (KIND == kHalves8) {
            return lds_window8(at, nB);
        } else {
            return FULL ? lds128(at) : keep_if(hasB, lds128(at));
        }
    };
    auto storeA = [&](uint32_t at, const Oct& o) {
        const uint4 v = oct_pack<F16>(o);
        if constexpr (KIND == kHalves8) sts_window8(at, v, nA);
        else if (FULL || nA == 8) sts128(at, v);
        else if constexpr (KIND == kHalvesAny) sts_window(at, v, nA);
    };
    auto storeB = [&](uint32_t at, const Oct& o) {
        const uint4 v = oct_pack<F16>(o);
        if constexpr (KIND == kHalves8) {
            sts_window8(at, v, nB);
        } else if constexpr (KIND == kHalvesAny) {
            if (words) sts_words(at, v, nB);
            else sts_window(at, v, nB);
        } else if (FULL || nB == 8) {
            sts128(at, v);
        }
    };
    uint32_t phase = 0;  // of the stage that comes next
    int cur = 0;
    // Forward: every warp takes turns of q and of k. Backward: the first a.ctas_q
    // CTAs take those of q, the others those of k, for one weight's gradient each.
    const bool of_k = BWD && static_cast<int>(blockIdx.x) >= a.ctas_q;
    const int Hq = of_k ? 0 : a.H[0], Hk = BWD && !of_k ? 0 : a.H[1];
    const int cta = blockIdx.x - (of_k ? a.ctas_q : 0);
    const int ctas = !BWD ? gridDim.x : of_k ? gridDim.x - a.ctas_q : a.ctas_q;
    Turns now((a.T + tokens - 1) / tokens, (Hq + step - 1) / step, (Hk + step - 1) / step, step, static_cast<int64_t>(cta) * nw + warp,
              static_cast<int64_t>(ctas) * nw);
    Turns ahead = now;
    // Place of row r (n heads a token) among the heads of all tokens.
    auto in_tokens = [](int r, int n, int H) { return n == H ? r : r / n * H + r % n; };
    // The copies of a turn, one a lane: a token's heads where they lie side by side, else a head.
    auto pieces = [&](bool dense, int64_t token, int64_t head_stride, int64_t t0, int h, int n, int tk, uint32_t bytes, auto&& copy) {
        if (dense) {
            if (lane < tk) copy((t0 + lane) * token + h * head_stride, lane * n * pitch, n * pitch);
        } else if (lane < tk * n) {
            const int j = MANY ? lane / n : 0;
            copy((t0 + j) * token + (h + lane - j * n) * head_stride, lane * pitch, bytes);
        }
    };
    int fs = 0;
    auto fetch = [&]() {
        if (ahead.left > 0) {
            const int s = ahead.s, n = min(step, a.H[s] - ahead.h);
            const int64_t t0 = static_cast<int64_t>(ahead.t) * tokens;
            const int tk = MANY ? static_cast<int>(min(static_cast<int64_t>(tokens), a.T - t0)) : 1;
            const uint32_t bytes = a.row_bytes[s];
            if (lane == 0) mbar_arrive_expect_tx(&full[fs], static_cast<uint32_t>(tk * n) * OPS * bytes);
            __syncwarp();  // and every lane's copies out of the stage have read it
            unsigned char* to = smem + static_cast<size_t>(warp * S + fs) * stage_bytes;
#pragma unroll
            for (int op = 0; op < OPS; ++op) {
                const HeadsIn& in = op ? a.x[s] : a.in[s];
                pieces(a.dense[op][s], in.token, in.head, t0, ahead.h, n, tk, bytes, [&](int64_t from, uint32_t at, uint32_t size) {
                    bulk_g2s(to + op * op_bytes + at, in.p + from, size, &full[fs], pol);
                });
            }
            if constexpr (BWD) {
                const float* p = a.rstd[s] + t0 * a.H[s] + ahead.h;
#pragma unroll
                for (int i = 0; i < rows; i += 32)
                    if (i + lane < tk * n) cp_async4(rs + fs * rows + i + lane, p + (MANY ? in_tokens(i + lane, n, a.H[s]) : i + lane));
            }
            ahead.next(Hq, Hk, step);
        }
        if constexpr (BWD) cp_async_commit();
        fs = fs + 1 == S ? 0 : fs + 1;
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch();
    // While the first rows come:
    for (int i = half + lane; i < hp; i += 32) cs[i] = cs[hp + i] = 0.0f;  // zeros are turned there
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
    long long p32 = 0;  // lane i: the position of token t32 + i
    int64_t t32 = -32;
    Oct accA = oct_zero(), accB = oct_zero(), wA = oct_zero(), wB = oct_zero();
    float2 accX = make_float2(0.0f, 0.0f), wX = accX;
    Oct c = oct_zero(), sn = oct_zero();  // cos and sin of this lane's pairs (kNeighbours: four of A, four of B)
    int t_have = -1, s_have = -1;
    while (now.left > 0) {
        const int64_t t0 = static_cast<int64_t>(now.t) * tokens;
        if (now.t != t_have) {
            t_have = now.t;
            if (t0 - t32 >= 32) {
                t32 = t0;
                if (t32 + lane < a.T) p32 = position(a, t32 + lane);
            }
            const long long pos = __shfl_sync(0xffffffffu, p32, static_cast<int>(t0 - t32) + (MANY ? head : 0));
            if constexpr (!MANY) token_angles(cs, hp, half, F, pos, a.scale, BWD || a.back, lane);
            if constexpr (MANY) {  // this lane's own
                if (KIND == kNeighbours || turned) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int pair = KIND == kNeighbours ? ((e < 4 ? atA : atB) >> 1) + (e & 3) : atA + e;
                        float2 v = rope_cos_sin(pos, F[min(pair, half - 1)], a.scale);
                        if (BWD || a.back) v.y = -v.y;
                        if (e & 1) {
                            c.p[e / 2].y = v.x;
                            sn.p[e / 2].y = v.y;
                        } else {
                            c.p[e / 2].x = v.x;
                            sn.p[e / 2].x = v.y;
                        }
                    }
                }
            } else if constexpr (KIND == kNeighbours) {
                const float4* q = reinterpret_cast<const float4*>(cs);
                const int iA = min(atA >> 3, (hp >> 2) - 1), iB = min(atB >> 3, (hp >> 2) - 1);
                c = oct_of(q[iA], q[iB]);
                sn = oct_of(q[(hp >> 2) + iA], q[(hp >> 2) + iB]);
            } else if (turned) {
                const float4* q = reinterpret_cast<const float4*>(cs + atA);
                c = oct_of(q[0], q[1]);
                sn = oct_of(q[hp >> 2], q[(hp >> 2) + 1]);
            }
        }
        const int s = now.s;
        if (NORM && s != s_have) {
            s_have = s;
            const float* w = wsm + s * D;
            if constexpr (!ANY) {
                const float4 *p = reinterpret_cast<const float4*>(w + atA), *q = reinterpret_cast<const float4*>(w + atB);
                wA = oct_of(p[0], p[1]);
                wB = oct_of(q[0], q[1]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    wA.p[i] = make_float2(2 * i < nA ? w[atA + 2 * i] : 0.0f, 2 * i + 1 < nA ? w[atA + 2 * i + 1] : 0.0f);
                    wB.p[i] = make_float2(2 * i < nB ? w[atB + 2 * i] : 0.0f, 2 * i + 1 < nB ? w[atB + 2 * i + 1] : 0.0f);
                }
                if (hasX) wX = *reinterpret_cast<const float2*>(w + atX);
            }
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
        // Heads and tokens of this turn; what is computed of others is sent nowhere.
        const int n = min(step, a.H[s] - now.h);
        const int tk = MANY ? static_cast<int>(min(static_cast<int64_t>(tokens), a.T - t0)) : 1, there = tk * n;
        const int row0 = MANY ? head * n : head;
        if constexpr (BWD) {  // a head that is not there adds zeros to the weight gradients
            const int last = MANY ? per * n : min(rows, (n + per * RBATCH - 1) / (per * RBATCH) * (per * RBATCH));
            if (there < last) {
                for (int i = there * (D >> 3) + lane; i < last * (D >> 3); i += 32) {
                    sts128(st + 16 * i, make_uint4(0, 0, 0, 0));
                    sts128(st + op_bytes + 16 * i, make_uint4(0, 0, 0, 0));
                }
                for (int i = there + lane; i < last; i += 32) rs[cur * rows + i] = 0.0f;
                __syncwarp();
            }
        }
        auto turn = [&](Oct& A, Oct& B) {
            if constexpr (KIND == kNeighbours) {
                const float2 c0[2] = {c.p[0], c.p[1]}, c1[2] = {c.p[2], c.p[3]}, s0[2] = {sn.p[0], sn.p[1]}, s1[2] = {sn.p[2], sn.p[3]};
                if (tA > 0) turn_neighbours(A, c0, s0, tA);
                if (tB > 0) turn_neighbours(B, c1, s1, tB);
            } else if (turned) {
                turn_halves(A, B, c, sn);
            }
        };
        // A batch of RB heads a group, from the i0-th on.
        auto batch = [&](auto count, const int i0) {
            constexpr int RB = decltype(count)::value;
            const uint32_t at = st + (row0 + i0 * spread) * pitch;
            uint4 rawA[RB], rawB[RB];
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const uint32_t p = at + i * spread * pitch;
                if (NORM || KIND == kNeighbours || turned) {
                    rawA[i] = loadA(p + rowA);
                    rawB[i] = loadB(p + rowB);
                }
            }
            if constexpr (MODE == kTurn) {
                if constexpr (ANY) __syncwarp();  // windows share words: all are read before any is written
#pragma unroll
                for (int i = 0; i < RB; ++i) {
                    const uint32_t p = at + i * spread * pitch;
                    if constexpr (KIND == kNeighbours) {
                        // What is not turned stays where it is, or keeps its bits.
                        Oct A = oct_unpack<F16>(rawA[i]), B = oct_unpack<F16>(rawB[i]);
                        turn(A, B);
                        auto put = [&](uint32_t q, const Oct& o, const uint4& raw, int t) {
                            uint4 v = oct_pack<F16>(o);
                            if (t < 4) {
                                if (t < 2) v.y = raw.y;
                                if (t < 3) v.z = raw.z;
                                v.w = raw.w;
                            }
                            if (t > 0) sts128(q, v);
                        };
                        put(p + rowA, A, rawA[i], tA);
                        put(p + rowB, B, rawB[i], tB);
                    } else if (turned) {
                        Oct A = oct_unpack<F16>(rawA[i]), B = oct_unpack<F16>(rawB[i]);
                        turn(A, B);
                        storeA(p + rowA, A);
                        storeB(p + rowB, B);
                    }
                }
            } else {
                Oct A[RB], B[RB], xA[RB], xB[RB];
                float sum[RB], r[RB];
                float2 X[RB], xX[RB];
#pragma unroll
                for (int i = 0; i < RB; ++i) {
                    const uint32_t p = at + i * spread * pitch;
                    const int row = row0 + (i0 + i) * spread;
                    float2 sum2 = make_float2(0.0f, 0.0f);
                    r[i] = 0.0f;
                    X[i] = xX[i] = make_float2(0.0f, 0.0f);
                    if (hasX) X[i] = widen2<F16>(lds32(p + rowX));
                    if constexpr (BWD) {
                        A[i] = oct_unpack<F16>(rawA[i]);
                        B[i] = oct_unpack<F16>(rawB[i]);
                        xA[i] = oct_unpack<F16>(loadA(p + op_bytes + rowA));
                        xB[i] = oct_unpack<F16>(loadB(p + op_bytes + rowB));
                        r[i] = rs[cur * rows + row];
                        turn(A[i], B[i]);
                        if (hasX) {
                            xX[i] = widen2<F16>(lds32(p + op_bytes + rowX));
                            accX = fma2(X[i], fmul2(xX[i], both(r[i])), accX);
                            X[i] = fmul2(X[i], wX);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            accA.p[e] = fma2(A[i].p[e], fmul2(xA[i].p[e], both(r[i])), accA.p[e]);
                            accB.p[e] = fma2(B[i].p[e], fmul2(xB[i].p[e], both(r[i])), accB.p[e]);
                            A[i].p[e] = fmul2(A[i].p[e], wA.p[e]);
                            B[i].p[e] = fmul2(B[i].p[e], wB.p[e]);
                            sum2 = fma2(A[i].p[e], xA[i].p[e], sum2);
                            sum2 = fma2(B[i].p[e], xB[i].p[e], sum2);
                        }
                        if constexpr (ANY) sum2 = fma2(X[i], xX[i], sum2);
                        sum[i] = fadd(sum2.x, sum2.y);
                    } else {
                        A[i] = oct_unpack<F16>(rawA[i]);
                        B[i] = oct_unpack<F16>(rawB[i]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            sum2 = fma2(A[i].p[e], A[i].p[e], sum2);
                            sum2 = fma2(B[i].p[e], B[i].p[e], sum2);
                        }
                        if constexpr (ANY) sum2 = fma2(X[i], X[i], sum2);
                        sum[i] = fadd(sum2.x, sum2.y);
                    }
                }
                if constexpr (ANY) __syncwarp();  // windows share words: all are read before any is written
#pragma unroll
                for (int i = 0; i < RB; ++i) sum[i] = group_sum<(1 << LG)>(sum[i]);
#pragma unroll
                for (int i = 0; i < RB; ++i) {
                    const uint32_t p = at + i * spread * pitch;
                    if constexpr (BWD) {
                        // r with the sum, r^2 apart: r^3 leaves fp32's range long before the result does.
                        const float coef = -fmul(fmul(r[i], r[i]), fmul(fmul(sum[i], r[i]), a.rcp_d));
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            A[i].p[e] = fma2(A[i].p[e], both(r[i]), fmul2(xA[i].p[e], both(coef)));
                            B[i].p[e] = fma2(B[i].p[e], both(r[i]), fmul2(xB[i].p[e], both(coef)));
                        }
                        if (hasX) sts32(p + rowX, narrow2<F16>(fma2(X[i], both(r[i]), fmul2(xX[i], both(coef)))));
                    } else {
                        r[i] = rsqrtf(fadd(fmul(sum[i], a.rcp_d), a.eps));
                        if (l == 0) rs[cur * rows + row0 + (i0 + i) * spread] = r[i];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            A[i].p[e] = fmul2(fmul2(A[i].p[e], both(r[i])), wA.p[e]);
                            B[i].p[e] = fmul2(fmul2(B[i].p[e], both(r[i])), wB.p[e]);
                        }
                        turn(A[i], B[i]);
                        if (hasX) sts32(p + rowX, narrow2<F16>(fmul2(fmul2(X[i], both(r[i])), wX)));
                    }
                    storeA(p + rowA, A[i]);
                    storeB(p + rowB, B[i]);
                }
            }
        };
#pragma unroll
        for (int i0 = 0; i0 < NR; i0 += RBATCH) {
            const int rest = n - i0 * spread;
            if (rest <= 0) break;  // the same for all lanes
            if (RBATCH > 1 && rest <= spread) batch(std::integral_constant<int, 1>(), i0);
            else batch(std::integral_constant<int, RBATCH>(), i0);
        }
        fence_proxy_async_smem();  // the results, before the copy that sends them and the one that refills the stage
        __syncwarp();
        const HeadsOut& o = a.out[s];
        pieces(a.dense[2][s], o.token, o.head, t0, now.h, n, tk, a.row_bytes[s],
               [&](int64_t to, uint32_t at, uint32_t size) { bulk_s2g(o.p + to, st + at, size, pol); });
        bulk_commit();
        bulk_wait_read<1>();  // the stage of the turn before is sent: it is filled next
        if constexpr (NORM && !BWD) {
            float* p = a.rstd[s] + t0 * a.H[s] + now.h;
#pragma unroll
            for (int i = 0; i < rows; i += 32)
                if (i + lane < there) p[MANY ? in_tokens(i + lane, n, a.H[s]) : i + lane] = rs[cur * rows + i + lane];
        }
        if (++cur == S) {
            cur = 0;
            phase ^= 1u;
        }
        now.next(Hq, Hk, step);
        fetch();
    }
    bulk_wait_all();
    if constexpr (BWD) {
        cp_async_wait<0>();
        // The groups' sums in group order, through the stages' memory.
        float* part = reinterpret_cast<float*>(smem);  // [groups][D]
        const int groups = nt >> LG, group = tid >> LG;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e < nA) part[group * D + atA + e] = e & 1 ? accA.p[e / 2].y : accA.p[e / 2].x;
            if (e < nB) part[group * D + atB + e] = e & 1 ? accB.p[e / 2].y : accB.p[e / 2].x;
        }
        if (hasX) *reinterpret_cast<float2*>(part + group * D + atX) = accX;
        __syncthreads();
        float* row = a.partials + static_cast<int64_t>(blockIdx.x) * D;
        for (int col = tid; col < D; col += nt) {
            float v = part[col];
            for (int g = 1; g < groups; ++g) v = fadd(v, part[g * D + col]);
            row[col] = v;
        }
    }
    pdl_release();
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
template <int MODE, int KIND, bool F16, int LG, bool FULL, bool MANY, int NR, int RB, int S, int MINB>
cudaError_t rope_run_as(const RopeArgs& a, int* ctas_q, cudaStream_t st) {
    constexpr bool NORM = MODE != kTurn, BWD = MODE == kNormTurnBwd;
    constexpr int per = 32 >> LG, rows = per * NR, tokens = MANY ? per : 1, step = MANY ? NR : rows;
    const auto kern = rope_kernel<MODE, KIND, F16, LG, FULL, MANY, NR, RB, S, MINB>;
    const int hp = (a.R / 2 + 7) & ~7;
    const size_t warp_bytes = static_cast<size_t>(S) * (BWD ? 2 : 1) * rows * a.D * 2 + hp * 8 + (NORM ? S * rows * 4 : 0) + S * 8;
    const size_t fixed = (NORM ? static_cast<size_t>(a.D) * 8 : 0) + static_cast<size_t>(a.R / 2) * 8;
    const int64_t sms = sm_count();
    const int64_t turns = (a.T + tokens - 1) / tokens * ((a.H[0] + step - 1) / step + (a.H[1] + step - 1) / step);
    // Threads: few turns spread over the SMs in smaller CTAs. The backward's CTAs
    // are a function of the problem (rope_bwd_ctas).
    int threads = kRopeThreads;
    if (!BWD)
        while (threads > 32 && turns * 32 < sms * threads) threads /= 2;
    size_t smem = warp_bytes * (threads / 32) + fixed;
    if (BWD) smem = std::max(smem, static_cast<size_t>(threads >> LG) * a.D * 4);
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    int64_t grid = rope_bwd_ctas(a.T, a.H[0], a.H[1], a.D);
    if (!BWD) {
        const int occ = ctas_per_sm(reinterpret_cast<const void*>(kern), threads, static_cast<int>(smem));
        if (occ < 1) return cudaErrorInvalidConfiguration;
        grid = std::min<int64_t>((turns + threads / 32 - 1) / (threads / 32), sms * occ);
    }
    RopeArgs b = a;
    if (BWD && a.H[1] > 0) {
        // The CTAs split by the work of a token (MANY: of as many): one for a batch of
        // heads, four for a turn, whose chain of waits counts most (32 + 8 heads of 64:
        // 76 % of the copy rate; by batches alone 64 %, by turns alone 73 %). MANY: two
        // a turn and two for the angles that each lane computes (4 + 1 heads of 128:
        // 57 %; by four and four a point less, 14 + 2 heads 81 and 80).
        auto cost = [&](int64_t H) {
            constexpr int64_t batch = MANY ? RB : per * RB;
            return H / step * (NR / RB) + (H % step + batch - 1) / batch + (MANY ? 2 : 4) * ((H + step - 1) / step) + (MANY ? 2 : 0);
        };
        const int64_t q = cost(a.H[0]), k = cost(a.H[1]);
        b.ctas_q = static_cast<int>(std::min(std::max<int64_t>((grid * q + (q + k) / 2) / (q + k), 1), grid - 1));
    } else {
        b.ctas_q = static_cast<int>(grid);
    }
    *ctas_q = b.ctas_q;
    return launch_kernel(kern, static_cast<unsigned>(grid), threads, smem, st, b);
}

// One token a turn or one a group of lanes: the second where it leaves half the
// turns or fewer at as many heads a group (the norm's kernels, with more to do a
// turn: three quarters), and still kRopeManyFrom turns. 65536 x 4 + 1 x 128:
// rotation 48 -> 79 % of the copy rate, norm and rotation 33 -> 67, its backward
// 32 -> 57; 14 + 2 heads: 88 both ways, 55 -> 79, 46 -> 81. With as many turns
// (32 + 8 heads of 128) its shorter copies cost: 83 -> 80, 76 -> 66, 75 -> 72,
// measured in one kernel for both.
template <int MODE, int KIND, bool F16, int LG, bool FULL, int NR, int RB, int S, int MINB>
cudaError_t rope_run_kernel(const RopeArgs& a, int* ctas_q, cudaStream_t st) {
    constexpr int per = 32 >> LG;
    if constexpr (per > 1) {
        // Forward with the norm: then four heads a group (8 + 1 heads of 128: 75 % for two heads' 58).
        constexpr bool wider = MODE == kNormTurn;
        auto turns_of = [&](int step) -> int64_t { return (a.H[0] + step - 1) / step + (a.H[1] + step - 1) / step; };
        const int64_t one = a.T * turns_of(per * NR), many = (a.T + per - 1) / per * turns_of(NR);
        const bool fewer = MODE == kTurn ? 2 * many <= one : 4 * many <= 3 * one;
        if (fewer && many >= kRopeManyFrom)
            return rope_run_as<MODE, KIND, F16, LG, FULL, true, wider ? 4 : NR, wider ? 2 : RB, wider ? 3 : S, MINB>(a, ctas_q, st);
    }
    return rope_run_as<MODE, KIND, F16, LG, FULL, false, NR, RB, S, MINB>(a, ctas_q, st);
}

// Heads a group and turn, of them in registers at a time, stages, CTAs an SM: the
// fastest measured of each kind. More heads a turn cost fewer turns' waits and
// more shared memory, which has to leave room for two CTAs an SM. Some kernels
// spill: most backward ones of several tokens whose heads leave lanes idle or are
// cut (4 to 56 bytes at 128 registers), two forward ones with the norm (4 bytes),
// and of the rotation those of neighbours in fp16 and of several tokens (4 to 20
// bytes at 80 registers, three CTAs an SM).
template <int MODE, int KIND, bool F16, int LG, bool FULL>
cudaError_t rope_shape_of(const RopeArgs& a, int* ctas_q, cudaStream_t st) {
    if constexpr (MODE == kTurn) {
        return rope_run_kernel<MODE, KIND, F16, LG, FULL, 4, 1, 2, 3>(a, ctas_q, st);
    } else if constexpr (MODE == kNormTurn) {
        // 16384 x 32 + 8 x 128: 84 % of the copy rate (with 4 heads 80); 80 wide: 78 % (with 2 heads 61).
        if constexpr (FULL && LG < 5) return rope_run_kernel<MODE, KIND, F16, LG, FULL, 2, 1, 3, 2>(a, ctas_q, st);
        else return rope_run_kernel<MODE, KIND, F16, LG, FULL, 4, 2, 3, 2>(a, ctas_q, st);
    } else if constexpr (LG == 5) {
        return rope_run_kernel<MODE, KIND, F16, LG, FULL, 2, 1, 2, 2>(a, ctas_q, st);  // 3 heads: one CTA an SM, 58 % for 76
    } else if constexpr (FULL && LG != 3) {
        return rope_run_kernel<MODE, KIND, F16, LG, FULL, 2, 1, 3, 2>(a, ctas_q, st);
    } else {
        if constexpr (!FULL)  // narrower than its lanes could hold: four heads fit (80 wide: 70 % for 62)
            if (4 * a.D <= 3 * (16 << LG)) return rope_run_kernel<MODE, KIND, F16, LG, FULL, 4, 1, 2, 2>(a, ctas_q, st);
        return rope_run_kernel<MODE, KIND, F16, LG, FULL, 3, 1, 2, 2>(a, ctas_q, st);
    }
}

template <int MODE, int KIND, bool F16, int LG>
cudaError_t rope_full(const RopeArgs& a, int* ctas_q, cudaStream_t st) {
    if constexpr (KIND == kHalves || KIND == kNeighbours)
        if (a.D == 16 << LG) return rope_shape_of<MODE, KIND, F16, LG, true>(a, ctas_q, st);
    return rope_shape_of<MODE, KIND, F16, LG, false>(a, ctas_q, st);
}

template <int MODE, int KIND, bool F16>
cudaError_t rope_lanes(const RopeArgs& a, int* ctas_q, cudaStream_t st) {
    switch (rope_lanes_log2(a.D, a.R, KIND == kHalvesAny || KIND == kHalves8, MODE != kTurn)) {
        case 2: return rope_full<MODE, KIND, F16, 2>(a, ctas_q, st);
        case 3: return rope_full<MODE, KIND, F16, 3>(a, ctas_q, st);
        case 4: return rope_full<MODE, KIND, F16, 4>(a, ctas_q, st);
        default: return rope_full<MODE, KIND, F16, 5>(a, ctas_q, st);
    }
}

// *ctas_q: the CTAs (and so the partial rows) of q in a norm backward.
template <int MODE, bool F16>
cudaError_t rope_kinds(const RopeArgs& a, int* ctas_q, cudaStream_t st) {
    if (a.layout == ROPE_INTERLEAVED) return rope_lanes<MODE, kNeighbours, F16>(a, ctas_q, st);
    if (a.R % 16 == 0) return rope_lanes<MODE, kHalves, F16>(a, ctas_q, st);
    if (a.R % 8 == 0) return rope_lanes<MODE, kHalves8, F16>(a, ctas_q, st);
    return rope_lanes<MODE, kHalvesAny, F16>(a, ctas_q, st);
}

}  // namespace
}  // namespace rmsn
