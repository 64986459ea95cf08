// Rotary positions of q and k, alone and fused with the heads' RMSNorm, forward
// and backward: kernels and C-ABI entry points.
#include <algorithm>
#include <cmath>

#include "checks.h"
#include "common.cuh"
#include "kernels.h"
#include "reduce_columns.h"
#include "rope.h"
#include "rope_math.cuh"

namespace rmsn {
namespace {

constexpr int kMaxHeadD = 512;

enum RopeMode : int { kTurn = 0, kNormTurn = 1, kNormTurnBwd = 2 };

// A [T][H][D] tensor by its strides in elements.
struct HeadsIn { const uint16_t* p; int64_t token, head; };
struct HeadsOut { uint16_t* p; int64_t token, head; };

struct RopeArgs {
    HeadsIn in[2];       // q, k (forward) / gq, gk (backward)
    HeadsIn x[2];        // q, k of the forward (norm backward)
    HeadsOut out[2];
    const float* w[2];   // norm weights
    float* rstd[2];      // written by the forward, read by the backward
    float* partials;     // norm backward: [chunks][D] of dwq, then of dwk
    const double* inv_freq;
    const void* pos;     // null: the token's index
    int64_t T;
    int H[2];
    int D, R, layout, pos64, back, zc, chunk;
    float scale, eps;
};

constexpr int kRopeThreads = 128;

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

// A warp a head; lane l has the slots p = l, l + 32, ... of D/2. Slot p is two
// values: a pair of the rotation (p < R/2), or two neighbours of the rest.
template <int MODE, bool F16, int NJ>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
    constexpr bool NORM = MODE != kTurn, BWD = MODE == kNormTurnBwd;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = kRopeThreads / 32;
    const int D = a.D, NV = D >> 3, half = a.R >> 1;
    unsigned long long* F = reinterpret_cast<unsigned long long*>(smem);             // [half]
    float2* cs = reinterpret_cast<float2*>(F + half) + warp * half;                  // [warps][half]
    uint16_t* rows = reinterpret_cast<uint16_t*>(smem + (((half * 8 * (1 + nw)) + 15) & ~15));
    uint16_t* ri = rows + warp * 2 * D;                                              // [warps][2][D]
    uint16_t* rx = ri + D;
    pdl_wait();
    for (int i = threadIdx.x; i < half; i += kRopeThreads) F[i] = rope_turns(a.inv_freq[i]);
    __syncthreads();

    const int H = a.H[0] + a.H[1];
    const bool backward = BWD || a.back;
    float acc[2][NJ][2];  // weight gradients: q's and k's
    if constexpr (BWD)
        for (int s = 0; s < 2; ++s)
            for (int j = 0; j < NJ; ++j) acc[s][j][0] = acc[s][j][1] = 0.0f;
    const int64_t t0 = BWD ? static_cast<int64_t>(blockIdx.x) * a.chunk + warp : static_cast<int64_t>(blockIdx.x) * nw + warp;
    const int64_t t1 = BWD ? min(static_cast<int64_t>(blockIdx.x + 1) * a.chunk, a.T) : a.T;
    const int64_t step = BWD ? nw : static_cast<int64_t>(gridDim.x) * nw;
    for (int64_t t = t0; t < t1; t += step) {
        const long long p = position(a, t);
        for (int i = lane; i < half; i += 32) {
            float2 c = rope_cos_sin(p, F[i], a.scale);
            if (backward) c.y = -c.y;
            cs[i] = c;
        }
        __syncwarp();
        for (int h = 0; h < H; ++h) {
            const int s = h >= a.H[0];
            const int hh = s ? h - a.H[0] : h;
            const uint4* in = reinterpret_cast<const uint4*>(a.in[s].p + t * a.in[s].token + hh * a.in[s].head);
            const uint4* x = BWD ? reinterpret_cast<const uint4*>(a.x[s].p + t * a.x[s].token + hh * a.x[s].head) : nullptr;
            for (int v = lane; v < NV; v += 32) {
                reinterpret_cast<uint4*>(ri)[v] = in[v];
                if (BWD) reinterpret_cast<uint4*>(rx)[v] = x[v];
            }
            __syncwarp();
            float u[NJ][2], xs[NJ][2], w[NJ][2];
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int q = lane + 32 * j;
                if (2 * q < D) {
                    const bool turn = q < half;
                    const int i0 = turn && a.layout == ROPE_HALF ? q : 2 * q;
                    const int i1 = turn && a.layout == ROPE_HALF ? q + half : 2 * q + 1;
                    u[j][0] = widen<F16>(ri[i0]);
                    u[j][1] = widen<F16>(ri[i1]);
                    if (NORM) {
                        w[j][0] = a.w[s][i0];
                        w[j][1] = a.w[s][i1];
                        if (a.zc) {
                            w[j][0] = fadd(w[j][0], 1.0f);
                            w[j][1] = fadd(w[j][1], 1.0f);
                        }
                    }
                    if (BWD) {
                        xs[j][0] = widen<F16>(rx[i0]);
                        xs[j][1] = widen<F16>(rx[i1]);
                        if (turn) {
                            const float2 r = rope_turn(u[j][0], u[j][1], cs[q]);
                            u[j][0] = r.x;
                            u[j][1] = r.y;
                        }
                        for (int e = 0; e < 2; ++e) sum = fadd(sum, fmul(fmul(u[j][e], w[j][e]), xs[j][e]));
                    } else if (NORM) {
                        for (int e = 0; e < 2; ++e) sum = fadd(sum, fmul(u[j][e], u[j][e]));
                    }
                }
            }
            float r = 0.0f, coef = 0.0f;
            if (NORM) {
                sum = group_sum<32>(sum);
                float* rs = a.rstd[s] + t * a.H[s] + hh;
                if (BWD) {
                    r = *rs;
                    coef = fmul(__fdiv_rn(fmul(fmul(r, r), r), static_cast<float>(D)), sum);
                } else {
                    r = rsqrtf(fadd(__fdiv_rn(sum, static_cast<float>(D)), a.eps));
                    if (lane == 0) *rs = r;
                }
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int q = lane + 32 * j;
                if (2 * q < D) {
                    const bool turn = q < half;
                    const int i0 = turn && a.layout == ROPE_HALF ? q : 2 * q;
                    const int i1 = turn && a.layout == ROPE_HALF ? q + half : 2 * q + 1;
                    if (BWD) {
                        for (int e = 0; e < 2; ++e) {
                            const float g = u[j][e];
                            acc[s][j][e] = fadd(acc[s][j][e], fmul(fmul(g, xs[j][e]), r));
                            u[j][e] = fsub(fmul(fmul(g, w[j][e]), r), fmul(xs[j][e], coef));
                        }
                    } else {
                        if (NORM)
                            for (int e = 0; e < 2; ++e) u[j][e] = fmul(fmul(u[j][e], r), w[j][e]);
                        if (turn) {
                            const float2 o = rope_turn(u[j][0], u[j][1], cs[q]);
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
            uint4* out = reinterpret_cast<uint4*>(a.out[s].p + t * a.out[s].token + hh * a.out[s].head);
            for (int v = lane; v < NV; v += 32) out[v] = reinterpret_cast<const uint4*>(ri)[v];
            __syncwarp();
        }
    }
    if constexpr (BWD) {
        // The warps' sums, added in warp order.
        __syncthreads();
        float* sum = reinterpret_cast<float*>(smem);  // [2][D]
        for (int k = 0; k < nw; ++k) {
            if (warp == k)
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const int q = lane + 32 * j;
                        if (2 * q < D) {
                            const bool hl = q < half && a.layout == ROPE_HALF;
                            float* o0 = sum + s * D + (hl ? q : 2 * q);
                            float* o1 = sum + s * D + (hl ? q + half : 2 * q + 1);
                            *o0 = k == 0 ? acc[s][j][0] : fadd(*o0, acc[s][j][0]);
                            *o1 = k == 0 ? acc[s][j][1] : fadd(*o1, acc[s][j][1]);
                        }
                    }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < 2 * D; i += kRopeThreads) {
            const int s = i >= D;
            if (a.H[s] > 0) a.partials[(static_cast<int64_t>(s) * gridDim.x + blockIdx.x) * D + (s ? i - D : i)] = sum[i];
        }
    }
    pdl_release();
}

template <int MODE, bool F16, int NJ>
cudaError_t rope_launch(const RopeArgs& a, unsigned grid, cudaStream_t st) {
    const int nw = kRopeThreads / 32, half = a.R / 2;
    size_t smem = ((half * 8 * (1 + nw) + 15) & ~15) + static_cast<size_t>(nw) * 2 * a.D * 2;
    smem = std::max<size_t>(smem, static_cast<size_t>(a.D) * 8);
    return launch_kernel(rope_kernel<MODE, F16, NJ>, grid, kRopeThreads, smem, st, a);
}

template <int MODE, bool F16>
cudaError_t rope_width(const RopeArgs& a, unsigned grid, cudaStream_t st) {
    if (a.D <= 64) return rope_launch<MODE, F16, 1>(a, grid, st);
    if (a.D <= 128) return rope_launch<MODE, F16, 2>(a, grid, st);
    if (a.D <= 256) return rope_launch<MODE, F16, 4>(a, grid, st);
    return rope_launch<MODE, F16, 8>(a, grid, st);
}

template <int MODE>
cudaError_t rope_run(const RopeArgs& a, int flags, unsigned grid, cudaStream_t st) {
    return flags ? rope_width<MODE, true>(a, grid, st) : rope_width<MODE, false>(a, grid, st);
}

unsigned rope_grid(int64_t T) {
    return static_cast<unsigned>(std::min<int64_t>((T + 3) / 4, static_cast<int64_t>(sm_count()) * 8));
}

constexpr int64_t kRopeChunks = 608;
int64_t rope_chunk(int64_t T) { return std::max<int64_t>(1, (T + kRopeChunks - 1) / kRopeChunks); }
int64_t rope_chunks(int64_t T) { return (T + rope_chunk(T) - 1) / rope_chunk(T); }

// ---------------------------------------------------------------------------
// Argument checks
// ---------------------------------------------------------------------------
int check_sizes(int64_t T, int64_t Hq, int64_t Hk, int64_t D) {
    if (T < 0 || T >= (int64_t(1) << 31)) return RMSN_EINVAL;
    if (Hq < 1 || Hk < 0 || Hq > 65536 || Hk > 65536) return RMSN_EINVAL;
    if (D < 8 || D > kMaxHeadD || D % 8 != 0) return RMSN_EUNSUPPORTED;
    return RMSN_OK;
}

int check_rope(int64_t D, int64_t R, float scale, int layout, int pos_dtype) {
    if (layout != ROPE_HALF && layout != ROPE_INTERLEAVED) return RMSN_EINVAL;
    if (pos_dtype != ROPE_POS_I32 && pos_dtype != ROPE_POS_I64) return RMSN_EINVAL;
    if (!std::isfinite(scale)) return RMSN_EINVAL;
    if (R < 2 || R > D || R % 2 != 0) return RMSN_EUNSUPPORTED;
    return RMSN_OK;
}

constexpr int64_t kMaxExtent = int64_t(1) << 47;  // elements from the first to the last of a tensor

int check_heads_in(const HeadsIn& a, int64_t T, int64_t H) {
    if (a.p == nullptr || a.token < 0 || a.head < 0) return RMSN_EINVAL;
    if (a.token > kMaxExtent / T || a.head > kMaxExtent / H) return RMSN_EINVAL;  // no product below overflows
    if (!aligned16(a.p) || a.token % 8 != 0 || a.head % 8 != 0) return RMSN_EALIGN;
    return RMSN_OK;
}

// An output's rows must not overlap: either its tokens lie outside its heads or
// its heads outside its tokens (a stride that is never taken does not count).
int check_heads_out(const HeadsOut& o, int64_t T, int64_t H, int64_t D) {
    RMSN_TRY(check_heads_in({o.p, o.token, o.head}, T, H));
    const bool tokens_outside = (H == 1 || o.head >= D) && (T == 1 || o.token >= (H - 1) * o.head + D);
    const bool heads_outside = (T == 1 || o.token >= D) && (H == 1 || o.head >= (T - 1) * o.token + D);
    return tokens_outside || heads_outside ? RMSN_OK : RMSN_EINVAL;
}

// In place only with the input's own strides.
int check_in_place(const HeadsIn& i, const HeadsOut& o, int64_t T, int64_t H) {
    if (i.p != o.p) return RMSN_OK;
    return (T == 1 || i.token == o.token) && (H == 1 || i.head == o.head) ? RMSN_OK : RMSN_EINVAL;
}

int check_pos(const void* pos, int pos_dtype, const double* inv_freq) {
    if (inv_freq == nullptr) return RMSN_EINVAL;
    if (!aligned16(inv_freq)) return RMSN_EALIGN;
    if (reinterpret_cast<uintptr_t>(pos) % (pos_dtype == ROPE_POS_I64 ? 8 : 4) != 0) return RMSN_EALIGN;
    return RMSN_OK;
}

int check_in_out(const RopeArgs& a, int64_t T, int64_t D) {
    for (int s = 0; s < 2; ++s) {
        if (a.H[s] == 0) continue;
        RMSN_TRY(check_heads_in(a.in[s], T, a.H[s]));
        RMSN_TRY(check_heads_out(a.out[s], T, a.H[s], D));
        RMSN_TRY(check_in_place(a.in[s], a.out[s], T, a.H[s]));
    }
    return RMSN_OK;
}

int turn_impl(bool back, const HeadsIn& q, const HeadsIn& k, const double* inv_freq, const void* positions,
              int pos_dtype, const HeadsOut& qo, const HeadsOut& ko, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
              int64_t R, float scale, int layout, int dtype, cudaStream_t stream) {
    int flags = 0;
    RMSN_TRY(dtype_flags(dtype, &flags));
    RMSN_TRY(check_sizes(T, Hq, Hk, D));
    RMSN_TRY(check_rope(D, R, scale, layout, pos_dtype));
    if (T == 0) return RMSN_OK;
    RopeArgs a{};
    a.in[0] = q; a.in[1] = k; a.out[0] = qo; a.out[1] = ko;
    a.T = T; a.H[0] = static_cast<int>(Hq); a.H[1] = static_cast<int>(Hk);
    a.D = static_cast<int>(D); a.R = static_cast<int>(R); a.layout = layout;
    a.inv_freq = inv_freq; a.pos = positions; a.pos64 = pos_dtype == ROPE_POS_I64; a.scale = scale; a.back = back;
    RMSN_TRY(check_in_out(a, T, D));
    RMSN_TRY(check_pos(positions, pos_dtype, inv_freq));
    return cuda_status(rope_run<kTurn>(a, flags, rope_grid(T), stream));
}

}  // namespace
}  // namespace rmsn

using namespace rmsn;

extern "C" {

int rope_frequencies(int64_t R, double theta, int scaling, double factor, double low, double high, double length,
                     double* inv_freq) {
    constexpr double kTwoPi = 6.283185307179586477;
    if (inv_freq == nullptr || R < 2 || R % 2 != 0 || R > kMaxHeadD) return RMSN_EINVAL;
    if (!std::isfinite(theta) || theta <= 1.0 || !std::isfinite(factor) || factor < 1.0) return RMSN_EINVAL;
    const bool ramp = scaling == ROPE_SCALING_RAMP_TURNS || scaling == ROPE_SCALING_RAMP_INDEX;
    if (!ramp && scaling != ROPE_SCALING_NONE && scaling != ROPE_SCALING_LINEAR && scaling != ROPE_SCALING_BASE)
        return RMSN_EINVAL;
    if (ramp && !(std::isfinite(low) && std::isfinite(high) && low > 0.0 && high > low && std::isfinite(length) &&
                  length > 0.0))
        return RMSN_EINVAL;
    if (scaling == ROPE_SCALING_BASE) {
        if (R == 2) return RMSN_EINVAL;
        theta *= std::pow(factor, static_cast<double>(R) / static_cast<double>(R - 2));
    }
    const int64_t n = R / 2;
    // The (fractional) index of the pair that turns `turns` times over `length`.
    auto index_of = [&](double turns) {
        return static_cast<double>(R) * std::log(length / (kTwoPi * turns)) / (2.0 * std::log(theta));
    };
    const double last = static_cast<double>(n - 1);
    double from = 0.0, to = 0.0;
    if (scaling == ROPE_SCALING_RAMP_INDEX) {
        from = std::min(std::max(std::floor(index_of(high)), 0.0), last);
        to = std::min(std::max(std::ceil(index_of(low)), 0.0), last);
    }
    for (int64_t i = 0; i < n; ++i) {
        const double f = std::pow(theta, -2.0 * static_cast<double>(i) / static_cast<double>(R));
        double keep = 1.0;
        if (scaling == ROPE_SCALING_LINEAR) keep = 0.0;
        if (scaling == ROPE_SCALING_RAMP_TURNS)
            keep = std::min(1.0, std::max(0.0, (length * f / kTwoPi - low) / (high - low)));
        if (scaling == ROPE_SCALING_RAMP_INDEX)
            keep = to > from ? 1.0 - std::min(1.0, std::max(0.0, (static_cast<double>(i) - from) / (to - from)))
                             : (static_cast<double>(i) <= from ? 1.0 : 0.0);
        inv_freq[i] = f * (keep + (1.0 - keep) / factor);
    }
    return RMSN_OK;
}

int rope_fwd(const rmsn_act16* q, int64_t q_token, int64_t q_head, const rmsn_act16* k, int64_t k_token,
             int64_t k_head, const double* inv_freq, const void* positions, int pos_dtype, rmsn_act16* q_out,
             int64_t qo_token, int64_t qo_head, rmsn_act16* k_out, int64_t ko_token, int64_t ko_head, int64_t T,
             int64_t Hq, int64_t Hk, int64_t D, int64_t R, float scale, int layout, int dtype, rmsn_stream stream) {
    return turn_impl(false, {q, q_token, q_head}, {k, k_token, k_head}, inv_freq, positions, pos_dtype,
                     {q_out, qo_token, qo_head}, {k_out, ko_token, ko_head}, T, Hq, Hk, D, R, scale, layout, dtype,
                     stream);
}

int rope_bwd(const rmsn_act16* gq, int64_t gq_token, int64_t gq_head, const rmsn_act16* gk, int64_t gk_token,
             int64_t gk_head, const double* inv_freq, const void* positions, int pos_dtype, rmsn_act16* dq,
             int64_t dq_token, int64_t dq_head, rmsn_act16* dk, int64_t dk_token, int64_t dk_head, int64_t T,
             int64_t Hq, int64_t Hk, int64_t D, int64_t R, float scale, int layout, int dtype, rmsn_stream stream) {
    return turn_impl(true, {gq, gq_token, gq_head}, {gk, gk_token, gk_head}, inv_freq, positions, pos_dtype,
                     {dq, dq_token, dq_head}, {dk, dk_token, dk_head}, T, Hq, Hk, D, R, scale, layout, dtype, stream);
}

int rmsnorm_rope_fwd(const rmsn_act16* q, int64_t q_token, int64_t q_head, const rmsn_act16* k, int64_t k_token,
                     int64_t k_head, const float* wq, const float* wk, const double* inv_freq, const void* positions,
                     int pos_dtype, rmsn_act16* q_out, int64_t qo_token, int64_t qo_head, rmsn_act16* k_out,
                     int64_t ko_token, int64_t ko_head, float* rstd_q, float* rstd_k, int64_t T, int64_t Hq,
                     int64_t Hk, int64_t D, int64_t R, float scale, int layout, float eps, int zero_centered_gamma,
                     int dtype, rmsn_stream stream) {
    int flags = 0;
    RMSN_TRY(dtype_flags(dtype, &flags));
    RMSN_TRY(check_sizes(T, Hq, Hk, D));
    RMSN_TRY(check_rope(D, R, scale, layout, pos_dtype));
    RMSN_TRY(check_eps(eps));
    if (T == 0) return RMSN_OK;
    RopeArgs a{};
    a.in[0] = {q, q_token, q_head}; a.in[1] = {k, k_token, k_head};
    a.out[0] = {q_out, qo_token, qo_head}; a.out[1] = {k_out, ko_token, ko_head};
    a.w[0] = wq; a.w[1] = wk; a.rstd[0] = rstd_q; a.rstd[1] = rstd_k;
    a.T = T; a.H[0] = static_cast<int>(Hq); a.H[1] = static_cast<int>(Hk);
    a.D = static_cast<int>(D); a.R = static_cast<int>(R); a.layout = layout;
    a.inv_freq = inv_freq; a.pos = positions; a.pos64 = pos_dtype == ROPE_POS_I64; a.scale = scale;
    a.eps = eps; a.zc = zero_centered_gamma ? 1 : 0;
    RMSN_TRY(check_in_out(a, T, D));
    for (int s = 0; s < 2; ++s) {
        if (a.H[s] == 0) continue;
        RMSN_TRY(check_vec(a.w[s]));
        RMSN_TRY(check_vec(a.rstd[s]));
    }
    RMSN_TRY(check_pos(positions, pos_dtype, inv_freq));
    return cuda_status(rope_run<kNormTurn>(a, flags, rope_grid(T), stream));
}

size_t rmsnorm_rope_bwd_workspace_bytes(int64_t T, int64_t Hq, int64_t Hk, int64_t D) {
    if (check_sizes(T, Hq, Hk, D) != RMSN_OK || T == 0) return 0;
    return static_cast<size_t>(rope_chunks(T)) * static_cast<size_t>(D) * 8u;
}

int rmsnorm_rope_bwd(const rmsn_act16* gq, int64_t gq_token, int64_t gq_head, const rmsn_act16* gk, int64_t gk_token,
                     int64_t gk_head, const rmsn_act16* q, int64_t q_token, int64_t q_head, const rmsn_act16* k,
                     int64_t k_token, int64_t k_head, const float* wq, const float* wk, const double* inv_freq,
                     const void* positions, int pos_dtype, const float* rstd_q, const float* rstd_k, rmsn_act16* dq,
                     int64_t dq_token, int64_t dq_head, rmsn_act16* dk, int64_t dk_token, int64_t dk_head, float* dwq,
                     float* dwk, void* ws, size_t ws_bytes, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R,
                     float scale, int layout, int zero_centered_gamma, int dtype, rmsn_stream stream) {
    int flags = 0;
    RMSN_TRY(dtype_flags(dtype, &flags));
    RMSN_TRY(check_sizes(T, Hq, Hk, D));
    RMSN_TRY(check_rope(D, R, scale, layout, pos_dtype));
    RMSN_TRY(check_vec(dwq));
    if (Hk > 0) RMSN_TRY(check_vec(dwk));
    if (T == 0) {  // the sums over no rows
        cudaError_t e = cudaMemsetAsync(dwq, 0, static_cast<size_t>(D) * 4u, stream);
        if (e == cudaSuccess && Hk > 0) e = cudaMemsetAsync(dwk, 0, static_cast<size_t>(D) * 4u, stream);
        return cuda_status(e);
    }
    RopeArgs a{};
    a.in[0] = {gq, gq_token, gq_head}; a.in[1] = {gk, gk_token, gk_head};
    a.x[0] = {q, q_token, q_head}; a.x[1] = {k, k_token, k_head};
    a.out[0] = {dq, dq_token, dq_head}; a.out[1] = {dk, dk_token, dk_head};
    a.w[0] = wq; a.w[1] = wk;
    a.rstd[0] = const_cast<float*>(rstd_q); a.rstd[1] = const_cast<float*>(rstd_k);  // read only here
    a.T = T; a.H[0] = static_cast<int>(Hq); a.H[1] = static_cast<int>(Hk);
    a.D = static_cast<int>(D); a.R = static_cast<int>(R); a.layout = layout;
    a.inv_freq = inv_freq; a.pos = positions; a.pos64 = pos_dtype == ROPE_POS_I64; a.scale = scale; a.back = 1;
    a.zc = zero_centered_gamma ? 1 : 0; a.chunk = static_cast<int>(rope_chunk(T));
    RMSN_TRY(check_in_out(a, T, D));
    for (int s = 0; s < 2; ++s) {
        if (a.H[s] == 0) continue;
        RMSN_TRY(check_heads_in(a.x[s], T, a.H[s]));
        RMSN_TRY(check_vec(a.w[s]));
        RMSN_TRY(check_vec(a.rstd[s]));
    }
    RMSN_TRY(check_pos(positions, pos_dtype, inv_freq));
    if (ws == nullptr || ws_bytes < rmsnorm_rope_bwd_workspace_bytes(T, Hq, Hk, D)) return RMSN_EWORKSPACE;
    if (!aligned16(ws)) return RMSN_EALIGN;
    a.partials = static_cast<float*>(ws);
    const int64_t n = rope_chunks(T);
    cudaError_t e = rope_run<kNormTurnBwd>(a, flags, static_cast<unsigned>(n), stream);
    if (e == cudaSuccess) e = launch_reduce_columns(a.partials, n, a.D, dwq, Hk > 0 ? dwk : nullptr, stream);
    return cuda_status(e);
}

}  // extern "C"
