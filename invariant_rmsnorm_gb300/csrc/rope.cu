// Rotary positions of q and k, alone and fused with the heads' RMSNorm, forward
// and backward: the C-ABI entry points.
#include <algorithm>
#include <cmath>

#include "checks.h"
#include "reduce_columns.h"
#include "rope_launch.h"

namespace rmsn {

namespace {

int rope_run(RopeMode mode, RopeArgs& a, int flags, cudaStream_t s, int* ctas_q = nullptr) {
    int unused = 0;
    if (ctas_q == nullptr) ctas_q = &unused;
    a.rcp_d = 1.0f / static_cast<float>(a.D);
    for (int i = 0; i < 2; ++i) {
        const bool in_place = mode == kTurn && a.out[i].p == a.in[i].p;
        a.row_bytes[i] = static_cast<uint32_t>(in_place ? (a.R + 7) / 8 * 16 : a.D * 2);
        const bool whole = a.row_bytes[i] == static_cast<uint32_t>(a.D) * 2u;
        a.dense[0][i] = whole && a.in[i].head == a.D;
        a.dense[1][i] = whole && a.x[i].head == a.D;
        a.dense[2][i] = whole && a.out[i].head == a.D;
    }
    const bool axes = a.axis != nullptr;
    switch (mode) {
        case kTurn:
            if (axes) return cuda_status(flags ? launch_rope_axes_turn_f16(a, ctas_q, s) : launch_rope_axes_turn(a, ctas_q, s));
            return cuda_status(flags ? launch_rope_turn_f16(a, ctas_q, s) : launch_rope_turn(a, ctas_q, s));
        case kNormTurn:
            if (axes) return cuda_status(flags ? launch_rope_axes_norm_f16(a, ctas_q, s) : launch_rope_axes_norm(a, ctas_q, s));
            return cuda_status(flags ? launch_rope_norm_f16(a, ctas_q, s) : launch_rope_norm(a, ctas_q, s));
        default:
            if (axes) return cuda_status(flags ? launch_rope_axes_norm_bwd_f16(a, ctas_q, s) : launch_rope_axes_norm_bwd(a, ctas_q, s));
            return cuda_status(flags ? launch_rope_norm_bwd_f16(a, ctas_q, s) : launch_rope_norm_bwd(a, ctas_q, s));
    }
}

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

// Positions of several axes: [axes][T] by two strides, and the axis of every pair.
struct Axes {
    const uint8_t* axis;
    int64_t n;
    int64_t pos_axis, pos_token;
};

int check_axes(const Axes& x, const void* pos, int64_t T) {
    if (x.axis == nullptr || pos == nullptr || x.n < 1 || x.n > 256 || x.pos_axis < 0 || x.pos_token < 0) return RMSN_EINVAL;
    return x.pos_axis > kMaxExtent / x.n || x.pos_token > kMaxExtent / T ? RMSN_EINVAL : RMSN_OK;
}

// Positions and frequencies into the arguments (axes null: one position a token).
int set_angles(RopeArgs& a, const double* inv_freq, const Axes* axes, const void* pos, int pos_dtype) {
    RMSN_TRY(check_pos(pos, pos_dtype, inv_freq));
    if (axes != nullptr) {
        RMSN_TRY(check_axes(*axes, pos, a.T));
        a.axis = axes->axis; a.axes = static_cast<int>(axes->n);
        a.pos_axis = axes->pos_axis; a.pos_token = axes->pos_token;
    }
    a.inv_freq = inv_freq; a.pos = pos; a.pos64 = pos_dtype == ROPE_POS_I64;
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

int turn_impl(bool back, const HeadsIn& q, const HeadsIn& k, const double* inv_freq, const Axes* axes,
              const void* positions, int pos_dtype, const HeadsOut& qo, const HeadsOut& ko, int64_t T, int64_t Hq,
              int64_t Hk, int64_t D, int64_t R, float scale, int layout, int dtype, cudaStream_t stream) {
    int flags = 0;
    RMSN_TRY(dtype_flags(dtype, &flags));
    RMSN_TRY(check_sizes(T, Hq, Hk, D));
    RMSN_TRY(check_rope(D, R, scale, layout, pos_dtype));
    if (T == 0) return RMSN_OK;
    RopeArgs a{};
    a.in[0] = q; a.in[1] = k; a.out[0] = qo; a.out[1] = ko;
    a.T = T; a.H[0] = static_cast<int>(Hq); a.H[1] = static_cast<int>(Hk);
    a.D = static_cast<int>(D); a.R = static_cast<int>(R); a.layout = layout; a.scale = scale; a.back = back;
    RMSN_TRY(check_in_out(a, T, D));
    RMSN_TRY(set_angles(a, inv_freq, axes, positions, pos_dtype));
    return rope_run(kTurn, a, flags, stream);
}

int norm_fwd_impl(const HeadsIn& q, const HeadsIn& k, const float* wq, const float* wk, const double* inv_freq, const Axes* axes,
                  const void* positions, int pos_dtype, const HeadsOut& qo, const HeadsOut& ko, float* rstd_q, float* rstd_k,
                  int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R, float scale, int layout, float eps,
                  int zero_centered_gamma, int dtype, cudaStream_t stream) {
    int flags = 0;
    RMSN_TRY(dtype_flags(dtype, &flags));
    RMSN_TRY(check_sizes(T, Hq, Hk, D));
    RMSN_TRY(check_rope(D, R, scale, layout, pos_dtype));
    RMSN_TRY(check_eps(eps));
    if (T == 0) return RMSN_OK;
    RopeArgs a{};
    a.in[0] = q; a.in[1] = k; a.out[0] = qo; a.out[1] = ko;
    a.w[0] = wq; a.w[1] = wk; a.rstd[0] = rstd_q; a.rstd[1] = rstd_k;
    a.T = T; a.H[0] = static_cast<int>(Hq); a.H[1] = static_cast<int>(Hk);
    a.D = static_cast<int>(D); a.R = static_cast<int>(R); a.layout = layout;
    a.scale = scale; a.eps = eps; a.zc = zero_centered_gamma ? 1 : 0;
    RMSN_TRY(check_in_out(a, T, D));
    for (int s = 0; s < 2; ++s) {
        if (a.H[s] == 0) continue;
        RMSN_TRY(check_vec(a.w[s]));
        RMSN_TRY(check_vec(a.rstd[s]));
    }
    RMSN_TRY(set_angles(a, inv_freq, axes, positions, pos_dtype));
    return rope_run(kNormTurn, a, flags, stream);
}

int norm_bwd_impl(const HeadsIn& gq, const HeadsIn& gk, const HeadsIn& q, const HeadsIn& k, const float* wq, const float* wk,
                  const double* inv_freq, const Axes* axes, const void* positions, int pos_dtype, const float* rstd_q,
                  const float* rstd_k, const HeadsOut& dq, const HeadsOut& dk, float* dwq, float* dwk, void* ws, size_t ws_bytes,
                  int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R, float scale, int layout, int zero_centered_gamma,
                  int dtype, cudaStream_t stream) {
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
    a.in[0] = gq; a.in[1] = gk; a.x[0] = q; a.x[1] = k; a.out[0] = dq; a.out[1] = dk;
    a.w[0] = wq; a.w[1] = wk;
    a.rstd[0] = const_cast<float*>(rstd_q); a.rstd[1] = const_cast<float*>(rstd_k);  // read only here
    a.T = T; a.H[0] = static_cast<int>(Hq); a.H[1] = static_cast<int>(Hk);
    a.D = static_cast<int>(D); a.R = static_cast<int>(R); a.layout = layout;
    a.scale = scale; a.back = 1; a.zc = zero_centered_gamma ? 1 : 0;
    RMSN_TRY(check_in_out(a, T, D));
    for (int s = 0; s < 2; ++s) {
        if (a.H[s] == 0) continue;
        RMSN_TRY(check_heads_in(a.x[s], T, a.H[s]));
        RMSN_TRY(check_vec(a.w[s]));
        RMSN_TRY(check_vec(a.rstd[s]));
    }
    RMSN_TRY(set_angles(a, inv_freq, axes, positions, pos_dtype));
    if (ws == nullptr || ws_bytes < rmsnorm_rope_bwd_workspace_bytes(T, Hq, Hk, D)) return RMSN_EWORKSPACE;
    if (!aligned16(ws)) return RMSN_EALIGN;
    a.partials = static_cast<float*>(ws);
    int of_q = 0;
    RMSN_TRY(rope_run(kNormTurnBwd, a, flags, stream, &of_q));
    const int64_t n = rope_bwd_ctas(T, Hq, Hk, D);
    return cuda_status(launch_reduce_columns({a.partials, of_q, dwq}, {a.partials + of_q * D, n - of_q, Hk > 0 ? dwk : nullptr},
                                             a.D, stream));
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
        return static_cast<double>(R) * (std::log(length) - std::log(kTwoPi) - std::log(turns)) / (2.0 * std::log(theta));
    };
    // The ramp's ends, wherever they lie: a head that ends within the ramp, or
    // begins there, has that part of it.
    double from = 0.0, to = 0.0;
    if (scaling == ROPE_SCALING_RAMP_INDEX) {
        from = std::floor(index_of(high));
        to = std::ceil(index_of(low));
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

int rope_axes_map(const int64_t* sections, int64_t axes, int cycled, uint8_t* axis) {
    if (sections == nullptr || axis == nullptr || axes < 1 || axes > 256) return RMSN_EINVAL;
    int64_t n = 0;
    for (int64_t a = 0; a < axes; ++a) {
        if (sections[a] < 1 || sections[a] > kMaxHeadD / 2) return RMSN_EINVAL;
        n += sections[a];
    }
    if (n > kMaxHeadD / 2) return RMSN_EINVAL;
    if (cycled) {  // the last pair dealt to an axis has to be there
        for (int64_t a = 1; a < axes; ++a)
            if (axes * (sections[a] - 1) + a >= n) return RMSN_EINVAL;
        for (int64_t i = 0; i < n; ++i) axis[i] = static_cast<uint8_t>(i < axes * sections[i % axes] ? i % axes : 0);
    } else {
        for (int64_t a = 0; a < axes; ++a)
            for (int64_t i = 0; i < sections[a]; ++i) *axis++ = static_cast<uint8_t>(a);
    }
    return RMSN_OK;
}

int rope_fwd(const rmsn_act16* q, int64_t q_token, int64_t q_head, const rmsn_act16* k, int64_t k_token,
             int64_t k_head, const double* inv_freq, const void* positions, int pos_dtype, rmsn_act16* q_out,
             int64_t qo_token, int64_t qo_head, rmsn_act16* k_out, int64_t ko_token, int64_t ko_head, int64_t T,
             int64_t Hq, int64_t Hk, int64_t D, int64_t R, float scale, int layout, int dtype, rmsn_stream stream) {
    return turn_impl(false, {q, q_token, q_head}, {k, k_token, k_head}, inv_freq, nullptr, positions, pos_dtype,
                     {q_out, qo_token, qo_head}, {k_out, ko_token, ko_head}, T, Hq, Hk, D, R, scale, layout, dtype,
                     stream);
}

int rope_bwd(const rmsn_act16* gq, int64_t gq_token, int64_t gq_head, const rmsn_act16* gk, int64_t gk_token,
             int64_t gk_head, const double* inv_freq, const void* positions, int pos_dtype, rmsn_act16* dq,
             int64_t dq_token, int64_t dq_head, rmsn_act16* dk, int64_t dk_token, int64_t dk_head, int64_t T,
             int64_t Hq, int64_t Hk, int64_t D, int64_t R, float scale, int layout, int dtype, rmsn_stream stream) {
    return turn_impl(true, {gq, gq_token, gq_head}, {gk, gk_token, gk_head}, inv_freq, nullptr, positions, pos_dtype,
                     {dq, dq_token, dq_head}, {dk, dk_token, dk_head}, T, Hq, Hk, D, R, scale, layout, dtype, stream);
}

int rope_axes_fwd(const rmsn_act16* q, int64_t q_token, int64_t q_head, const rmsn_act16* k, int64_t k_token,
                  int64_t k_head, const double* inv_freq, const uint8_t* axis, int64_t axes, const void* positions,
                  int64_t pos_axis, int64_t pos_token, int pos_dtype, rmsn_act16* q_out, int64_t qo_token, int64_t qo_head,
                  rmsn_act16* k_out, int64_t ko_token, int64_t ko_head, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                  int64_t R, float scale, int layout, int dtype, rmsn_stream stream) {
    const Axes x{axis, axes, pos_axis, pos_token};
    return turn_impl(false, {q, q_token, q_head}, {k, k_token, k_head}, inv_freq, &x, positions, pos_dtype,
                     {q_out, qo_token, qo_head}, {k_out, ko_token, ko_head}, T, Hq, Hk, D, R, scale, layout, dtype,
                     stream);
}

int rope_axes_bwd(const rmsn_act16* gq, int64_t gq_token, int64_t gq_head, const rmsn_act16* gk, int64_t gk_token,
                  int64_t gk_head, const double* inv_freq, const uint8_t* axis, int64_t axes, const void* positions,
                  int64_t pos_axis, int64_t pos_token, int pos_dtype, rmsn_act16* dq, int64_t dq_token, int64_t dq_head,
                  rmsn_act16* dk, int64_t dk_token, int64_t dk_head, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                  int64_t R, float scale, int layout, int dtype, rmsn_stream stream) {
    const Axes x{axis, axes, pos_axis, pos_token};
    return turn_impl(true, {gq, gq_token, gq_head}, {gk, gk_token, gk_head}, inv_freq, &x, positions, pos_dtype,
                     {dq, dq_token, dq_head}, {dk, dk_token, dk_head}, T, Hq, Hk, D, R, scale, layout, dtype, stream);
}

int rmsnorm_rope_fwd(const rmsn_act16* q, int64_t q_token, int64_t q_head, const rmsn_act16* k, int64_t k_token,
                     int64_t k_head, const float* wq, const float* wk, const double* inv_freq, const void* positions,
                     int pos_dtype, rmsn_act16* q_out, int64_t qo_token, int64_t qo_head, rmsn_act16* k_out,
                     int64_t ko_token, int64_t ko_head, float* rstd_q, float* rstd_k, int64_t T, int64_t Hq,
                     int64_t Hk, int64_t D, int64_t R, float scale, int layout, float eps, int zero_centered_gamma,
                     int dtype, rmsn_stream stream) {
    return norm_fwd_impl({q, q_token, q_head}, {k, k_token, k_head}, wq, wk, inv_freq, nullptr, positions, pos_dtype,
                         {q_out, qo_token, qo_head}, {k_out, ko_token, ko_head}, rstd_q, rstd_k, T, Hq, Hk, D, R, scale, layout,
                         eps, zero_centered_gamma, dtype, stream);
}

int rmsnorm_rope_axes_fwd(const rmsn_act16* q, int64_t q_token, int64_t q_head, const rmsn_act16* k, int64_t k_token,
                          int64_t k_head, const float* wq, const float* wk, const double* inv_freq, const uint8_t* axis,
                          int64_t axes, const void* positions, int64_t pos_axis, int64_t pos_token, int pos_dtype,
                          rmsn_act16* q_out, int64_t qo_token, int64_t qo_head, rmsn_act16* k_out, int64_t ko_token,
                          int64_t ko_head, float* rstd_q, float* rstd_k, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                          int64_t R, float scale, int layout, float eps, int zero_centered_gamma, int dtype,
                          rmsn_stream stream) {
    const Axes x{axis, axes, pos_axis, pos_token};
    return norm_fwd_impl({q, q_token, q_head}, {k, k_token, k_head}, wq, wk, inv_freq, &x, positions, pos_dtype,
                         {q_out, qo_token, qo_head}, {k_out, ko_token, ko_head}, rstd_q, rstd_k, T, Hq, Hk, D, R, scale, layout,
                         eps, zero_centered_gamma, dtype, stream);
}

int rmsnorm_rope_bwd(const rmsn_act16* gq, int64_t gq_token, int64_t gq_head, const rmsn_act16* gk, int64_t gk_token,
                     int64_t gk_head, const rmsn_act16* q, int64_t q_token, int64_t q_head, const rmsn_act16* k,
                     int64_t k_token, int64_t k_head, const float* wq, const float* wk, const double* inv_freq,
                     const void* positions, int pos_dtype, const float* rstd_q, const float* rstd_k, rmsn_act16* dq,
                     int64_t dq_token, int64_t dq_head, rmsn_act16* dk, int64_t dk_token, int64_t dk_head, float* dwq,
                     float* dwk, void* ws, size_t ws_bytes, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R,
                     float scale, int layout, int zero_centered_gamma, int dtype, rmsn_stream stream) {
    return norm_bwd_impl({gq, gq_token, gq_head}, {gk, gk_token, gk_head}, {q, q_token, q_head}, {k, k_token, k_head}, wq, wk,
                         inv_freq, nullptr, positions, pos_dtype, rstd_q, rstd_k, {dq, dq_token, dq_head}, {dk, dk_token, dk_head},
                         dwq, dwk, ws, ws_bytes, T, Hq, Hk, D, R, scale, layout, zero_centered_gamma, dtype, stream);
}

int rmsnorm_rope_axes_bwd(const rmsn_act16* gq, int64_t gq_token, int64_t gq_head, const rmsn_act16* gk, int64_t gk_token,
                          int64_t gk_head, const rmsn_act16* q, int64_t q_token, int64_t q_head, const rmsn_act16* k,
                          int64_t k_token, int64_t k_head, const float* wq, const float* wk, const double* inv_freq,
                          const uint8_t* axis, int64_t axes, const void* positions, int64_t pos_axis, int64_t pos_token,
                          int pos_dtype, const float* rstd_q, const float* rstd_k, rmsn_act16* dq, int64_t dq_token,
                          int64_t dq_head, rmsn_act16* dk, int64_t dk_token, int64_t dk_head, float* dwq, float* dwk,
                          void* ws, size_t ws_bytes, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R, float scale,
                          int layout, int zero_centered_gamma, int dtype, rmsn_stream stream) {
    const Axes x{axis, axes, pos_axis, pos_token};
    return norm_bwd_impl({gq, gq_token, gq_head}, {gk, gk_token, gk_head}, {q, q_token, q_head}, {k, k_token, k_head}, wq, wk,
                         inv_freq, &x, positions, pos_dtype, rstd_q, rstd_k, {dq, dq_token, dq_head}, {dk, dk_token, dk_head},
                         dwq, dwk, ws, ws_bytes, T, Hq, Hk, D, R, scale, layout, zero_centered_gamma, dtype, stream);
}

size_t rmsnorm_rope_bwd_workspace_bytes(int64_t T, int64_t Hq, int64_t Hk, int64_t D) {
    if (check_sizes(T, Hq, Hk, D) != RMSN_OK || T == 0) return 0;
    return static_cast<size_t>(rope_bwd_ctas(T, Hq, Hk, D)) * static_cast<size_t>(D) * 4u;
}

}  // extern "C"
