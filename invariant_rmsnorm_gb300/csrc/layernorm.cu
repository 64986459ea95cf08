// LayerNorm with bf16 activations (the instantiations of layernorm_impl.cuh) and
// its C-ABI entry points for both formats.
#include "checks.h"
#include "layernorm_impl.cuh"
#include "reduce_columns.h"

namespace rmsn {

cudaError_t layernorm_read_error(unsigned* flags, bool clear) { return read_ln_error_word(flags, clear); }
cudaError_t launch_ln_fwd(const LnFwdArgs& a, cudaStream_t s) { return ln_fwd_dispatch<false>(a, s); }
cudaError_t launch_ln_bwd(const LnBwdArgs& a, unsigned chunks, bool bias, cudaStream_t s) {
    return bias ? ln_bwd_dispatch<false, true>(a, chunks, s) : ln_bwd_dispatch<false, false>(a, chunks, s);
}

namespace {

// The weight gradients' chunks, one a CTA: as many as the CTAs that a GPU of 152
// SMs holds at once, so that all work to the end, and whole rounds of them where
// a chunk would pass kLnMaxChunk rows (which bounds the fp32 chain of a sum, and
// the row statistics that a wide kernel keeps in shared memory). A function of T
// and D alone: 152 stands for the GPU.
constexpr int64_t kLnSms = 152;
constexpr int64_t kLnMaxChunk = 256;
struct LnChunks { int64_t rows, count; };

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

LnChunks ln_chunks(int64_t T, int64_t D) {
    const LnShape s = ln_shape(D);
    const int64_t round = kLnSms * s.per_sm;
    const int64_t ctas = ceil_div(T, round * kLnMaxChunk * s.step) * round;
    const int64_t rows = ceil_div(ceil_div(T, ctas), s.step) * s.step;
    return {rows, ceil_div(T, rows)};
}

// No T up to T_max has more chunks: their count passes neither T_max / step nor
// the CTAs of T_max's rounds.
int64_t ln_chunks_max(int64_t T_max, int64_t D) {
    const LnShape s = ln_shape(D);
    const int64_t round = kLnSms * s.per_sm;
    return std::min(ceil_div(T_max, s.step), ceil_div(T_max, round * kLnMaxChunk * s.step) * round);
}

size_t ws_need(int64_t T, int64_t D) {
    return static_cast<size_t>(ln_chunks(T, D).count) * static_cast<size_t>(D) * 8u;
}

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
    const LnFwdArgs a{x, ldx, w, b, y, ldy, mean, rstd, T, static_cast<int>(D), eps, zero_centered_gamma ? 1 : 0,
                      1.0f / static_cast<float>(D)};
    return cuda_status(flags ? launch_ln_fwd_f16(a, stream) : launch_ln_fwd(a, stream));
}

size_t layernorm_bwd_workspace_bytes(int64_t T, int64_t D) {
    if (check_shape(T, D) != RMSN_OK || T == 0) return 0;
    return ws_need(T, D);
}

size_t layernorm_bwd_workspace_bytes_max(int64_t T_max, int64_t D) {
    if (check_shape(T_max, D) != RMSN_OK || T_max <= 0) return 0;
    return static_cast<size_t>(ln_chunks_max(T_max, D)) * static_cast<size_t>(D) * 8u;
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
    const LnChunks c = ln_chunks(T, D);
    const LnBwdArgs a{g, ldg, x, ldx, w, mean, rstd, dx, lddx, static_cast<float*>(ws), T, static_cast<int>(D),
                      zero_centered_gamma ? 1 : 0, static_cast<int>(c.rows), 1.0f / static_cast<float>(D)};
    const unsigned n = static_cast<unsigned>(c.count);
    cudaError_t e = flags ? launch_ln_bwd_f16(a, n, db != nullptr, stream) : launch_ln_bwd(a, n, db != nullptr, stream);
    if (e == cudaSuccess) e = launch_reduce_columns({a.partials, c.count, dw}, {a.partials + c.count * D, c.count, db}, a.D, stream);
    return cuda_status(e);
}

}  // extern "C"
