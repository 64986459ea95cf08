/*
 * layernorm.h — LayerNorm entry points of the GB300 (sm_103a) norm library.
 *
 * Forward, per row t of x [T][D]:
 *   mu_t  = (sum_j x_tj) / D                            saved as fp32 mean[t]
 *   r_t   = rsqrt( (sum_j (x_tj - mu_t)^2) / D + eps )  saved as fp32 rstd[t]
 *   n_tj  = (x_tj - mu_t) * r_t
 *   y_tj  = round( n_tj * w_eff_j + b_j )               w_eff = w, or (fp32) w + 1 (zero-centred gamma)
 * The variance is the second pass over the row's deviations from its mean, not
 * a difference of two sums, so a mean far from zero costs no digits. A row whose
 * sum of squared deviations passes fp32's range (3.4e38) has rstd 0 and y = b.
 * Backward, per row (g = dL/dy, the saved mu and r):
 *   c1    = (sum_j g_j w_eff_j) / D,   c2 = (sum_j g_j w_eff_j n_j) / D
 *   dx_j  = round( r * (g_j w_eff_j - c1 - n_j * c2) )
 *   dw_j  = sum_t g_tj n_tj,   db_j = sum_t g_tj        fp32
 *
 * Layouts, alignment, ownership, streams and errors are those of rmsnorm.h:
 * 16-bit activations [T][D] with a row stride of a multiple of 8 elements,
 * fp32 vectors, every pointer a 16-byte aligned DEVICE pointer, D a multiple of
 * 8 with 8 <= D <= 16384, 0 <= T < 2^31. `dtype` is an enum rmsn_dtype: the
 * format of every activation argument. Sums, statistics and gradients of the
 * weights are fp32. The current device is the stream's.
 *
 * Batch invariance: y[t], mean[t], rstd[t] and dx[t] are bitwise independent of
 * T, of the row's position, of the other rows and of the GPU's SM count: a
 * row's reduction tree is a function of D alone. dw and db are summed with no atomics, over row
 * chunks whose size depends on T and D alone and then over the chunks in a
 * fixed order: the same bits from run to run and on GPUs with different SM counts.
 */
#ifndef LAYERNORM_GB300_H_
#define LAYERNORM_GB300_H_

#include "rmsnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Forward. b may be NULL (no bias). T == 0 returns RMSN_OK and launches nothing.
 *   x [T][ldx], w [D], b [D] in; y [T][ldy], mean [T], rstd [T] out. */
int layernorm_fwd(const rmsn_act16* x, int64_t ldx, const float* w, const float* b,
                  rmsn_act16* y, int64_t ldy, float* mean, float* rstd,
                  int64_t T, int64_t D, float eps, int zero_centered_gamma,
                  int dtype, rmsn_stream stream);

/* Bytes of workspace layernorm_bwd needs for T rows of width D, with or without
 * a bias (0 for T == 0 and for an unsupported D). Not monotone in T. */
size_t layernorm_bwd_workspace_bytes(int64_t T, int64_t D);

/* One size that serves every T up to T_max (0 for T_max <= 0 or an unsupported D). */
size_t layernorm_bwd_workspace_bytes_max(int64_t T_max, int64_t D);

/* Backward. db may be NULL (the norm has no bias, or its gradient is not wanted).
 *   g [T][ldg], x [T][ldx], w [D], mean [T], rstd [T] (the forward's) in;
 *   dx [T][lddx], dw [D], db [D] out; ws workspace (contents never read back
 *   after the call). T == 0 sets dw and db to zero. */
int layernorm_bwd(const rmsn_act16* g, int64_t ldg, const rmsn_act16* x, int64_t ldx,
                  const float* w, const float* mean, const float* rstd,
                  rmsn_act16* dx, int64_t lddx, float* dw, float* db,
                  void* ws, size_t ws_bytes,
                  int64_t T, int64_t D, int zero_centered_gamma,
                  int dtype, rmsn_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* LAYERNORM_GB300_H_ */
