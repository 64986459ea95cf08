/*
 * linear.h — projections of the GB300 (sm_103a) norm library: a matrix product
 * with bias, activation and residual in its epilogue, and a gated feed-forward
 * block's two projections with their activation and product, with their gradients.
 *
 * Forward, x [T][K], w [N][K]:
 *   z_tn = sum_k x_tk w_nk + b_n                      fp32
 *   y_tn = round( act(z_tn) + res_tn )                one rounding, of the fp32 value
 * and, if asked for, z rounded (the backward's input). Gated, wg and wu [N][K]:
 *   gate = x wg^T, up = x wu^T                        fp32
 *   h    = round( act(gate) * up )                    of the fp32 values
 * and, if asked for, gate and up rounded.
 * Backward, from the saved (rounded) z, or gate and up:
 *   dz   = g * act'(z)                dgate = g * up * act'(gate),  dup = g * act(gate)
 *   dx   = dz w                       dx    = dgate wg + dup wu
 *   dw   = dz^T x,  db = sum_t dz     dwg   = dgate^T x,  dwu = dup^T x
 * The gradient of res is g itself.
 *
 * Products are of 16-bit values on the tensor cores, their sums fp32, in steps of 16 that are cut off at fp32's
 * last place, not rounded: a long sum of one sign comes out low, by 2e-5 of itself at K = 4096, 4e-4 at 65536 and
 * 6e-3 at 2^20 (half a step of fp16 is 5e-4, of bf16 4e-3); the weights' gradients likewise by the rows of a range. dz, dgate and
 * dup are rounded to the activation format before their products (they are these
 * products' operands; an fp16 one that passes 65504 becomes infinite), but db sums
 * the unrounded fp32 values. Without an activation dz is g and nothing is rounded.
 * An fp16 z, gate or up that passed 65504 was saved as infinite: the backward takes act' at its limit there,
 * and a zero factor beside it gives zero (NaN stays NaN).
 *
 * Layouts, ownership, streams and errors are those of rmsnorm.h: 16-bit
 * activations and weights [rows][ld] with a row stride of a multiple of 8
 * elements, fp32 vectors, every pointer a 16-byte aligned DEVICE pointer. K and N are multiples of 8 with
 * 8 <= K, N <= 2^20; 0 <= T < 2^31. `dtype` is an enum rmsn_dtype: the format of every
 * 16-bit argument, weights included. The current device is the stream's. Outputs
 * must not overlap inputs or each other, but y may be res (same stride): the call
 * then adds to the residual stream in place. T == 0 launches no product and
 * returns RMSN_OK (the weights' gradients are set to zero).
 *
 * Batch invariance: y[t], z[t], h[t], gate[t], up[t] and dx[t] are bitwise
 * independent of T, of the row's position and of the other rows: every value is
 * one chain of sums over the reduced axis in ascending order, at every tile size.
 * The weights' gradients are summed with no atomics, over ranges of rows that
 * depend on T, N and K alone: the same bits from run to run. (Tiles are chosen by the sizes, as of a GPU of 152
 * SMs, and by whether every operand's rows start on lines of 128 bytes; no bits depend on them, so a view between
 * other columns has those of a matrix of its own.)
 *
 * Calls that may run at the same time (on two streams, in two graphs) need
 * workspaces of their own.
 */
#ifndef LINEAR_GB300_H_
#define LINEAR_GB300_H_

#include "rmsnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum linear_act {
    LINEAR_ACT_NONE = 0,
    LINEAR_ACT_SILU = 1,       /* z sigmoid(z)                                             */
    LINEAR_ACT_SIGMOID = 2,
    LINEAR_ACT_GELU = 3,       /* z (1 + erf(z / sqrt 2)) / 2                              */
    LINEAR_ACT_GELU_TANH = 4,  /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2         */
    LINEAR_ACT_RELU = 5
};

/* b [N], res [T][ldr] and z [T][ldz] may be NULL: no bias, no residual, z not kept. */
int linear_fwd(const rmsn_act16* x, int64_t ldx, const rmsn_act16* w, int64_t ldw, const float* b,
               const rmsn_act16* res, int64_t ldr, rmsn_act16* y, int64_t ldy, rmsn_act16* z, int64_t ldz,
               int64_t T, int64_t N, int64_t K, int act, int dtype, rmsn_stream stream);

/* Bytes of workspace linear_bwd needs for all of its outputs (0 for T == 0 and unsupported sizes). They are not monotone in T:
 * rows are split for the weights' gradient where that pays, and a larger T can need far fewer bytes than a
 * smaller one (N = K = 4096, no activation: 136 MB at T = 23680, 2 MB at 23681). To size one buffer for every T up to
 * a maximum, use linear_bwd_workspace_bytes_max. */
size_t linear_bwd_workspace_bytes(int64_t T, int64_t N, int64_t K, int act);

/* One size that serves every T up to T_max (0 for T_max <= 0 and unsupported sizes). */
size_t linear_bwd_workspace_bytes_max(int64_t T_max, int64_t N, int64_t K, int act);

/* g [T][ldg] is the gradient of y. z is read where there is an activation (else it may
 * be NULL). dx [T][lddx], dw [N][lddw] and db [N] may each be NULL: not wanted. x is read
 * for dw, w for dx alone, and may be NULL without them. ws: contents never read back after the call. Of its bytes
 * a call asks for what its outputs take: 2 T N (to a multiple of 256) for dx or dw with an activation, db's partial rows for db, the split sums
 * for dw. Without any of these (dx alone and no activation, say) ws may be NULL. */
int linear_bwd(const rmsn_act16* g, int64_t ldg, const rmsn_act16* x, int64_t ldx, const rmsn_act16* w, int64_t ldw,
               const rmsn_act16* z, int64_t ldz, rmsn_act16* dx, int64_t lddx, rmsn_act16* dw, int64_t lddw, float* db,
               void* ws, size_t ws_bytes, int64_t T, int64_t N, int64_t K, int act, int dtype, rmsn_stream stream);

/* gate [T][ldgate] and up [T][ldup] may be NULL together: not kept. */
int linear_gated_fwd(const rmsn_act16* x, int64_t ldx, const rmsn_act16* wg, int64_t ldwg, const rmsn_act16* wu, int64_t ldwu,
                     rmsn_act16* h, int64_t ldh, rmsn_act16* gate, int64_t ldgate, rmsn_act16* up, int64_t ldup,
                     int64_t T, int64_t N, int64_t K, int act, int dtype, rmsn_stream stream);

/* Bytes of workspace linear_gated_bwd needs for all of its outputs (0 for T == 0 and unsupported sizes); not monotone in T either. */
size_t linear_gated_bwd_workspace_bytes(int64_t T, int64_t N, int64_t K);

/* One size that serves every T up to T_max (0 for T_max <= 0 and unsupported sizes). */
size_t linear_gated_bwd_workspace_bytes_max(int64_t T_max, int64_t N, int64_t K);

/* g [T][ldg] is the gradient of h. dx may be NULL, and dwg and dwu together; without these two the call asks for no
 * split sums (4 T N bytes, each half of them to a multiple of 256, are enough). */
int linear_gated_bwd(const rmsn_act16* g, int64_t ldg, const rmsn_act16* x, int64_t ldx,
                     const rmsn_act16* wg, int64_t ldwg, const rmsn_act16* wu, int64_t ldwu,
                     const rmsn_act16* gate, int64_t ldgate, const rmsn_act16* up, int64_t ldup,
                     rmsn_act16* dx, int64_t lddx, rmsn_act16* dwg, int64_t lddwg, rmsn_act16* dwu, int64_t lddwu,
                     void* ws, size_t ws_bytes, int64_t T, int64_t N, int64_t K, int act, int dtype, rmsn_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* LINEAR_GB300_H_ */
