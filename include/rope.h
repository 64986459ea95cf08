/*
 * rope.h — rotary positions, an entry point of the GB300 (sm_103a) norm library.
 * (The head norm fused with them, rmsnorm_rope_fwd / _bwd, is in rmsnorm.h.)
 *
 * The first R values of every head (R even, 2 <= R <= D) are R/2 pairs; pair i
 * of token t is turned by the angle a = pos_t * inv_freq_i and scaled:
 *   (u, v) -> scale * (u cos a - v sin a,  v cos a + u sin a)
 * in fp32, each output rounded once to the activation format. The other D - R
 * values of the head are copied bit for bit. The pairs' places (enum rope_layout):
 *   ROPE_HALF         values i and i + R/2
 *   ROPE_INTERLEAVED  values 2i and 2i + 1
 * The backward turns the gradients by -a with the same scale.
 *
 * Angles: inv_freq_i / 2 pi is taken in fp64 to a 64-bit fraction of a turn, and
 * pos * that fraction modulo one turn is an exact 64-bit integer product. The
 * angle's error is about |a| 2^-52 + |pos| 2^-62 rad from the frequency, whatever
 * the position, and 2^-52 rad from the product's lowest bits: there is no table of
 * cosines and no longest context. Every 64-bit position is allowed, negative
 * ones too. cos and sin are fp32, each right to about 2^-22 of itself beside that.
 *
 * q is [T][Hq][D] and k [T][Hk][D], 16-bit values given by two strides in
 * ELEMENTS, from token to token and from head to head (multiples of 8; an
 * input's may be zero, outputs must not overlap themselves). D is a multiple of
 * 8 with 8 <= D <= 512. Hk == 0 (k and k_out NULL) turns q alone. q_out may be q
 * and k_out may be k, with the same strides: the call then works in place, and
 * reads and writes the 16-byte vectors that hold the rotated part alone (up to 7
 * values beyond R are written again with their own bits). Any other overlap of
 * outputs with inputs is not allowed. inv_freq: fp64 [R/2], finite. positions: [T] of enum
 * rope_pos_dtype, or NULL for 0, 1, 2, ... Pointers are DEVICE pointers, 16-byte
 * aligned (positions: aligned to its type). scale is finite. T == 0 returns
 * RMSN_OK and launches nothing. Otherwise as rmsnorm.h.
 *
 * Each output value is a function of its own pair, position and frequency:
 * bitwise independent of T, the heads, the strides and the GPU.
 */
#ifndef ROPE_GB300_H_
#define ROPE_GB300_H_

#include "rmsnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Scalings of the frequencies for contexts longer than those of training. */
enum rope_scaling {
    ROPE_SCALING_NONE = 0,       /* f_i = theta^(-2i/R)                                              */
    ROPE_SCALING_LINEAR = 1,     /* f_i / factor: positions interpolated                             */
    ROPE_SCALING_BASE = 2,       /* theta * factor^(R/(R-2)) in theta's place (R > 2)                */
    ROPE_SCALING_RAMP_TURNS = 3, /* f_i (k + (1-k)/factor), k rising from 0 to 1 while the pair's
                                    turns over `length` positions rise from `low` to `high`          */
    ROPE_SCALING_RAMP_INDEX = 4  /* the same, k falling from 1 to 0 linearly in the pair's index, from
                                    the pair that turns `high` times over `length` positions (rounded
                                    down) to the one that turns `low` times (rounded up), whether
                                    or not the head has these pairs                                  */
};

/* HOST function: the R/2 frequencies (radians a position) of a scaling, in fp64.
 * theta > 1, factor >= 1; `low` < `high` and `length` > 0 are used by the ramps alone.
 * RMSN_EINVAL for anything else, and nothing is written. */
int rope_frequencies(int64_t R, double theta, int scaling, double factor, double low, double high,
                     double length, double* inv_freq);

int rope_fwd(const rmsn_act16* q, int64_t q_token, int64_t q_head,
             const rmsn_act16* k, int64_t k_token, int64_t k_head,
             const double* inv_freq, const void* positions, int pos_dtype,
             rmsn_act16* q_out, int64_t qo_token, int64_t qo_head,
             rmsn_act16* k_out, int64_t ko_token, int64_t ko_head,
             int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R, float scale, int layout,
             int dtype, rmsn_stream stream);

/* The gradients gq, gk of q_out, k_out to dq, dk (which may be gq, gk themselves). */
int rope_bwd(const rmsn_act16* gq, int64_t gq_token, int64_t gq_head,
             const rmsn_act16* gk, int64_t gk_token, int64_t gk_head,
             const double* inv_freq, const void* positions, int pos_dtype,
             rmsn_act16* dq, int64_t dq_token, int64_t dq_head,
             rmsn_act16* dk, int64_t dk_token, int64_t dk_head,
             int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R, float scale, int layout,
             int dtype, rmsn_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* ROPE_GB300_H_ */
