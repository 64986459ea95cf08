/*
 * slots.h — LayerNorm, rotary positions and the head norm with their arguments
 * in an array, for callers whose foreign-function interface converts every
 * argument by itself (a call of 20 to 40 arguments through such an interface
 * costs more than the launch of its kernel).
 */
#ifndef SLOTS_GB300_H_
#define SLOTS_GB300_H_

#include "layernorm.h"
#include "rmsnorm.h"
#include "rope.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One argument: an integer or an enum in i, a float in f (rounded to fp32 by the
 * call), a pointer (the stream too) in p, with i in whole where p is narrower. */
union norm_slot {
    int64_t i;
    double f;
    const void* p;
};

enum norm_entry {
    NORM_LAYERNORM_FWD = 0,
    NORM_LAYERNORM_BWD = 1,
    NORM_ROPE_FWD = 2,
    NORM_ROPE_BWD = 3,
    NORM_RMSNORM_ROPE_FWD = 4,
    NORM_RMSNORM_ROPE_BWD = 5
};

/* Calls the entry point with the n arguments args[0 .. n-1] in its prototype's
 * order and returns what it returns. RMSN_EINVAL for an unknown entry, a number
 * of arguments other than the prototype's, or an integer that does not fit its
 * argument's type. The array is read before the call returns. */
int norm_call(int entry, const union norm_slot* args, int64_t n);

#ifdef __cplusplus
}
#endif

#endif /* SLOTS_GB300_H_ */
