// Activations of the projections and their derivatives, in fp32, each to a few
// roundings of the exact value of its fp32 argument:
//   silu       z s(z)                        s + z s (1 - s)
//   sigmoid    s(z)                          s (1 - s)
//   gelu       z P(z), P = erfc(-z / sqrt 2) / 2      P + z exp(-z^2 / 2) / sqrt(2 pi)
//   gelu_tanh  z s(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3)   (1 + tanh u = 2 s(2 u))
//              s + z s (1 - s) 2 u'
//   relu       z where z > 0, else 0         1 where z > 0, else 0
// 1 - s comes as s(-z), and P from erfc, not 1 + erf: neither cancels in a tail.
#pragma once

#include "common.cuh"
#include "linear.h"

namespace rmsn {

// s(z) and s(-z) = 1 - s(z).
__device__ __forceinline__ float2 sigmoid_pair(float z) {
    const float e = exp_neg(fabsf(z));
    const float s = rcp_1to2(fadd(1.0f, e)), t = fmul(e, s);
    return z >= 0.0f ? make_float2(s, t) : make_float2(t, s);
}

// 2 u of gelu_tanh and its derivative. Past |z| = 16 s(2 u) is 0 or 1 in fp32
// (2 u is over 300 there) and the slope is held at its value there, so that z^3
// cannot pass fp32's range and leave 0 times infinity.
__device__ __forceinline__ float2 gelu_tanh_arg(float z) {
    constexpr float k = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float v = fminf(fmaxf(z, -16.0f), 16.0f), v2 = fmul(v, v);
    return make_float2(fmul(fmul(k, v), __fmaf_rn(0.044715f, v2, 1.0f)), fmul(k, __fmaf_rn(0.134145f, v2, 1.0f)));
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == LINEAR_ACT_SILU) return fmul(z, sigmoidf_rn(z));
    else if constexpr (ACT == LINEAR_ACT_SIGMOID) return sigmoidf_rn(z);
    else if constexpr (ACT == LINEAR_ACT_GELU) return fmul(z, fmul(0.5f, erfcf(fmul(z, -0.70710678118654752f))));
    else if constexpr (ACT == LINEAR_ACT_GELU_TANH) {
        const float a = gelu_tanh_arg(z).x;
        return fmul(z, sigmoidf_rn(z != z ? z : a));  // fmin and fmax drop a NaN
    } else if constexpr (ACT == LINEAR_ACT_RELU) return z > 0.0f || z != z ? z : 0.0f;
    else return z;
}

// The activation and its derivative.
template <int ACT>
__device__ __forceinline__ float2 act_slope(float z) {
    if constexpr (ACT == LINEAR_ACT_SILU) {
        const float2 s = sigmoid_pair(z);
        const float q = fmul(z, s.x);
        return make_float2(q, __fmaf_rn(q, s.y, s.x));
    } else if constexpr (ACT == LINEAR_ACT_SIGMOID) {
        const float2 s = sigmoid_pair(z);
        return make_float2(s.x, fmul(s.x, s.y));
    } else if constexpr (ACT == LINEAR_ACT_GELU) {
        const float p = fmul(0.5f, erfcf(fmul(z, -0.70710678118654752f)));
        const float d = fmul(0.39894228040143268f, exp_neg(fmul(0.5f, fmul(z, z))));
        return make_float2(fmul(z, p), __fmaf_rn(z, d, p));
    } else if constexpr (ACT == LINEAR_ACT_GELU_TANH) {
        const float2 a = gelu_tanh_arg(z);
        const float2 s = sigmoid_pair(z != z ? z : a.x);
        const float q = fmul(z, s.x);
        return make_float2(q, __fmaf_rn(fmul(q, s.y), a.y, s.x));
    } else if constexpr (ACT == LINEAR_ACT_RELU) {
        return z > 0.0f || z != z ? make_float2(z, z != z ? z : 1.0f) : make_float2(0.0f, 0.0f);
    } else {
        return make_float2(z, 1.0f);
    }
}

// f(ACT) with the activation as a compile-time constant, for a valid `act`.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case LINEAR_ACT_SILU: f(std::integral_constant<int, LINEAR_ACT_SILU>()); break;
        case LINEAR_ACT_SIGMOID: f(std::integral_constant<int, LINEAR_ACT_SIGMOID>()); break;
        case LINEAR_ACT_GELU: f(std::integral_constant<int, LINEAR_ACT_GELU>()); break;
        case LINEAR_ACT_GELU_TANH: f(std::integral_constant<int, LINEAR_ACT_GELU_TANH>()); break;
        case LINEAR_ACT_RELU: f(std::integral_constant<int, LINEAR_ACT_RELU>()); break;
        default: f(std::integral_constant<int, LINEAR_ACT_NONE>()); break;
    }
}

}  // namespace rmsn
