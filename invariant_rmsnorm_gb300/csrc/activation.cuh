// Activations of the projections and their derivatives, in fp32:
//   silu       z s(z)                        s + z s (1 - s)
//   sigmoid    s(z)                          s (1 - s)
//   gelu       z P(z), P = (1 + erf(z / sqrt 2)) / 2  P + z exp(-z^2 / 2) / sqrt(2 pi)
//   gelu_tanh  z s(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3)   (1 + tanh u = 2 s(2 u))
//              s + z s (1 - s) 2 u'
//   relu       z where z > 0, else 0         1 where z > 0, else 0
// 1 - s comes as s(-z), and P of a negative z as the tail itself: neither cancels.
//
// Relative error, of the exact value at the fp32 argument (a derivative's of the larger of its two terms): a few roundings
// (2^-24 each; gelu's fit 3.3e-7) near zero and above. In the tail below zero the value is an exponential e^-a, and its
// error grows with a: that of exp_neg, (5 + a) 2^-24, and a times that of a itself. Together at most about a roundings for
// silu and sigmoid (a = |z|: 80 at z = -80), 2 a for gelu (a = z^2 / 2: 100 at z = -10) and 5 a for gelu_tanh (a = |2 u|: 250 at
// z = -8), of the 2^15 and more that half a step of bf16 is, 2^12 of fp16.
#pragma once

#include <type_traits>

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

// P(z) of gelu and exp(-z^2 / 2). The tail beyond |z| is exp(-x^2) w(x) / 2 with x = |z| / sqrt 2 and
// w(x) = exp(x^2) erfc(x) = t q(t), t = 1 / (1 + 0.38 x); q, of degree 8, is a fit of w(x) / t
// over 0 <= x <= 14 (reweighted least squares of the relative error, which is 2.5e-8 at most; evaluated
// in fp32 3.3e-7). Beyond 14 the exponential is zero in fp32. One exponential and one reciprocal serve the value and
// the slope: slopes of 8192 x 16384 in 266 us with CUDA's erfcf beside an exponential.
__device__ __forceinline__ float2 normal_cdf(float z) {
    const float a = fabsf(z);
    float t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(__fmaf_rn(a, 0.26870057685088806f, 1.0f)));  // 0.38 / sqrt 2
    float q = __fmaf_rn(5.842188462318101e-2f, t, -2.5986075030418665e-1f);
    q = __fmaf_rn(q, t, 3.593394501458925e-1f);
    q = __fmaf_rn(q, t, -1.5683961581211492e-1f);
    q = __fmaf_rn(q, t, 2.2721908166812357e-1f);
    q = __fmaf_rn(q, t, 1.3968038468555605e-1f);
    q = __fmaf_rn(q, t, 2.0368526881511956e-1f);
    q = __fmaf_rn(q, t, 2.1394445150561897e-1f);
    q = __fmaf_rn(q, t, 2.1440983279273618e-1f);
    const float e = exp_neg(fmul(0.5f, fmul(a, a)));
    const float tail = fmul(fmul(0.5f, e), fmul(q, t));
    return make_float2(z < 0.0f ? tail : fsub(1.0f, tail), e);
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == LINEAR_ACT_SILU) return fmul(z, sigmoidf_rn(z));
    else if constexpr (ACT == LINEAR_ACT_SIGMOID) return sigmoidf_rn(z);
    else if constexpr (ACT == LINEAR_ACT_GELU) return fmul(z, normal_cdf(z).x);
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
        const float2 p = normal_cdf(z);
        return make_float2(fmul(z, p.x), __fmaf_rn(fmul(z, 0.39894228040143268f), p.y, p.x));
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
