// Angles of rotary positions, as fractions of a turn in 64-bit integers.
//
// A frequency f (radians a position) becomes F = frac(f / 2 pi) 2^64. The angle
// of position p is then p F modulo 2^64, an exact integer product: the only
// errors are F's own (the fp64 rounding of f / 2 pi, 2^-53 relative, and half a
// step of 2^-64 turns), both multiplied by p, as in an fp64 product p f. No
// range reduction of a large angle is left to do, and no fp64 arithmetic
// remains per position.
#pragma once

#include "common.cuh"

namespace rmsn {

__device__ __forceinline__ unsigned long long rope_turns(double inv_freq) {
    const double t = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
    return __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
}

// scale (cos, sin) of position p at the frequency F. The phase, a signed 64-bit
// number of half turns / 2^63, keeps 24 bits as a float: an error of at most
// pi 2^-25 in the angle.
__device__ __forceinline__ float2 rope_cos_sin(long long p, unsigned long long F, float scale) {
    const long long phase = static_cast<long long>(static_cast<unsigned long long>(p) * F);
    float s, c;
    sincospif(__ll2float_rn(phase) * 1.0842021724855044e-19f, &s, &c);  // 2^-63
    return make_float2(fmul(c, scale), fmul(s, scale));
}

// (u, v) turned by the angle of cs = scale (cos, sin); backward: by minus it.
__device__ __forceinline__ float2 rope_turn(float u, float v, float2 cs) {
    return make_float2(fsub(fmul(u, cs.x), fmul(v, cs.y)), fadd(fmul(v, cs.x), fmul(u, cs.y)));
}

}  // namespace rmsn
