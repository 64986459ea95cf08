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

// A negative frequency is the complement of its size's fraction: the fraction of
// the frequency itself, 1 less a small number, would be rounded at 2^-54 turns.
__device__ __forceinline__ unsigned long long rope_turns(double inv_freq) {
    const double t = fabs(inv_freq) * 0.15915494309189533577;  // 1 / (2 pi)
    const unsigned long long F = __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
    return inv_freq < 0.0 ? 0ull - F : F;
}

// scale (cos, sin) of position p at the frequency F. Of the phase (64 bits of a
// turn) the nearest quarter turn is taken off in integers. Of what is left, |y| <=
// pi / 4, the upper 32 bits and 23 of the lower ones become the angle: a small
// angle keeps fp32's relative precision down to 2^-32 turns, and its error is
// below 2^-55 turns throughout (with the upper 32 bits alone it was up to 2^-32:
// 1 % of the sine of a pair of frequency 1e-7 at position 1; the three
// instructions more cost calls of tokens with one to four heads 1 to 2 %, others
// none). It goes through the Taylor series of sine (to y^9,
// remainder below 2^-29) and cosine (to y^10, below 2^-31) in fp32.
__device__ __forceinline__ float2 rope_cos_sin(long long p, unsigned long long F, float scale) {
    constexpr float kStep = 1.4629180792671596e-9f;  // 2 pi / 2^32
    const unsigned long long turn = static_cast<unsigned long long>(p) * F;  // modulo one turn
    const uint32_t hi = static_cast<uint32_t>(turn >> 32), lo = static_cast<uint32_t>(turn);
    const uint32_t quarter = (hi + 0x20000000u) >> 30;
    // 2^23 + the lower half's 23 bits, then their part of a step: both exact but for one rounding.
    const float low = __fmaf_rn(__uint_as_float(0x4b000000u | (lo >> 9)), kStep * 0x1p-23f, -kStep);
    const float y = __fmaf_rn(static_cast<float>(static_cast<int>(hi - (quarter << 30))), kStep, low);
    const float z = fmul(y, y);
    float s = __fmaf_rn(z, 2.7557319223985893e-6f, -1.9841269841269841e-4f);  // 1/9!, -1/7!
    s = __fmaf_rn(s, z, 8.3333333333333333e-3f);
    s = __fmaf_rn(s, z, -1.6666666666666667e-1f);
    s = __fmaf_rn(fmul(s, z), y, y);
    float c = __fmaf_rn(z, -2.7557319223985891e-7f, 2.4801587301587302e-5f);  // -1/10!, 1/8!
    c = __fmaf_rn(c, z, -1.3888888888888889e-3f);
    c = __fmaf_rn(c, z, 4.1666666666666667e-2f);
    c = __fmaf_rn(c, z, -0.5f);
    c = __fmaf_rn(c, z, 1.0f);
    const bool odd = quarter & 1u;
    float cq = odd ? s : c, sq = odd ? c : s;  // quarter turns: (c, s), (-s, c), (-c, -s), (s, -c)
    cq = ((quarter + 1u) & 2u) ? -cq : cq;
    sq = (quarter & 2u) ? -sq : sq;
    return make_float2(fmul(cq, scale), fmul(sq, scale));
}

}  // namespace rmsn
