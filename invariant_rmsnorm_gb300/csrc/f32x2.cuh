// Eight values of a 16-byte vector as four pairs of fp32, and arithmetic on pairs.
//
// A pair's operations are one instruction, each half rounded as the scalar
// operation is: half the issue slots. Every product that feeds a sum is an
// explicit fused multiply-add, so nothing is left for ptxas to contract.
#pragma once

#include "common.cuh"

namespace rmsn {

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

struct Oct { float2 p[4]; };

__device__ __forceinline__ Oct oct_zero() {
    Oct o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.p[i] = make_float2(0.0f, 0.0f);
    return o;
}

template <bool F16>
__device__ __forceinline__ Oct oct_unpack(const uint4 v) {
    float f[8];
    unpack_act<F16>(v, f);
    Oct o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.p[i] = pair(f, 2 * i);
    return o;
}

template <bool F16>
__device__ __forceinline__ uint4 oct_pack(const Oct& o) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = o.p[i].x;
        f[2 * i + 1] = o.p[i].y;
    }
    return pack_act<F16>(f);
}

__device__ __forceinline__ Oct oct_of(float4 lo, float4 hi) {
    Oct o;
    o.p[0] = make_float2(lo.x, lo.y); o.p[1] = make_float2(lo.z, lo.w);
    o.p[2] = make_float2(hi.x, hi.y); o.p[3] = make_float2(hi.z, hi.w);
    return o;
}

__device__ __forceinline__ Oct load_oct(const float* p) {
    return oct_of(__ldg(reinterpret_cast<const float4*>(p)), __ldg(reinterpret_cast<const float4*>(p) + 1));
}

// Effective weights of vector v.
__device__ __forceinline__ Oct oct_weights(const float* w, int zc, int v) {
    Oct o = load_oct(w + 8 * v);
    if (zc) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o.p[i] = fadd2(o.p[i], both(1.0f));
    }
    return o;
}

// Asynchronous 16-byte copies past L1 to shared memory, in groups. A thread that
// reads only what it copied itself needs no other synchronisation than its wait.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

}  // namespace rmsn
