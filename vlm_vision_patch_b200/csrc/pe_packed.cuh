// Packed fp32 arithmetic of sm_100: one instruction for two values.
#pragma once

#include <cstdint>

namespace pe {

// Two fp32 lanes per instruction.
__device__ __forceinline__ uint64_t bits2(float2 v) { return (uint64_t)__float_as_uint(v.x) | (uint64_t)__float_as_uint(v.y) << 32; }
__device__ __forceinline__ float2 float2_of(uint64_t b) {
    return make_float2(__uint_as_float((uint32_t)b), __uint_as_float((uint32_t)(b >> 32)));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return float2_of(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
    return float2_of(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
    return float2_of(d);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

}  // namespace pe
