// Two floats at once (packed 32-bit operations).
#pragma once

namespace sdm {

__device__ __forceinline__ unsigned long long &pair_bits(float2 &x) { return reinterpret_cast<unsigned long long &>(x); }

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(pair_bits(d)) : "l"(pair_bits(a)), "l"(pair_bits(b)), "l"(pair_bits(c)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(pair_bits(d)) : "l"(pair_bits(a)), "l"(pair_bits(b)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(pair_bits(d)) : "l"(pair_bits(a)), "l"(pair_bits(b)));
    return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

}  // namespace sdm
