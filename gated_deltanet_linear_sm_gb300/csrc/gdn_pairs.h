// Internal to libgdnspec: FP32 arithmetic on pairs (fma.rn.f32x2 and its like:
// each half rounds as the scalar instruction would, at half the instructions).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace gdn_common {

typedef unsigned long long u64;

__device__ __forceinline__ u64 pk2(float a, float b) {
    return (static_cast<u64>(__float_as_uint(b)) << 32) | __float_as_uint(a);
}
__device__ __forceinline__ float lo2(u64 v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi2(u64 v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ u64 ffma2(u64 a, u64 b, u64 c) {
    u64 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ u64 fmul2(u64 a, u64 b) {
    u64 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ u64 add2(u64 a, u64 b) {
    u64 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ u64 dup2(float x) { return pk2(x, x); }
__device__ __forceinline__ u64 raw2(uint32_t a, uint32_t b) { return (static_cast<u64>(b) << 32) | a; }
// the two bf16 of a word as a pair of floats
__device__ __forceinline__ u64 widen(uint32_t w) { return raw2(w << 16, w & 0xffff0000u); }
__device__ __forceinline__ u64 sub2(u64 a, u64 b) { return ffma2(b, dup2(-1.0f), a); }

}  // namespace gdn_common
