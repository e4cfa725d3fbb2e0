// Packed fp32 arithmetic: two values in a register pair, both done in one issue
// slot.
#pragma once

#include <cuda_runtime.h>

namespace bq {

typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 two(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ f32x2 both(float v) { return two(v, v); }

__device__ __forceinline__ float2 parts_of(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float sum2(f32x2 v) {
    const float2 p = parts_of(v);
    return p.x + p.y;
}

}  // namespace bq
