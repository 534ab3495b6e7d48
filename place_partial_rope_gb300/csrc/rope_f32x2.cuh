// rope_f32x2.cuh -- fp32 arithmetic on pairs.
#pragma once
#include <cuda_runtime.h>
#include <string.h>

namespace rope {

// Two fp32 operations in one instruction, each rounded as the single one.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long x, y, z, d;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    memcpy(&z, &c, 8);
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
    float2 r;
    memcpy(&r, &d, 8);
    return r;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long x, y, d;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    float2 r;
    memcpy(&r, &d, 8);
    return r;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long x, y, d;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    float2 r;
    memcpy(&r, &d, 8);
    return r;
}

}  // namespace rope
