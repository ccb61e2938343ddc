// The 8-bit cache: codes are e4m3 floats (largest 448, no infinities), a value
// is code * scale with an fp32 scale for each page and kv head.
#pragma once

#include <cuda_fp8.h>

#include "pa_device.cuh"

namespace pa {

constexpr float kE4m3Max = 448.f;
// Scales that the append writes, and that the attention takes, lie in here.
constexpr float kMinScale8 = 0x1p-60f, kMaxScale8 = 0x1p60f;

// The smallest power of two s with amax <= 448 s, inside the limits.  448 is
// 1.75 * 2^8: the exponent of amax less 8, or less 7 where its mantissa is
// above 1.75.
__device__ __forceinline__ float scale_for(float amax) {
    const uint32_t u = __float_as_uint(amax);
    int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = amax == 0.f ? -60 : min(max(e, -60), 60);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two codes, x0's in the low byte; what e4m3 cannot hold (past 448, infinite)
// becomes NaN instead of the largest code.
__device__ __forceinline__ uint32_t encode2(float x0, float x1) {
    x0 = fabsf(x0) <= kE4m3Max ? x0 : __int_as_float(0x7fffffff);
    x1 = fabsf(x1) <= kE4m3Max ? x1 : __int_as_float(0x7fffffff);
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
    return r;
}
// The values of two codes as packed fp16, which holds each of them exactly.
__device__ __forceinline__ uint32_t decode2(uint16_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
    return r;
}

}  // namespace pa
