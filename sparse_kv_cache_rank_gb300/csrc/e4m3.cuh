// e4m3.cuh -- conversions between fp32 and E4M3 (round to nearest even, saturating; NaN stays NaN), and
// the power-of-two scales (E8M0: byte b stands for 2^(b - 127)) of the 8-bit pages.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace dllm {

// Two values to two codes, `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_of_half2(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}
// Two codes (the low 16 bits) to fp16: exact.
__device__ __forceinline__ uint32_t half2_of_e4m3x2(uint32_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)c));
    return r;
}
__device__ __forceinline__ float2 f32_of_e4m3x2(uint32_t c) {
    const uint32_t h = half2_of_e4m3x2(c);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

__device__ __forceinline__ float e8m0_f32(int byte) { return __uint_as_float((uint32_t)byte << 23); }   // (byte 0: 0)

// The scale's byte for values of at most `amax`: the least exponent e from -64 to 63 with
// amax <= 448 2^e (448 = 1.75 2^8; larger values saturate).
__device__ __forceinline__ int e8m0_for(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);
    return 127 + min(max(e, -64), 63);
}
// 2^(127 - byte): the factor that brings values to codes under that scale (byte 63 .. 190).
__device__ __forceinline__ float e8m0_inverse(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }

}  // namespace dllm
