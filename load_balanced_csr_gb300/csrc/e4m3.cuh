// 8-bit floating-point codes: four exponent and three mantissa bits, no
// infinities, largest value 448, NaN 0x7f.
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

namespace lbcsr {

// Two codes of two 32-bit values, rounded to the nearest, ties to even; values
// past 448 become 448, NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two codes as two 16-bit values, exactly: every code is one.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
    return r;
}
// Four codes.
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t codes, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
    const uint32_t pair = e4m3x2_to_half2(codes);
    __half2 h;
    memcpy(&h, &pair, 4);
    return __half22float2(h);
}

}  // namespace lbcsr
