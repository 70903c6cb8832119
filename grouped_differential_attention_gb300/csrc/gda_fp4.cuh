// Conversions of the 4-bit cache format: e2m1 codes, two to a byte (the even
// element in the low half), one e4m3 scale for 16 consecutive elements of a
// head row, one float32 scale for each head.  value = code * block * head.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

namespace gda {

constexpr int kFp4Block = 16;   // elements that share one e4m3 scale

// The two e4m3 values in the low 16 bits of `b` (element 0 in the low byte) as half2; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(r)
        : "r"(b));
    return r;
}

// Four bytes of two e2m1 codes each as four half2 (low code in the low half); exact.
__device__ __forceinline__ void e2m1x8_to_half2x4(uint32_t (&h)[4], uint32_t codes) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

__device__ __forceinline__ float2 half2_bits_to_float2(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

__device__ __forceinline__ float e4m3_to_float(uint8_t b) { return half2_bits_to_float2(e4m3x2_to_half2(b)).x; }

// The e4m3 byte nearest to x >= 0 (ties to even, at most 448; NaN gives NaN).
__device__ __forceinline__ uint8_t float_to_e4m3(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return static_cast<uint8_t>(r);
}

// The byte of two e2m1 codes nearest to lo and hi (ties to even, at most 6 in magnitude).
__device__ __forceinline__ uint32_t float2_to_e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
        "cvt.u32.u8 %0, b;\n\t}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}

}  // namespace gda
