// Conversions of the 8-bit cache format: e4m3 codes, one float32 scale for
// each block of tokens and head.  value = code * scale.
#pragma once

#include <cstdint>

#include "gda_device.cuh"
#include "gda_fp4.cuh"

namespace gda {

// The e4m3 bytes nearest to lo and hi (ties to even, at most 448 in magnitude; NaN gives NaN), lo in the low byte.
__device__ __forceinline__ uint32_t float2_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four e4m3 bytes as two half2; exact.
__device__ __forceinline__ uint2 e4m3x4_to_half2x2(uint32_t codes) {
    return make_uint2(e4m3x2_to_half2(codes), e4m3x2_to_half2(codes >> 16));
}

// The least power of two s >= 2^-126 with amax <= 448 s, for amax >= 0 given by its float32 bits (finite).
__device__ __forceinline__ float fp8_scale_of(uint32_t amax_bits) {
    // 448 = 1.75 * 2^8: the exponent of amax less 8, and one more where its digits are above 1.75
    const int e = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u);
    return __uint_as_float(static_cast<uint32_t>(e < 1 ? 1 : e) << 23);
}

}  // namespace gda
