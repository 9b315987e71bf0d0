// mx8.cuh -- the arithmetic of the 8-bit block-scaled format (e4m3 elements,
// one power-of-two scale per 32), shared by the norm, the quantiser and the
// grouped product.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {

// The scale byte of a block, from the bits of its largest magnitude (as
// unsigned numbers those order like the values, then infinity, then NaNs): the
// least power of two, 2^-127 at least, that brings it to 448 = 1.75 * 2^8 or
// less; 255 for an infinity or a NaN.
__device__ __forceinline__ uint32_t mx8_scale(uint32_t top) {
    const int field = static_cast<int>(top >> 23);
    if (field == 255) return 255u;
    return static_cast<uint32_t>(max(field - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0), 0));
}

// 2^(127 - byte), exact: byte <= 247; for 255, where elements are zeros, 0
__device__ __forceinline__ float mx8_inverse(uint32_t byte) {
    return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127); byte 255 is NaN
__device__ __forceinline__ float mx8_factor(uint32_t byte) {
    if (byte == 255u) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(byte ? byte << 23 : 1u << 22);
}

// the largest magnitude of three, NaN if one of them is
__device__ __forceinline__ float largest(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// two elements, a in the low byte: to nearest even
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
    return r;
}

// Four elements to a word, first in the lowest byte, each times `by`.  A block
// whose scale byte is 255 holds zeros: their product with the scale is NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float by, bool bad) {
    const uint32_t w = e4m3x2(a * by, b * by) | e4m3x2(c * by, d * by) << 16;
    return bad ? 0u : w;
}

// the two elements in the low 16 bits, low byte first, exact
__device__ __forceinline__ float2 e4m3x2_values(uint32_t bits) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(bits));
    return unpack2<kF16>(r);
}

}  // namespace moe
