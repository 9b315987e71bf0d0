// mx4.cuh -- the arithmetic of the 4-bit block-scaled format, shared by the
// quantiser and the grouped product.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {

// the scale byte of a block whose largest magnitude is `top`: floor(log2) is
// in the exponent field; 255 for a NaN or an infinity
__device__ __forceinline__ uint32_t mx4_scale(float top) {
    const int field = static_cast<int>(__float_as_uint(top) >> 23) & 255;
    if (field == 255) return 255u;
    return static_cast<uint32_t>(max(field - 2, 0));
}

// 2^(127 - byte) for byte <= 252, exact
__device__ __forceinline__ float mx4_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 2^(byte - 127); byte 255 is NaN
__device__ __forceinline__ float mx4_factor(uint32_t byte) {
    if (byte == 255u) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(byte ? byte << 23 : 1u << 22);
}

// eight elements to a word, first in the lowest nibble: each times `by`, to
// nearest even, limited to 6
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8], float by) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0] * by), "f"(v[1] * by), "f"(v[2] * by), "f"(v[3] * by), "f"(v[4] * by), "f"(v[5] * by), "f"(v[6] * by),
          "f"(v[7] * by));
    return r;
}

// the two elements of a byte, low nibble first
__device__ __forceinline__ float2 e2m1x2_values(uint32_t byte) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(byte));
    return unpack2<kF16>(r);
}

struct Mx4Block {
    int g, m_start, rows;
};

// How many of an expert's `size` rows from row `first` on there are: the tables
// lie on the device, and those of a larger batch name rows past the call's own,
// which are neither read nor written.
__device__ __forceinline__ int64_t rows_there(const MxTables &t, int size, int first, int32_t *err) {
    const int64_t there = first < 0 ? 0 : t.n_rows - first;
    if (size > there && err) atomicExch(err, kErrDeviceFlag);
    return min(static_cast<int64_t>(size), there);
}

// Rows of M block bx of the dispatch tables: expert, first row, count.  Units of
// ROWS rows: every block, or every other one of an expert with the block behind it.
template <int ROWS> __device__ __forceinline__ Mx4Block mx_unit_of(const MxTables &t, int bx, int m_blocks, int32_t *err) {
    const int g = t.gidx[bx];
    if (g < 0 || g >= t.E) return {0, 0, 0};
    const int64_t at = static_cast<int64_t>(bx) * 128, off = at - t.padded[g], here = static_cast<int64_t>(m_blocks) * 128 - at;
    if (off < 0 || off % ROWS != 0) return {g, 0, 0};
    const int first = t.offsets[g];
    const int64_t rows = min(min(rows_there(t, t.sizes[g], first, err) - off, here), static_cast<int64_t>(ROWS));
    return rows > 0 ? Mx4Block{g, static_cast<int>(first + off), static_cast<int>(rows)} : Mx4Block{g, 0, 0};
}

}  // namespace moe
