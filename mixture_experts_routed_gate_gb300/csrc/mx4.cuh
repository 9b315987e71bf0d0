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

// How many of `size` rows from row `first` on there are (none: 0 or less): the
// tables lie on the device, and those of a larger batch name rows past the call's own,
// which are neither read nor written; nor are rows below 0.  Minima alone: a selection
// by one of an expert's entries becomes a branch with the loads of the others behind
// it, and this stands before the first copy of every launch (a 4-bit product of 384
// rows of 64 experts, 2048 x 768: 12.6 us for 12.1).
__device__ __forceinline__ int rows_there(const MxTables &t, int size, int first) {
    const int behind = static_cast<int>(static_cast<uint32_t>(t.n_rows) - static_cast<uint32_t>(first));
    return min(min(size, behind), first | INT32_MAX);  // the last: -1 below 0
}

// Rows of M block bx of the dispatch tables: expert, first row, count.  Units of
// ROWS rows: every block, or every other one of an expert with the block behind it.
// A block's end may pass 32 bits, its rows' offsets do not.
template <int ROWS> __device__ __forceinline__ Mx4Block mx_unit_of(const MxTables &t, int bx, int m_blocks) {
    Mx4Block b;
    b.g = static_cast<int>(min(static_cast<unsigned>(t.gidx[bx]), static_cast<unsigned>(t.E - 1)));
    const int off = static_cast<int>(static_cast<uint32_t>(bx) * 128u - static_cast<uint32_t>(t.padded[b.g]));
    b.m_start = off + t.offsets[b.g];
    b.rows = max(0, rows_there(t, min(t.sizes[b.g] - off, ROWS), b.m_start));
    if (ROWS > 128) b.rows = off % ROWS != 0 ? 0 : bx + 1 == m_blocks ? min(b.rows, 128) : b.rows;
    return b;
}

}  // namespace moe
