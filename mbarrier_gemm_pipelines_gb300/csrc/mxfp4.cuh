// mxfp4.cuh -- microscaled 4-bit floating point: blocks of 32 values with one
// power of two.
//
//   scale    2^(floor(log2 max |x|) - 2), stored as the biased exponent (E8M0),
//            at least 2^-127; 255 (NaN) where the block holds Inf or NaN
//   element  x / scale to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (E2M1, ties
//            to the even code), at most 6 in size
// as published for the format (Open Compute Project, microscaling formats).
// Both steps are exact but for the one rounding: a power of two divides without
// an error, or what underflows is nearest to 0 anyway.
//
// Scales lie in tiles of 128 rows x 4 blocks, 512 bytes: byte
// (row % 32) * 16 + (row % 128) / 32 * 4 + block % 4, which is the order in which
// the tensor core's copy into Tensor Memory takes them.
#pragma once
#include <cstdint>

namespace gbr {

constexpr int32_t kMxBlock = 32;                        // values
constexpr uint32_t kMxTileBytes = 512;                  // scales of 128 rows x 4 blocks

__host__ __device__ constexpr int64_t mx_scale_offset(int64_t row, int64_t block, int64_t block_tiles) {
    return (row / 128 * block_tiles + block / 4) * int64_t(kMxTileBytes) + row % 32 * 16 + row % 128 / 32 * 4 + block % 4;
}

// The scale's byte for the largest of the absolute values' bit patterns (as
// unsigned numbers: Inf and NaN are above every finite value).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
    if (top >= 0x7F800000u) return 255u;
    const uint32_t e = top >> 23;                       // 0 also below 2^-126, where the scale is 2^-127 anyway
    return e > 2u ? e - 2u : 0u;
}
// 1 / scale.
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
    return byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float mx_scale(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

// Eight values in [-8, 8] to eight 4-bit codes, the first in the low bits.
__device__ __forceinline__ uint32_t mx_pack8(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

__device__ __forceinline__ float mx_value(uint32_t code) {
    const uint32_t m = code & 7u;                       // 2 bits of exponent, 1 of mantissa
    const float size = m < 2u ? 0.5f * float(m) : __uint_as_float((126u + (m >> 1)) << 23 | (m & 1u) << 22);
    return code & 8u ? -size : size;
}

}  // namespace gbr
