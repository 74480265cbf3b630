// dropout.cuh -- the dropout mask as a pure function of (seed, offset, row,
// column): Philox-4x32 with 10 rounds, the counter-based generator of J. K.
// Salmon, M. A. Moraes, R. O. Dror and D. E. Shaw, "Parallel random numbers:
// as easy as 1, 2, 3" (SC 2011).  Nothing is stored: the backward pass, or any
// other kernel that knows the position, computes the same mask again.
//
// One call of the generator serves 8 neighbouring columns:
//   counter = (column / 8, row, offset low, offset high), key = (seed low, high)
//   column c takes 16 bits: word (c % 8) / 2, the low half for even c
//   keep when those 16 bits, as an unsigned number, are >= threshold,
//   threshold = round(65536 p); kept values are multiplied by
//   65536 / (65536 - threshold), so the mean is exactly the input's.
// 16 bits a column (p in steps of 1.5e-5) cost half the generator calls of 32.
#pragma once
#include <cstdint>

namespace gbr {

struct Dropout {
    uint32_t threshold;          // 0: keep everything (no generator calls)
    float scale;
    uint32_t key0, key1;         // seed
    uint32_t off0, off1;         // offset
};

__device__ __forceinline__ uint4 philox4x32_10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                               uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = uint64_t(0xD2511F53u) * c0, b = uint64_t(0xCD9E8D57u) * c2;
        c0 = uint32_t(b >> 32) ^ c1 ^ k0;
        c1 = uint32_t(b);
        c2 = uint32_t(a >> 32) ^ c3 ^ k1;
        c3 = uint32_t(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// The 128 random bits of columns [8 col8, 8 col8 + 8) of `row`.
__device__ __forceinline__ uint4 dropout_bits(const Dropout& d, uint32_t row, uint32_t col8) {
    return philox4x32_10(col8, row, d.off0, d.off1, d.key0, d.key1);
}

// Whether column 8 col8 + i (0 <= i < 8) of those bits is kept.
__device__ __forceinline__ bool dropout_keep(const Dropout& d, const uint4& bits, int i) {
    const uint32_t w = i < 2 ? bits.x : i < 4 ? bits.y : i < 6 ? bits.z : bits.w;
    return ((i & 1) ? (w >> 16) : (w & 0xFFFFu)) >= d.threshold;
}

}  // namespace gbr
