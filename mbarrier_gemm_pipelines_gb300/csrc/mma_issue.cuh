// mma_issue.cuh -- issuing small MMAs from one thread without losing time.
//
// A tcgen05.mma of M = 128 and N <= 64 keeps the tensor core busy for 40 to 50
// cycles, no longer than it takes one thread to build two 64-bit descriptors,
// a predicate and a ring position for it: measured, 77 cycles an MMA with the
// descriptors made for each, 46 with running ones.  So the constant halves of
// the descriptors are made once, the low words (the shared-memory address in
// 16-byte units) advance by additions, and the four MMAs of a 64-k slice are
// one block.
#pragma once
#include <cstdint>

#include "gbr_ptx.cuh"

namespace gbr {

// High and low words of a shared-memory matrix descriptor with the 128-byte
// swizzle (bit layout: see sw128_desc in gemm_umma.cuh).
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo) {
    return ((sbo >> 4) & 0x3FFFu) | (1u << 14) | (2u << 29);
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
    return ((saddr >> 4) & 0x3FFFu) | (((lbo >> 4) & 0x3FFFu) << 16);
}
// From one K = 16 step to the next, in 16-byte units: 32 bytes along a K-major
// row, 16 rows of 128 bytes of an MN-major panel.
constexpr uint32_t kStepK = 2, kStepMN = 128;

// Four steps of K = 16 (a 64-k slice): d (+)= a b, bf16; `accumulate` 0 starts
// the sum with the first.
template <uint32_t A_STEP, uint32_t B_STEP>
__device__ __forceinline__ void mma_slice(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b32 a1, a2, a3, b1, b2, b3;\n\t"
        ".reg .b64 A0, A1, A2, A3, B0, B1, B2, B3;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.u32 a1, %1, %6;\n\tadd.u32 a2, %1, %7;\n\tadd.u32 a3, %1, %8;\n\t"
        "add.u32 b1, %2, %9;\n\tadd.u32 b2, %2, %10;\n\tadd.u32 b3, %2, %11;\n\t"
        "mov.b64 A0, {%1, %3};\n\tmov.b64 A1, {a1, %3};\n\tmov.b64 A2, {a2, %3};\n\tmov.b64 A3, {a3, %3};\n\t"
        "mov.b64 B0, {%2, %3};\n\tmov.b64 B1, {b1, %3};\n\tmov.b64 B2, {b2, %3};\n\tmov.b64 B3, {b3, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], A0, B0, %4, p;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], A1, B1, %4, t;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], A2, B2, %4, t;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], A3, B3, %4, t;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "n"(A_STEP), "n"(2 * A_STEP), "n"(3 * A_STEP),
        "n"(B_STEP), "n"(2 * B_STEP), "n"(3 * B_STEP)
        : "memory");
}

// A stage of microscaled 4-bit operands (256 values of a row): the scales' copies into Tensor Memory and four MMAs of
// K = 64.  At s_lo lies 1 KiB for the 128 rows of A, then 1 KiB for each of
// N_TILES times 128 rows of B, each two tiles of 512 bytes (4 blocks); they go to 8 columns from sfa and 8 N_TILES from
// sfb, those of the first 4 blocks first.
template <int PAIR, int N_TILES>
__device__ __forceinline__ void mx_copy_scales(uint32_t s_lo, uint32_t s_hi, uint32_t sfa, uint32_t sfb) {
    auto copy = [&](uint32_t to, uint32_t from) {
        const uint64_t desc = uint64_t(from) | (uint64_t(s_hi) << 32);
        if (PAIR == 2) ptx::tmem_copy_32x128b_pair(to, desc);
        else ptx::tmem_copy_32x128b(to, desc);
    };
#pragma unroll
    for (uint32_t h = 0; h < 2; ++h) {
        copy(sfa + h * 4u, s_lo + h * 32u);
#pragma unroll
        for (uint32_t r = 0; r < uint32_t(N_TILES); ++r)
            copy(sfb + (h * N_TILES + r) * 4u, s_lo + 64u * (1u + r) + h * 32u);
    }
}

// `steps` (1 to 4) of the MMAs; idesc0 and idesc1 name the first and the second two of four blocks.
template <int PAIR, int N_TILES>
__device__ __forceinline__ void mx_mmas(int32_t steps, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t sfa,
                                        uint32_t sfb, uint32_t idesc0, uint32_t idesc1, uint32_t accumulate) {
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
        if (int32_t(k) >= steps) break;
        const uint64_t a = uint64_t(a_lo + kStepK * k) | (uint64_t(hi) << 32);
        const uint64_t b = uint64_t(b_lo + kStepK * k) | (uint64_t(hi) << 32);
        const uint32_t fa = sfa + k / 2u * 4u, fb = sfb + k / 2u * (4u * N_TILES), id = k % 2u ? idesc1 : idesc0;
        const uint32_t acc = k == 0 ? accumulate : 1u;
        if (PAIR == 2) ptx::mma_mxf4_pair(d, a, b, id, fa, fb, acc);
        else ptx::mma_mxf4(d, a, b, id, fa, fb, acc);
    }
}

}  // namespace gbr
