// row8.cuh -- a row of a matrix held by a group of threads, V times eight
// elements each, as fp32 (the operators that need a whole row at once), and
// sums over the group.
//
// VEC: the thread's eight are neighbours, moved 16 (bf16) or 32 bytes (fp32) at
// a time; rows start on 16 bytes and the columns are a multiple of 8.
// Otherwise they lie `tpr` columns apart, so that a warp touches whole lines at
// any alignment.
#pragma once
#include "gbr_ptx.cuh"
#include "vec8.cuh"

namespace gbr {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float* y) { *y = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16* y) { *y = __float2bfloat16_rn(x); }

// Column of element j of vector v of thread `t` of `tpr`.
template <bool VEC>
__device__ __forceinline__ int32_t row_col(int v, int j, int32_t t, int32_t tpr) {
    return VEC ? (v * tpr + t) * 8 + j : (v * 8 + j) * tpr + t;
}

// Eight elements as they are loaded; columns past the end are zero.
template <typename T>
struct Raw8 {
    uint32_t w[sizeof(T) * 2];
};

template <bool VEC>
__device__ __forceinline__ void load_raw8(Raw8<__nv_bfloat16>& r, const __nv_bfloat16* row, int v, int32_t t,
                                          int32_t tpr, int32_t cols) {
    if (VEC) {
        const int32_t c = row_col<true>(v, 0, t, tpr);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (c < cols) x = *reinterpret_cast<const uint4*>(row + c);
        r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const int32_t c = row_col<false>(v, j, t, tpr), d = c + tpr;
            const uint32_t lo = c < cols ? __bfloat16_as_ushort(row[c]) : 0u;
            const uint32_t hi = d < cols ? __bfloat16_as_ushort(row[d]) : 0u;
            r.w[j / 2] = lo | (hi << 16);
        }
    }
}
template <bool VEC>
__device__ __forceinline__ void load_raw8(Raw8<float>& r, const float* row, int v, int32_t t, int32_t tpr, int32_t cols) {
    if (VEC) {
        const int32_t c = row_col<true>(v, 0, t, tpr);
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (c < cols) {
            x = reinterpret_cast<const uint4*>(row + c)[0];
            y = reinterpret_cast<const uint4*>(row + c)[1];
        }
        r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
        r.w[4] = y.x, r.w[5] = y.y, r.w[6] = y.z, r.w[7] = y.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int32_t c = row_col<false>(v, j, t, tpr);
            r.w[j] = c < cols ? __float_as_uint(row[c]) : 0u;
        }
    }
}

__device__ __forceinline__ float raw_at(const Raw8<__nv_bfloat16>& r, int j) {
    return __uint_as_float(j % 2 ? r.w[j / 2] & 0xFFFF0000u : r.w[j / 2] << 16);
}
__device__ __forceinline__ float raw_at(const Raw8<float>& r, int j) { return __uint_as_float(r.w[j]); }

template <typename T, bool VEC>
__device__ __forceinline__ void load_row8(float (&x)[8], const T* row, int v, int32_t t, int32_t tpr, int32_t cols) {
    Raw8<T> r;
    load_raw8<VEC>(r, row, v, t, tpr, cols);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = raw_at(r, j);
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_row8(T* row, const float (&x)[8], int v, int32_t t, int32_t tpr, int32_t cols) {
    if (VEC) {
        const int32_t c = row_col<true>(v, 0, t, tpr);
        if (c < cols) store8(row + c, x);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int32_t c = row_col<false>(v, j, t, tpr);
            if (c < cols) from_f32(x[j], row + c);
        }
    }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// Sums of N values (at most 4) over groups of `tpr` threads (a multiple of 32 that divides the block).  Every thread of
// the block calls it; `buf` is this call's own until the next __syncthreads.  The order of the sum is fixed.
//
// Four values take 6 shuffles, not 20: after the first step each half of the warp goes on with two of them, after the
// second each quarter with one.  (Shuffles bound the gradients' rows: 4096 columns on 16 warps, three sums and one,
// 50 of them a warp and row one value at a time.)
template <int N>
__device__ __forceinline__ void warp_sums(float (&x)[N], int32_t lane) {
    if (N == 1) {
        x[0] = warp_sum(x[0]);
        return;
    }
    const bool upper = lane & 16, odd = lane & 8;
    const float x2 = N > 2 ? x[N > 2 ? 2 : 0] : 0.f, x3 = N > 3 ? x[N > 3 ? 3 : 0] : 0.f;
    float a = upper ? x2 : x[0], b = upper ? x3 : x[1];
    a += __shfl_xor_sync(0xffffffffu, upper ? x[0] : x2, 16);
    b += __shfl_xor_sync(0xffffffffu, upper ? x[1] : x3, 16);
    float c = odd ? b : a;
    c += __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
#pragma unroll
    for (int d = 4; d > 0; d /= 2) c += __shfl_xor_sync(0xffffffffu, c, d);
    // Value i is in the lanes from 8 i on.
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __shfl_sync(0xffffffffu, c, 8 * i);
}

template <int N>
__device__ __forceinline__ void group_sum(float (&x)[N], float (*buf)[32], int32_t tpr) {
    const int32_t lane = int32_t(threadIdx.x) % 32;
    warp_sums(x, lane);
    if (tpr == 32) return;
    const int32_t warp = int32_t(threadIdx.x) / 32, warps = tpr / 32;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) buf[i][warp] = x[i];
    __syncthreads();
    const int32_t first = warp / warps * warps;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = lane < warps ? buf[i][first + lane] : 0.f;
    warp_sums(x, lane);
}

// Asynchronous copies of a thread's own 16-byte pieces, group by group.
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Vector v of a row into shared memory, where the row lies as it is, and from there.
template <typename T>
__device__ __forceinline__ void copy_row8(uint32_t to, const T* row, int v, int32_t t, int32_t tpr, int32_t cols) {
    const int32_t c = row_col<true>(v, 0, t, tpr);
    if (c >= cols) return;
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i)
        ptx::cp_async_16(to + uint32_t(c) * uint32_t(sizeof(T)) + 16u * i, reinterpret_cast<const uint8_t*>(row + c) + 16 * i, 16);
}
template <typename T>
__device__ __forceinline__ void take_row8(Raw8<T>& r, uint32_t from, int v, int32_t t, int32_t tpr, int32_t cols) {
    const int32_t c = row_col<true>(v, 0, t, tpr);
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (c < cols) x = ptx::ld_shared_v4(from + uint32_t(c) * uint32_t(sizeof(T)) + 16u * i);
        r.w[4 * i] = x.x, r.w[4 * i + 1] = x.y, r.w[4 * i + 2] = x.z, r.w[4 * i + 3] = x.w;
    }
}

}  // namespace gbr
