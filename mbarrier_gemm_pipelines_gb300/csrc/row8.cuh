// row8.cuh -- a row of a matrix held by a group of threads, V times eight
// elements each, as fp32 (the operators that need a whole row at once), and
// sums over the group.
//
// VEC: the thread's eight are neighbours, moved 16 (bf16) or 32 bytes (fp32) at
// a time; rows start on 16 bytes and the columns are a multiple of 8.
// Otherwise they lie `tpr` columns apart, so that a warp touches whole lines at
// any alignment.
#pragma once
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

// Sums of N values over groups of `tpr` threads (a multiple of 32 that divides
// the block).  Every thread of the block calls it; `buf` is this call's own
// [N][32] floats until the next __syncthreads.  The order of the sum is fixed.
template <int N>
__device__ __forceinline__ void group_sum(float (&x)[N], float (*buf)[32], int32_t tpr) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = warp_sum(x[i]);
    if (tpr == 32) return;
    const int32_t warp = int32_t(threadIdx.x) / 32, lane = int32_t(threadIdx.x) % 32, warps = tpr / 32;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) buf[i][warp] = x[i];
    __syncthreads();
    const int32_t first = warp / warps * warps;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = warp_sum(lane < warps ? buf[i][first + lane] : 0.f);
}

}  // namespace gbr
