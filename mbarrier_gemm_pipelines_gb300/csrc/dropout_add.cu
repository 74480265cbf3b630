// dropout_add.cu -- Y = residual + keep * X / (1 - p), the mask recomputed from
// its position (dropout.cuh).  Bound by memory: X (and residual) are read once
// and Y is written once; the generator costs about ten instructions an element.
//
// Threads stand on a fixed group of 8 columns and walk down the rows, four at a
// time, so that no index needs a division and four rows' loads are under way
// together.  Two kernels, by a rule on alignment:
//   * all rows start on 16 bytes: a thread loads, decides and stores its 8
//     columns, 16 bytes at a time;
//   * otherwise a warp takes 256 columns of a row and each lane every 32nd of
//     them (whole 64- or 128-byte lines at any alignment); the 8 decisions of a
//     group are made once, by one lane, and handed round with shuffles.
#include "gbr_internal.h"
#include "operators.h"
#include "vec8.cuh"

#include <algorithm>

namespace gbr {
namespace {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float* y) { *y = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16* y) { *y = __float2bfloat16_rn(x); }

constexpr int kThreads = 256, kRows = 4;

template <typename T>
struct Args {
    const T *X, *R;
    T* Y;
    int64_t ldx, ldr, ldy;
    int32_t rows, cols;
    Dropout d;
};

// 1 << shift threads along the columns, the others along the rows.
template <typename T, bool HAS_R>
__global__ void __launch_bounds__(kThreads) dropout_add_vec_kernel(const Args<T> a, int shift) {
    ptx::griddep_wait();
    const int32_t g = int32_t((blockIdx.x << shift) + (threadIdx.x & ((1u << shift) - 1u)));
    const int32_t c = g * 8, per = kThreads >> shift, step = int32_t(gridDim.y) * per;
    if (c >= a.cols) return;
    const bool whole = a.cols - c >= 8;
    for (int64_t r0 = int64_t(blockIdx.y) * per + (threadIdx.x >> shift); r0 < a.rows; r0 += int64_t(step) * kRows) {
        float x[kRows][8], r[kRows][8];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t row = r0 + int64_t(i) * step;
            if (row >= a.rows) continue;
            if (whole) {
                load8(a.X + row * a.ldx + c, x[i]);
                if (HAS_R) load8(a.R + row * a.ldr + c, r[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < a.cols) {
                        x[i][j] = to_f32(a.X[row * a.ldx + c + j]);
                        if (HAS_R) r[i][j] = to_f32(a.R[row * a.ldr + c + j]);
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t row = r0 + int64_t(i) * step;
            if (row >= a.rows) continue;
            if (a.d.threshold != 0) {
                const uint4 bits = dropout_bits(a.d, uint32_t(row), uint32_t(g));
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = dropout_keep(a.d, bits, j) ? x[i][j] * a.d.scale : 0.f;
            }
            if (HAS_R)
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] += r[i][j];
            T* y = a.Y + row * a.ldy + c;
            if (whole) {
                store8(y, x[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < a.cols) from_f32(x[i][j], y + j);
            }
        }
    }
}

// A warp a row and 256 columns; blockIdx.x: the columns, 8 rows of warps a CTA.
template <typename T, bool HAS_R>
__global__ void __launch_bounds__(kThreads) dropout_add_any_kernel(const Args<T> a) {
    ptx::griddep_wait();
    const int32_t lane = int32_t(threadIdx.x) % 32, c0 = int32_t(blockIdx.x) * 256;
    for (int64_t row = int64_t(blockIdx.y) * 8 + threadIdx.x / 32; row < a.rows; row += int64_t(gridDim.y) * 8) {
        const T *X = a.X + row * a.ldx + c0 + lane, *R = HAS_R ? a.R + row * a.ldr + c0 + lane : nullptr;
        T* Y = a.Y + row * a.ldy + c0 + lane;
        const int32_t left = a.cols - c0 - lane;        // columns from this lane's first on
        float x[8], r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (32 * j < left) {
                x[j] = to_f32(X[32 * j]);
                if (HAS_R) r[j] = to_f32(R[32 * j]);
            }
        uint32_t keep = 0xFFu;                          // of columns c0 + 8 lane ...
        if (a.d.threshold != 0) {
            const uint4 bits = dropout_bits(a.d, uint32_t(row), uint32_t(c0 / 8 + lane));
            keep = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) keep |= uint32_t(dropout_keep(a.d, bits, j)) << j;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t k = __shfl_sync(0xffffffffu, keep, 4 * j + lane / 8);
            if (32 * j < left) {
                float y = (k >> (lane % 8)) & 1u ? x[j] * a.d.scale : 0.f;
                if (HAS_R) y += r[j];
                from_f32(y, Y + 32 * j);
            }
        }
    }
}

template <typename T>
cudaError_t launch(const DropoutAddArgs& s, int sm_count, cudaStream_t stream) {
    Args<T> a = {static_cast<const T*>(s.X), static_cast<const T*>(s.R), static_cast<T*>(s.Y), s.ldx, s.ldr, s.ldy,
                 s.rows, s.cols, s.drop};
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    cfg.numAttrs = programmatic_launch_attr(attr);
    cfg.attrs = attr;
    constexpr int64_t kAlign = 16 / sizeof(T);
    auto ready = [&](const void* p, int64_t ld) {
        return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld % kAlign == 0 || s.rows == 1));
    };
    // Enough CTAs for 16 an SM, as long as there are rows for them.
    const int64_t most = int64_t(sm_count) * 16;
    if (ready(s.X, s.ldx) && ready(s.R, s.ldr) && ready(s.Y, s.ldy)) {
        const int64_t groups = (int64_t(s.cols) + 7) / 8;
        int shift = 0;
        while (shift < 8 && (int64_t(1) << shift) < groups) ++shift;
        const int64_t gx = (groups + (int64_t(1) << shift) - 1) >> shift, per = kThreads >> shift;
        const int64_t gy = std::min<int64_t>((s.rows + per - 1) / per, std::max<int64_t>(1, most / gx));
        cfg.gridDim = dim3(unsigned(gx), unsigned(std::min<int64_t>(gy, 65535)));
        return s.R != nullptr ? cudaLaunchKernelEx(&cfg, dropout_add_vec_kernel<T, true>, a, shift)
                              : cudaLaunchKernelEx(&cfg, dropout_add_vec_kernel<T, false>, a, shift);
    }
    const int64_t gx = (int64_t(s.cols) + 255) / 256;
    const int64_t gy = std::min<int64_t>((s.rows + 7) / 8, std::max<int64_t>(1, most / gx));
    cfg.gridDim = dim3(unsigned(gx), unsigned(std::min<int64_t>(gy, 65535)));
    return s.R != nullptr ? cudaLaunchKernelEx(&cfg, dropout_add_any_kernel<T, true>, a)
                          : cudaLaunchKernelEx(&cfg, dropout_add_any_kernel<T, false>, a);
}

}  // namespace

cudaError_t launch_dropout_add(const DropoutAddArgs& a, int sm_count, cudaStream_t stream) {
    return a.bf16 ? launch<__nv_bfloat16>(a, sm_count, stream) : launch<float>(a, sm_count, stream);
}

}  // namespace gbr
