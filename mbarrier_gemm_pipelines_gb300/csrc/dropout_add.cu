// dropout_add.cu -- Y = residual + keep * X / (1 - p), the mask recomputed from
// its position (dropout.cuh).  Bound by memory: X (and residual) are read once
// and Y written once.
#include "gbr_internal.h"
#include "operators.h"

#include <cuda_bf16.h>

namespace gbr {
namespace {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float* y) { *y = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16* y) { *y = __float2bfloat16_rn(x); }

constexpr int kThreads = 256;

// One thread per group of 8 columns of a row (one generator call each).
template <typename T>
__global__ void __launch_bounds__(kThreads)
    dropout_add_kernel(const T* X, int64_t ldx, const T* R, int64_t ldr, T* Y, int64_t ldy,
                       int32_t rows, int32_t cols, int32_t groups, Dropout d) {
    ptx::griddep_wait();
    const int64_t total = int64_t(rows) * groups;
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += int64_t(gridDim.x) * kThreads) {
        const int32_t row = int32_t(i / groups), g = int32_t(i - int64_t(row) * groups);
        const uint4 bits = dropout_bits(d, uint32_t(row), uint32_t(g));
        for (int j = 0; j < 8 && 8 * g + j < cols; ++j) {
            const int64_t c = int64_t(8) * g + j;
            float y = dropout_keep(d, bits, j) ? to_f32(X[row * ldx + c]) * d.scale : 0.f;
            if (R != nullptr) y += to_f32(R[row * ldr + c]);
            from_f32(y, Y + row * ldy + c);
        }
    }
}

}  // namespace

cudaError_t launch_dropout_add(const DropoutAddArgs& a, int sm_count, cudaStream_t stream) {
    const int32_t groups = (a.cols + 7) / 8;
    const int64_t blocks = (int64_t(a.rows) * groups + kThreads - 1) / kThreads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks < int64_t(sm_count) * 8 ? blocks : int64_t(sm_count) * 8));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    cfg.numAttrs = programmatic_launch_attr(attr);
    cfg.attrs = attr;
    if (a.bf16) {
        using T = __nv_bfloat16;
        return cudaLaunchKernelEx(&cfg, dropout_add_kernel<T>, static_cast<const T*>(a.X), a.ldx,
                                  static_cast<const T*>(a.R), a.ldr, static_cast<T*>(a.Y), a.ldy,
                                  a.rows, a.cols, groups, a.drop);
    }
    return cudaLaunchKernelEx(&cfg, dropout_add_kernel<float>, static_cast<const float*>(a.X), a.ldx,
                              static_cast<const float*>(a.R), a.ldr, static_cast<float*>(a.Y), a.ldy,
                              a.rows, a.cols, groups, a.drop);
}

}  // namespace gbr
