// dropout_add.cu -- Y = residual + keep * X / (1 - p), the mask recomputed from
// its position (dropout.cuh).  Bound by memory: X (and residual) are read once
// and Y is written once; the generator costs about ten instructions an element.
//
// Threads stand on a fixed group of 8 columns and walk down the rows, two at a
// time, so that no index needs a division and two rows' loads are under way
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

// Two rows a turn; registers for four CTAs an SM (bf16) or three (fp32), by
// measurement: bf16 with residual, 16384 x 4096, 2 rows, 2 / 3 / 4 CTAs: 71 /
// 63 / 59 us, 1 row, 6 CTAs 60, 4 rows, 3 CTAs 64; fp32, 2 rows, 3 / 4 CTAs: 116 / 118.
constexpr int kThreads = 256, kRows = 2;
template <typename T>
constexpr int kMinCtas = sizeof(T) == 2 ? 4 : 3;

template <typename T>
struct Args {
    const T *X, *R;
    T* Y;
    int64_t ldx, ldr, ldy;
    int32_t rows, cols;
    Dropout d;
};

// Eight elements as they are loaded.
template <typename T>
struct Raw8 {
    uint4 v[sizeof(T) * 8 / 16];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T* p) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < int(sizeof(T) * 8 / 16); ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
    return r;
}
__device__ __forceinline__ void unpack(const Raw8<__nv_bfloat16>& r, float (&x)[8]) { unpack8(r.v[0], x); }
__device__ __forceinline__ void unpack(const Raw8<float>& r, float (&x)[8]) {
    const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[j]);
}

template <bool HAS_R>
__device__ __forceinline__ void drop_add8(const Dropout& d, uint32_t row, uint32_t g, float (&x)[8],
                                          const float (&r)[8]) {
    if (d.threshold != 0) {
        const uint4 bits = dropout_bits(d, row, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = dropout_keep(d, bits, j) ? x[j] * d.scale : 0.f;
    }
    if (HAS_R)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] += r[j];
}

// 1 << shift threads along the columns, the others along the rows.
template <typename T, bool HAS_R>
__global__ void __launch_bounds__(kThreads, kMinCtas<T>) dropout_add_vec_kernel(const Args<T> a, int shift) {
    ptx::griddep_wait();
    const int32_t g = int32_t((blockIdx.x << shift) + (threadIdx.x & ((1u << shift) - 1u)));
    const int32_t c = g * 8, per = kThreads >> shift, left = a.cols - c;
    const int64_t step = int64_t(gridDim.y) * per;
    if (left <= 0) return;
    int64_t row = int64_t(blockIdx.y) * per + (threadIdx.x >> shift);
    const T *X = a.X + row * a.ldx + c, *R = HAS_R ? a.R + row * a.ldr + c : nullptr;
    T* Y = a.Y + row * a.ldy + c;
    const int64_t sx = step * a.ldx, sr = step * a.ldr, sy = step * a.ldy;
    float x[8], r[8] = {};
    if (left >= 8) {
        for (; row + (kRows - 1) * step < a.rows; row += kRows * step) {
            Raw8<T> vx[kRows], vr[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                vx[i] = load_raw(X + i * sx);
                if (HAS_R) vr[i] = load_raw(R + i * sr);
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                unpack(vx[i], x);
                if (HAS_R) unpack(vr[i], r);
                drop_add8<HAS_R>(a.d, uint32_t(row + i * step), uint32_t(g), x, r);
                store8(Y + i * sy, x);
            }
            X += kRows * sx, Y += kRows * sy;
            if (HAS_R) R += kRows * sr;
        }
        for (; row < a.rows; row += step) {
            unpack(load_raw(X), x);
            if (HAS_R) unpack(load_raw(R), r);
            drop_add8<HAS_R>(a.d, uint32_t(row), uint32_t(g), x, r);
            store8(Y, x);
            X += sx, Y += sy;
            if (HAS_R) R += sr;
        }
        return;
    }
    for (; row < a.rows; row += step) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) {
                x[j] = to_f32(X[j]);
                if (HAS_R) r[j] = to_f32(R[j]);
            }
        drop_add8<HAS_R>(a.d, uint32_t(row), uint32_t(g), x, r);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) from_f32(x[j], Y + j);
        X += sx, Y += sy;
        if (HAS_R) R += sr;
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
