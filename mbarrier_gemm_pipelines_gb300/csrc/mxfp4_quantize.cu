// mxfp4_quantize.cu -- matrices to blocks of 4-bit values with a scale each
// (mxfp4.cuh) and back.  Bound by memory: the matrix is read once and 17 bytes
// are written for 32 values.
//   rows kept: a thread takes 16 neighbouring values, two threads a block; four
//     blocks' scales are one 32-bit store.
//   transposed (weights stored [K, N], wanted [N, K]): a thread takes 4 blocks of
//     its own column, neighbouring threads neighbouring columns.
#include "gbr.h"
#include "mxfp4.cuh"
#include "operators.h"
#include "row8.cuh"

#include <algorithm>
#include <cstdint>

namespace gbr {
namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kThreads = 256;

template <typename T>
struct QuantArgs {
    const T* X;
    int64_t ldx;
    uint8_t *data, *scales;
    int32_t rows, cols, blocks, block_tiles;
};

// The largest bit pattern of eight absolute values, and the values as fp32 pairs.
__device__ __forceinline__ uint32_t top8(const Raw8<__nv_bfloat16>& r) {
    uint32_t m = __vmaxu2(r.w[0] & 0x7FFF7FFFu, r.w[1] & 0x7FFF7FFFu);
    m = __vmaxu2(m, __vmaxu2(r.w[2] & 0x7FFF7FFFu, r.w[3] & 0x7FFF7FFFu));
    return max(m << 16, m & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t top8(const Raw8<float>& r) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, r.w[j] & 0x7FFFFFFFu);
    return m;
}

// A warp a row and 512 columns, 16 neighbouring values a lane, two lanes a block; rows up to the next multiple of 128,
// for the scales' padding.  4096 x 4096 bf16, bound by instructions as much as by memory: 8 values a lane, value by
// value and one row at a time 12.8 us, in pairs and two rows 10.5, 16 values 8.4.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) mxfp4_quantize_kernel(const QuantArgs<T> a) {
    ptx::griddep_wait();
    // A few rows: the product behind may set itself up meanwhile.  (More: its CTAs would take this kernel's places.)
    if (gridDim.x * gridDim.y <= 512) ptx::griddep_launch_dependents();
    const int32_t lane = int32_t(threadIdx.x) % 32, b = int32_t(blockIdx.x) * 16 + lane / 2, c = b * kMxBlock + lane % 2 * 16;
    const int64_t padded = (int64_t(a.rows) + 127) / 128 * 128, step = int64_t(gridDim.y) * (kThreads / 32);
    for (int64_t row = int64_t(blockIdx.y) * (kThreads / 32) + threadIdx.x / 32; row < padded; row += step) {
        Raw8<T> r[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            load_raw8<VEC ? kVec : kShifted>(r[h], a.X + row * a.ldx, 0, c / 8 + h, 1, row < a.rows ? a.cols : 0);
        uint32_t top = max(top8(r[0]), top8(r[1]));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        const uint32_t byte = mx_scale_byte(top);
        const F2 inv = f2(mx_inverse(byte));
        uint32_t code[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) split2(mul2(raw_pair(r[h], i), inv), y[2 * i], y[2 * i + 1]);
            code[h] = byte == 255u ? 0u : mx_pack8(y);          // of a NaN block any
        }
        if (row < a.rows && b < a.blocks)
            *reinterpret_cast<uint2*>(a.data + row * int64_t(a.blocks) * 16 + c / 2) = make_uint2(code[0], code[1]);
        uint32_t four = byte << (lane / 2 % 4 * 8);
        four |= __shfl_xor_sync(0xffffffffu, four, 2);
        four |= __shfl_xor_sync(0xffffffffu, four, 4);
        if (lane % 8 == 0 && b / 4 < a.block_tiles)
            *reinterpret_cast<uint32_t*>(a.scales + mx_scale_offset(row, b, a.block_tiles)) = four;
    }
}

// X [cols, rows]; a thread a row of the result and the 4 blocks of a tile.
template <typename T>
__global__ void __launch_bounds__(kThreads) mxfp4_quantize_columns_kernel(const QuantArgs<T> a) {
    ptx::griddep_wait();
    const int64_t row = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (row >= (int64_t(a.rows) + 127) / 128 * 128) return;
    for (int32_t tile = int32_t(blockIdx.y); tile < a.block_tiles; tile += int32_t(gridDim.y)) {
        uint32_t four = 0;
        for (int32_t i = 0; i < 4 && row < a.rows; ++i) {
            const int32_t b = tile * 4 + i;
            if (b >= a.blocks) break;
            float x[4][8];
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const int32_t c = b * kMxBlock + j;
                x[j / 8][j % 8] = c < a.cols ? to_f32(a.X[c * a.ldx + row]) : 0.f;
                top = max(top, __float_as_uint(x[j / 8][j % 8]) & 0x7FFFFFFFu);
            }
            const uint32_t byte = mx_scale_byte(top);
            const float inv = mx_inverse(byte);
            uint32_t code[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[j][e] = byte == 255u ? 0.f : x[j][e] * inv;
                code[j] = mx_pack8(x[j]);
            }
            *reinterpret_cast<uint4*>(a.data + (row * a.blocks + b) * 16) = make_uint4(code[0], code[1], code[2], code[3]);
            four |= byte << (8 * i);
        }
        *reinterpret_cast<uint32_t*>(a.scales + mx_scale_offset(row, tile * 4, a.block_tiles)) = four;
    }
}

template <typename T>
struct DequantArgs {
    const uint8_t *data, *scales;
    T* X;
    int64_t ldx;
    int32_t rows, cols, blocks, block_tiles;
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) mxfp4_dequantize_kernel(const DequantArgs<T> a) {
    ptx::griddep_wait();
    const int32_t c = int32_t(blockIdx.x) * 256 + int32_t(threadIdx.x) % 32 * 8, left = a.cols - c;
    if (left <= 0) return;
    for (int64_t row = int64_t(blockIdx.y) * (kThreads / 32) + threadIdx.x / 32; row < a.rows;
         row += int64_t(gridDim.y) * (kThreads / 32)) {
        const uint32_t code = *reinterpret_cast<const uint32_t*>(a.data + row * int64_t(a.blocks) * 16 + c / 2);
        const float scale = mx_scale(a.scales[mx_scale_offset(row, c / kMxBlock, a.block_tiles)]);
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = mx_value(code >> (4 * j) & 15u) * scale;
        T* out = a.X + row * a.ldx + c;
        if (VEC) {
            store8(out, x);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < left) from_f32(x[j], out + j);
        }
    }
}

template <typename T>
bool aligned16(const Mat& m, int64_t rows) {
    return reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && (rows <= 1 || m.ld % int64_t(16 / sizeof(T)) == 0);
}

template <typename T>
int quantize(const Mxfp4Quantize& s, const LibCtx& c, cudaStream_t stream) {
    QuantArgs<T> a = {static_cast<const T*>(s.X.p), s.X.ld, s.data, s.scales, s.rows, s.cols, int32_t(cdiv(s.cols, 32)),
                      int32_t(cdiv(s.cols, 128))};
    void* args[] = {&a};
    const int64_t padded = cdiv(s.rows, 128) * 128;
    cudaError_t e;
    if (s.transposed) {
        e = launch_kernel(reinterpret_cast<void*>(&mxfp4_quantize_columns_kernel<T>),
                          dim3(unsigned(cdiv(padded, kThreads)), unsigned(std::min<int64_t>(a.block_tiles, 65535))),
                          kThreads, 0, 1, args, stream);
    } else {
        const bool vec = s.cols % 8 == 0 && aligned16<T>(s.X, s.rows);
        const int64_t gx = cdiv(s.cols, 512), most = std::max<int64_t>(1, int64_t(c.sm_count) * 12 / gx);
        e = launch_kernel(vec ? reinterpret_cast<void*>(&mxfp4_quantize_kernel<T, true>)
                              : reinterpret_cast<void*>(&mxfp4_quantize_kernel<T, false>),
                          dim3(unsigned(gx), unsigned(std::min<int64_t>(padded / (kThreads / 32), most))), kThreads, 0, 1,
                          args, stream);
    }
    if (e != cudaSuccess) return report_cuda(e, "launching quantize_mxfp4");
    count_launch();
    return GBR_OK;
}

template <typename T>
int dequantize(const Mxfp4Dequantize& s, const LibCtx& c, cudaStream_t stream) {
    DequantArgs<T> a = {s.data, s.scales, static_cast<T*>(s.X.w()), s.X.ld, s.rows, s.cols, int32_t(cdiv(s.cols, 32)),
                        int32_t(cdiv(s.cols, 128))};
    void* args[] = {&a};
    const bool vec = s.cols % 8 == 0 && aligned16<T>(s.X, s.rows);
    const int64_t gx = cdiv(s.cols, 256), most = std::max<int64_t>(1, int64_t(c.sm_count) * 32 / gx);
    const cudaError_t e = launch_kernel(vec ? reinterpret_cast<void*>(&mxfp4_dequantize_kernel<T, true>)
                                            : reinterpret_cast<void*>(&mxfp4_dequantize_kernel<T, false>),
                                        dim3(unsigned(gx), unsigned(std::min<int64_t>(cdiv(s.rows, kThreads / 32), most))),
                                        kThreads, 0, 1, args, stream);
    if (e != cudaSuccess) return report_cuda(e, "launching dequantize_mxfp4");
    count_launch();
    return GBR_OK;
}

}  // namespace

int launch_mxfp4_quantize(const Mxfp4Quantize& a, const LibCtx& c, cudaStream_t stream) {
    return a.bf16 ? quantize<__nv_bfloat16>(a, c, stream) : quantize<float>(a, c, stream);
}
int launch_mxfp4_dequantize(const Mxfp4Dequantize& a, const LibCtx& c, cudaStream_t stream) {
    return a.bf16 ? dequantize<__nv_bfloat16>(a, c, stream) : dequantize<float>(a, c, stream);
}

}  // namespace gbr
