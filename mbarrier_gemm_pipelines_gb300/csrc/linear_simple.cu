// linear_simple.cu -- the fused linear layer and its gradients, as plain tiled
// kernels on CUDA cores: one thread computes 4 x 4 outputs of a 64 x 64 tile,
// operands staged through shared memory in steps of 16.
#include "operators.h"

#include <cuda_bf16.h>

namespace gbr {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kTile = 64, kStep = 16, kThreads = 256;

// C[i, j] = epilogue(sum_k a(i, k) b(k, j)); operand strides in elements.
struct SimpleArgs {
    const bf16 *a, *b;
    int64_t a_i, a_k, b_k, b_j;
    int32_t I, J, K;
    const float* bias;
    const bf16* R;
    bf16 *C, *Z;
    int64_t ldr, ldc, ldz;
    int act;
    Dropout drop;
};

__global__ void __launch_bounds__(kThreads) simple_gemm_kernel(const SimpleArgs s) {
    __shared__ float as[kStep][kTile + 1], bs[kStep][kTile + 1];
    ptx::griddep_wait();
    const int i0 = int(blockIdx.y) * kTile, j0 = int(blockIdx.x) * kTile;
    const int ti = int(threadIdx.x) / 16 * 4, tj = int(threadIdx.x) % 16 * 4;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < s.K; k0 += kStep) {
        for (int e = int(threadIdx.x); e < kTile * kStep; e += kThreads) {
            const int k = e % kStep, r = e / kStep;
            const bool kin = k0 + k < s.K;
            as[k][r] = kin && i0 + r < s.I
                           ? __bfloat162float(s.a[(i0 + r) * s.a_i + (k0 + k) * s.a_k]) : 0.f;
            bs[k][r] = kin && j0 + r < s.J
                           ? __bfloat162float(s.b[(k0 + k) * s.b_k + (j0 + r) * s.b_j]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStep; ++k)
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) acc[x][y] = fmaf(as[k][ti + x], bs[k][tj + y], acc[x][y]);
        __syncthreads();
    }
    for (int x = 0; x < 4; ++x)
        for (int y = 0; y < 4; ++y) {
            const int64_t i = i0 + ti + x, j = j0 + tj + y;
            if (i >= s.I || j >= s.J) continue;
            const float z = acc[x][y] + (s.bias != nullptr ? s.bias[j] : 0.f);
            if (s.Z != nullptr) s.Z[i * s.ldz + j] = __float2bfloat16_rn(z);
            float c = act_value(s.act, z);
            if (s.drop.threshold != 0) {
                const uint4 bits = dropout_bits(s.drop, uint32_t(i), uint32_t(j / 8));
                c = dropout_keep(s.drop, bits, int(j % 8)) ? c * s.drop.scale : 0.f;
            }
            if (s.R != nullptr) c += __bfloat162float(s.R[i * s.ldr + j]);
            s.C[i * s.ldc + j] = __float2bfloat16_rn(c);
        }
}

cudaError_t launch_simple(const SimpleArgs& s, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((s.J + kTile - 1) / kTile, (s.I + kTile - 1) / kTile);
    if (cfg.gridDim.y > 65535) return cudaErrorInvalidConfiguration;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    cfg.numAttrs = programmatic_launch_attr(attr);
    cfg.attrs = attr;
    return cudaLaunchKernelEx(&cfg, simple_gemm_kernel, s);
}

// One CTA per 32 columns: 8 rows of threads walk down the rows.
template <int ACT>
__global__ void __launch_bounds__(256) simple_dz_kernel(const LinearGradArgs a) {
    __shared__ float part[8][32];
    ptx::griddep_wait();
    const int n = int(blockIdx.x) * 32 + int(threadIdx.x) % 32;
    float sum = 0.f;
    for (int m = int(threadIdx.x) / 32; n < a.N && m < a.M; m += 8) {
        float d = __bfloat162float(static_cast<const bf16*>(a.dC.p)[m * a.dC.ld + n]);
        bool keep = true;
        if (a.drop.threshold != 0) {
            const uint4 bits = dropout_bits(a.drop, uint32_t(m), uint32_t(n / 8));
            keep = dropout_keep(a.drop, bits, n % 8);
            d *= a.drop.scale;
        }
        if (ACT != kActNone)
            d *= act_slope<ACT>(__bfloat162float(static_cast<const bf16*>(a.Z.p)[m * a.Z.ld + n]));
        if (!keep) d = 0.f;
        if (a.dZ) static_cast<bf16*>(a.dZ.w())[m * a.dZ.ld + n] = __float2bfloat16_rn(d);
        sum += d;
    }
    part[threadIdx.x / 32][threadIdx.x % 32] = sum;
    __syncthreads();
    if (threadIdx.x < 32 && n < a.N && a.dbias != nullptr) {
        float t = 0.f;
        for (int r = 0; r < 8; ++r) t += part[r][threadIdx.x];
        a.dbias[n] = t;
    }
}

const bf16* cp(const Mat& m) { return static_cast<const bf16*>(m.p); }
bf16* wp(const Mat& m) { return static_cast<bf16*>(m.w()); }

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, const LibCtx&, cudaStream_t stream) {
    SimpleArgs s = {};
    s.a = cp(a.A), s.a_i = a.A.ld, s.a_k = 1;
    s.b = cp(a.B), s.b_k = a.B.ld, s.b_j = 1;
    s.I = a.M, s.J = a.N, s.K = a.K;
    s.bias = a.bias;
    s.R = cp(a.R), s.ldr = a.R.ld;
    s.C = wp(a.C), s.ldc = a.C.ld;
    s.Z = wp(a.Z), s.ldz = a.Z.ld;
    s.act = a.act;
    s.drop = a.drop;
    return launch_simple(s, stream);
}

cudaError_t launch_linear_dz(const LinearGradArgs& a, const LibCtx&, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.N + 31) / 32);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    cfg.numAttrs = programmatic_launch_attr(attr);
    cfg.attrs = attr;
    switch (a.act) {
        case kActRelu: return cudaLaunchKernelEx(&cfg, simple_dz_kernel<kActRelu>, a);
        case kActGelu: return cudaLaunchKernelEx(&cfg, simple_dz_kernel<kActGelu>, a);
        case kActGeluTanh: return cudaLaunchKernelEx(&cfg, simple_dz_kernel<kActGeluTanh>, a);
        case kActSilu: return cudaLaunchKernelEx(&cfg, simple_dz_kernel<kActSilu>, a);
        default: return cudaLaunchKernelEx(&cfg, simple_dz_kernel<kActNone>, a);
    }
}

cudaError_t launch_linear_da(Mat dZ, Mat B, Mat dA, int32_t M, int32_t N, int32_t K, const LibCtx&,
                             cudaStream_t stream) {
    SimpleArgs s = {};
    s.a = cp(dZ), s.a_i = dZ.ld, s.a_k = 1;
    s.b = cp(B), s.b_k = 1, s.b_j = B.ld;
    s.I = M, s.J = K, s.K = N;
    s.C = wp(dA), s.ldc = dA.ld;
    return launch_simple(s, stream);
}

cudaError_t launch_linear_db(Mat A, Mat dZ, Mat dB, int32_t M, int32_t N, int32_t K, const LibCtx&,
                             cudaStream_t stream) {
    SimpleArgs s = {};
    s.a = cp(A), s.a_i = 1, s.a_k = A.ld;
    s.b = cp(dZ), s.b_k = dZ.ld, s.b_j = 1;
    s.I = K, s.J = N, s.K = M;
    s.C = wp(dB), s.ldc = dB.ld;
    return launch_simple(s, stream);
}

}  // namespace gbr
