// operators.h -- host-side interface between the entry points of the
// feed-forward operators (operators.cu) and their kernels.  Not installed.
#pragma once
#include "activation.cuh"
#include "dropout.cuh"
#include "gbr_internal.h"

namespace gbr {

// A row-major matrix: rows x cols elements, rows ld elements apart.
struct Mat {
    const void* p;
    int64_t ld;
    __host__ __device__ void* w() const { return const_cast<void*>(p); }
    __host__ __device__ explicit operator bool() const { return p != nullptr; }
};

// Scratch of one call, from the device's pool in stream order: given back on
// the stream when the object goes.
class Scratch {
public:
    Scratch(const LibCtx& c, cudaStream_t st) : c_(c), st_(st) {}
    ~Scratch() {
        for (int i = 0; i < n_; ++i) cudaFreeAsync(p_[i], st_);
    }
    Scratch(const Scratch&) = delete;
    Scratch& operator=(const Scratch&) = delete;
    int take(size_t bytes, const char* what, void** out);

private:
    const LibCtx& c_;
    cudaStream_t st_;
    void* p_[8] = {};
    int n_ = 0;
};

// A launch with programmatic overlap and an optional cluster along x.
cudaError_t launch_kernel(void* kernel, dim3 grid, int threads, size_t smem, int cluster, void** args,
                          cudaStream_t stream);
// Raises a kernel's dynamic shared-memory limit on a device as far as needed.
int raise_kernel_smem(void* kernel, size_t smem, int dev);

// The launches below count themselves and return a gbr_status.
// ------------------------------------------------------------ dropout_add
struct DropoutAddArgs {
    const void* X;
    const void* R;
    void* Y;
    int64_t ldx, ldr, ldy;
    int32_t rows, cols;
    bool bf16;                     // else fp32
    Dropout drop;
};
cudaError_t launch_dropout_add(const DropoutAddArgs& a, int sm_count, cudaStream_t stream);

// ------------------------------------------------------------ fused linear
// C[m, n] = R[m, n] + drop(act(Z[m, n])), Z = A B + bias.
struct LinearArgs {
    Mat A, B, R, C, Z;             // R and Z optional
    const float* bias;             // optional
    int32_t M, N, K;
    int act;
    Dropout drop;
};
int launch_linear(const LinearArgs& a, const LibCtx& c, cudaStream_t stream);

// Which kernel a bf16 product [rows, contraction] x [contraction, cols] runs on:
// CTA pairs, or single tiles of bt rows, `split` CTAs each, rings within `budget` bytes.
struct LinearPlan {
    bool pair;
    int32_t bt, split;
    int64_t budget;
};
LinearPlan plan_linear(int32_t rows, int32_t cols, int32_t contraction, int sms);

// dZ = drop(dC) * act'(Z) (bf16) and dbias = sum over rows of dZ (fp32).
struct LinearGradArgs {
    Mat dC, Z, dZ;                 // Z: unless act is none; dZ optional (not wanted)
    float* dbias;                  // optional
    int32_t M, N;
    int act;
    Dropout drop;
};
int launch_linear_dz(const LinearGradArgs& a, const LibCtx& c, cudaStream_t stream);

// The gradients' products: dA[M, K] = dZ[M, N] B[K, N]^T and
// dB[K, N] = A[M, K]^T dZ[M, N].
// Either may be wanted alone (the other's p NULL).
int launch_linear_grads(Mat A, Mat B, Mat dZ, Mat dA, Mat dB, int32_t M, int32_t N, int32_t K, const LibCtx& c,
                        cudaStream_t stream);

// ------------------------------------------------------------ expert layer
constexpr int kMoeMaxTokens = 64, kMoeMaxExperts = 256, kMoeMaxTopK = 8;
struct MoeArgs {
    const void* X;                 // [T, D] bf16
    const float* Wr;               // [D, E]
    const void* W1;                // [E, D, F or 2F] bf16
    const float* b1;               // [E, F or 2F], optional
    const void* W2;                // [E, F, D] bf16
    const float* b2;               // [E, D], optional
    void* Y;                       // [T, D] bf16
    int64_t* ids;                  // [T, top_k]
    float* weights;                // [T, top_k]
    int32_t T, D, F, E, top_k;
    int act;
    bool gated;
};
size_t moe_scratch_bytes(const MoeArgs& a, const LibCtx& c);
int launch_moe(const MoeArgs& a, void* scratch, const LibCtx& c, cudaStream_t stream);

// ------------------------------------------------------------ residual_norm
// y = norm(X) post;  S = R + scale G y;  H = norm(S) pre.  Rows of G are shared
// by per_gate rows each; gates = rows / per_gate, or 0 without G.
struct ResidualNormArgs {
    Mat X, R, G, S, H;             // R, G, S and H optional
    const float *post, *pre;       // optional; pre with H
    int32_t rows, cols, gates, per_gate;
    float scale, eps;
    bool bf16;                     // else fp32
};
int launch_residual_norm(const ResidualNormArgs& a, const LibCtx& c, cudaStream_t stream);

struct ResidualNormGradArgs {
    Mat dS, dH, X, S, G;           // dS optional; dH and S with pre; X unless there is neither post nor G
    const float *post, *pre;
    Mat dX, dR, dG;                // each optional (not wanted)
    float *dpost, *dpre;           // the same
    int32_t rows, cols, gates, per_gate;
    float scale, eps;
    bool bf16;
};
int launch_residual_norm_grad(const ResidualNormGradArgs& a, const LibCtx& c, cudaStream_t stream);

// ------------------------------------------------------------ rows by expert
constexpr int kSortMaxExperts = 1024;
struct MoeSortArgs {
    const int64_t* ids;            // [n]
    int32_t *positions, *offsets;  // [n], [experts + 1]
    int32_t n, experts;
};
int launch_moe_sort(const MoeSortArgs& a, const LibCtx& c, cudaStream_t stream);

// Rows of tokens [T, D] and of choices [T * k, D]; positions say where a choice's row is.
struct MoeRowsArgs {
    Mat X, Ys, R, Y;               // dispatch: X -> Ys; combine: Ys (and R) -> Y
    const int32_t *positions, *offsets;
    const float* weights;          // optional
    int32_t T, k, D, experts;
    bool bf16;
};
int launch_moe_dispatch(const MoeRowsArgs& a, const LibCtx& c, cudaStream_t stream);
int launch_moe_combine(const MoeRowsArgs& a, int64_t rows, const LibCtx& c, cudaStream_t stream);

struct MoeCombineGradArgs {
    Mat dY, Ys, dYs;               // Ys with dweights; dYs optional
    const int32_t *positions, *offsets;
    const float* weights;
    float* dweights;               // optional
    int32_t T, k, D, experts;
    bool bf16;
};
int launch_moe_combine_grad(const MoeCombineGradArgs& a, const LibCtx& c, cudaStream_t stream);

// ------------------------------------------------------------ 4-bit products
// Blocks of 32 along the columns: data [rows, 16 * blocks] bytes, scales in
// tiles of 128 rows x 4 blocks, 512 bytes each.
struct Mxfp4Quantize {
    Mat X;                         // [rows, cols], or [cols, rows] where transposed
    uint8_t *data, *scales;
    int32_t rows, cols;
    bool bf16, transposed;
};
int launch_mxfp4_quantize(const Mxfp4Quantize& a, const LibCtx& c, cudaStream_t stream);
struct Mxfp4Dequantize {
    const uint8_t *data, *scales;
    Mat X;
    int32_t rows, cols;
    bool bf16;
};
int launch_mxfp4_dequantize(const Mxfp4Dequantize& a, const LibCtx& c, cudaStream_t stream);

// C = R + act(A B^T + bias).
struct Mxfp4Args {
    const uint8_t *A, *As, *B, *Bs;
    const float* bias;             // optional
    Mat R, C;                      // R optional
    int32_t M, N, blocks;
    int act;
};
int launch_mxfp4(const Mxfp4Args& a, const LibCtx& c, cudaStream_t stream);

}  // namespace gbr
