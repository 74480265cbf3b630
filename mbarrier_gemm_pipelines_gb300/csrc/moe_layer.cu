// moe_layer.cu -- a whole mixture-of-experts layer for a few tokens, as plain
// kernels: the router (one CTA per token), the experts' hidden values (one
// thread per token, choice and hidden column), the outputs (one thread per
// token and output column, choices added in the order they were picked).
#include "operators.h"

#include <cuda_bf16.h>

namespace gbr {
namespace {

using bf16 = __nv_bfloat16;

// Softmax over the top_k largest logits of each token; ties go to the lowest
// expert.  Order: descending.  A NaN logit ranks last.
__global__ void __launch_bounds__(256) moe_router_kernel(const MoeArgs a) {
    __shared__ float logit[kMoeMaxExperts];
    ptx::griddep_wait();
    const int t = int(blockIdx.x), lane = int(threadIdx.x) % 32;
    const bf16* x = static_cast<const bf16*>(a.X) + int64_t(t) * a.D;
    for (int e = int(threadIdx.x) / 32; e < a.E; e += 8) {
        float v = 0.f;
        for (int d = lane; d < a.D; d += 32)
            v = fmaf(__bfloat162float(x[d]), a.Wr[int64_t(d) * a.E + e], v);
        for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) logit[e] = v;
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    int id[kMoeMaxTopK];
    float w[kMoeMaxTopK], sum = 0.f;
    for (int k = 0; k < a.top_k; ++k) {
        int best = -1;
        for (int e = 0; e < a.E; ++e) {
            bool taken = false;
            for (int j = 0; j < k; ++j) taken |= id[j] == e;
            if (taken) continue;
            if (best < 0 || logit[e] > logit[best] || (isnan(logit[best]) && !isnan(logit[e]))) best = e;
        }
        id[k] = best;
        w[k] = expf(logit[best] - logit[id[0]]);
        sum += w[k];
    }
    for (int k = 0; k < a.top_k; ++k) {
        a.ids[t * a.top_k + k] = id[k];
        a.weights[t * a.top_k + k] = w[k] / sum;
    }
}

__global__ void __launch_bounds__(128) moe_hidden_kernel(const MoeArgs a, float* h) {
    ptx::griddep_wait();
    const int pair = int(blockIdx.y), t = pair / a.top_k;
    const int f = int(blockIdx.x) * 128 + int(threadIdx.x);
    if (f >= a.F) return;
    const int e = int(a.ids[pair]);
    const int64_t F1 = a.gated ? 2 * int64_t(a.F) : a.F;
    const bf16* x = static_cast<const bf16*>(a.X) + int64_t(t) * a.D;
    const bf16* w = static_cast<const bf16*>(a.W1) + int64_t(e) * a.D * F1;
    float z = 0.f, u = 0.f;
    for (int d = 0; d < a.D; ++d) {
        const float xv = __bfloat162float(x[d]);
        z = fmaf(xv, __bfloat162float(w[d * F1 + f]), z);
        if (a.gated) u = fmaf(xv, __bfloat162float(w[d * F1 + a.F + f]), u);
    }
    if (a.b1 != nullptr) {
        z += a.b1[e * F1 + f];
        if (a.gated) u += a.b1[e * F1 + a.F + f];
    }
    z = act_value(a.act, z);
    h[int64_t(pair) * a.F + f] = a.gated ? z * u : z;
}

__global__ void __launch_bounds__(128) moe_output_kernel(const MoeArgs a, const float* h) {
    ptx::griddep_wait();
    const int t = int(blockIdx.y), d = int(blockIdx.x) * 128 + int(threadIdx.x);
    if (d >= a.D) return;
    float y = 0.f;
    for (int k = 0; k < a.top_k; ++k) {
        const int pair = t * a.top_k + k, e = int(a.ids[pair]);
        const bf16* w = static_cast<const bf16*>(a.W2) + int64_t(e) * a.F * a.D;
        float v = a.b2 != nullptr ? a.b2[int64_t(e) * a.D + d] : 0.f;
        for (int f = 0; f < a.F; ++f)
            v = fmaf(h[int64_t(pair) * a.F + f], __bfloat162float(w[int64_t(f) * a.D + d]), v);
        y = fmaf(a.weights[pair], v, y);
    }
    static_cast<bf16*>(a.Y)[int64_t(t) * a.D + d] = __float2bfloat16_rn(y);
}

}  // namespace

size_t moe_scratch_bytes(const MoeArgs& a, const LibCtx&) {
    return size_t(a.T) * size_t(a.top_k) * size_t(a.F) * sizeof(float);
}

cudaError_t launch_moe(const MoeArgs& a, void* scratch, const LibCtx&, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.numAttrs = programmatic_launch_attr(attr);
    cfg.attrs = attr;
    cfg.stream = stream;
    cfg.gridDim = dim3(a.T);
    cfg.blockDim = dim3(256);
    cudaError_t e = cudaLaunchKernelEx(&cfg, moe_router_kernel, a);
    if (e != cudaSuccess) return e;
    float* h = static_cast<float*>(scratch);
    cfg.blockDim = dim3(128);
    cfg.gridDim = dim3((a.F + 127) / 128, a.T * a.top_k);
    if ((e = cudaLaunchKernelEx(&cfg, moe_hidden_kernel, a, h)) != cudaSuccess) return e;
    cfg.gridDim = dim3((a.D + 127) / 128, a.T);
    return cudaLaunchKernelEx(&cfg, moe_output_kernel, a, static_cast<const float*>(h));
}

}  // namespace gbr
