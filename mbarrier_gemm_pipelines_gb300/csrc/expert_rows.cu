// expert_rows.cu -- rows sorted by expert for the experts' products and back to
// their tokens, with the routing weights applied, and the gradient.
//
//   sort      position of choice (t, j) = its place in the stable order by expert; -1 if it has none
//   dispatch  Ys[position(t, j)] = X[t], zero behind the last expert's rows
//   combine   Y[t] = R[t] + sum_j w(t, j) Ys[position(t, j)]
//   gradient  dYs[position(t, j)] = w(t, j) dY[t],  dw(t, j) = <dY[t], Ys[position(t, j)]>
//
// All but the sort are bound by memory: a token's row is read (or written) once
// and its k rows written (or read) once, each 16 bytes a thread where the rows
// are aligned.  Sums are fp32, in the order of the choices.
#include "gbr.h"
#include "operators.h"
#include "row8.cuh"

#include <algorithm>
#include <cstdint>

namespace gbr {
namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ------------------------------------------------------------ sort
// A stable counting sort in one launch: one CTA, or a cluster of 8 that share
// the choices as contiguous runs, each of their warps a contiguous part.  First
// every warp counts its part's experts in a row of shared memory that is its
// own; then the counts become places (over experts, CTAs and warps in order);
// then every warp goes over its part again and hands the places out.  Choices
// of one expert among a warp's 32 are ranked by lane, so the order is that of
// the choices and nothing depends on timing.
constexpr int kSortWarps = 32, kSortThreads = kSortWarps * 32, kSortCluster = 8;

struct SortParams {
    const int64_t* ids;
    int32_t *positions, *offsets;
    int32_t n, experts;
};

__global__ void __launch_bounds__(kSortThreads, 1) moe_sort_kernel(const SortParams p, uint32_t ctas) {
    extern __shared__ int32_t sm[];
    int32_t* count = sm;                                // [warps][experts]
    int32_t* total = count + kSortWarps * p.experts;    // [experts] of this CTA, read by the peers
    int32_t* start = total + p.experts;                 // [experts] first place of this CTA's choices
    int32_t* sums = start + p.experts;                  // [32]
    ptx::griddep_wait();
    const uint32_t rank = ctas > 1 ? ptx::cluster_ctarank() : 0u;
    const int32_t warp = int32_t(threadIdx.x) / 32, lane = int32_t(threadIdx.x) % 32, E = p.experts;
    for (int32_t i = int32_t(threadIdx.x); i < kSortWarps * E; i += kSortThreads) count[i] = 0;
    __syncthreads();
    const int64_t part = int64_t(rank) * kSortWarps + warp, parts = int64_t(ctas) * kSortWarps;
    const int32_t i0 = int32_t(p.n * part / parts), i1 = int32_t(p.n * (part + 1) / parts);
    int32_t* mine = count + warp * E;
    auto expert_of = [&](int64_t i) {
        if (i >= i1) return -1;
        const int64_t e = p.ids[i];
        return e >= 0 && e < E ? int32_t(e) : -1;
    };
    for (int64_t i = i0; i < i1; i += 32) {
        const int32_t e = expert_of(i + lane);
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && lane == __ffs(int(same)) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // Over the warps: each warp's count becomes the number of choices of that expert before it.
    for (int32_t e = int32_t(threadIdx.x); e < E; e += kSortThreads) {
        int32_t sum = 0;
#pragma unroll 8
        for (int32_t w = 0; w < kSortWarps; ++w) {
            const int32_t c = count[w * E + e];
            count[w * E + e] = sum;
            sum += c;
        }
        total[e] = sum;
    }
    if (ctas > 1)
        ptx::cluster_sync_all();
    else
        __syncthreads();
    // Over CTAs and experts (a thread an expert).
    int32_t all = 0, before = 0;
    if (int32_t(threadIdx.x) < E) {
        const uint32_t at = ptx::smem_addr(total + threadIdx.x);
        for (uint32_t r = 0; r < ctas; ++r) {
            const int32_t c = ctas > 1 ? int32_t(ptx::ld_shared_cluster_u32(ptx::mapa_shared(at, r))) : total[threadIdx.x];
            if (r < rank) before += c;
            all += c;
        }
    }
    int32_t scan = all;                                 // inclusive, over the warp
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int32_t x = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += x;
    }
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    int32_t below = lane < warp ? sums[lane] : 0;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) below += __shfl_xor_sync(0xffffffffu, below, d);
    if (int32_t(threadIdx.x) < E) {
        start[threadIdx.x] = below + scan - all + before;
        if (rank == 0) {
            p.offsets[threadIdx.x + 1] = below + scan;
            if (threadIdx.x == 0) p.offsets[0] = 0;
        }
    }
    __syncthreads();
    for (int64_t i = i0; i < i1; i += 32) {
        const int32_t e = expert_of(i + lane);
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        int32_t place = -1;
        if (e >= 0) place = start[e] + mine[e] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (e >= 0 && lane == __ffs(int(same)) - 1) mine[e] += __popc(same);
        __syncwarp();
        if (i + lane < i1) p.positions[i + lane] = place;
    }
    if (ctas > 1) ptx::cluster_sync_all();              // the peers have read `total`
}

// ------------------------------------------------------------ rows
template <typename T>
struct Rows {
    const T *X, *Ys, *R;
    T *Xs, *Y;
    int64_t ldx, ldys, ldr, ldxs, ldy;
    const int32_t *positions, *offsets;
    const float* weights;
    float* dweights;
    int32_t T_, k, D, experts;
    int64_t rows;                                       // of Ys or Xs
};

// blockDim.x / tpr tokens a CTA; a thread takes every tpr-th vector of the row.
// The token's k choices stand for k rows of Xs as well: those behind the last
// expert's are zeroed.
template <typename T, bool VEC>
__global__ void __launch_bounds__(512) moe_dispatch_kernel(const Rows<T> a, int32_t tpr) {
    ptx::griddep_wait();
    const int32_t t = int32_t(threadIdx.x) % tpr, per = int32_t(blockDim.x) / tpr;
    const int32_t total = a.offsets[a.experts];
    for (int64_t row = int64_t(blockIdx.x) * per + int32_t(threadIdx.x) / tpr; row < a.T_; row += int64_t(gridDim.x) * per) {
        const int32_t* pos = a.positions + row * a.k;
        for (int32_t c = 0, v = 0; c < a.D; c += tpr * 8, ++v) {
            float x[8];
            load_row8<T, VEC>(x, a.X + row * a.ldx, v, t, tpr, a.D);
            for (int32_t j = 0; j < a.k; ++j) {
                const int32_t at = pos[j];
                if (at >= 0 && at < a.rows) store_row8<T, VEC>(a.Xs + at * a.ldxs, x, v, t, tpr, a.D);
            }
            const float zero[8] = {};
            for (int64_t r = row * a.k > total ? row * a.k : int64_t(total); r < (row + 1) * a.k; ++r)
                store_row8<T, VEC>(a.Xs + r * a.ldxs, zero, v, t, tpr, a.D);
        }
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(512) moe_combine_rows_kernel(const Rows<T> a, int32_t tpr) {
    ptx::griddep_wait();
    const int32_t t = int32_t(threadIdx.x) % tpr, per = int32_t(blockDim.x) / tpr;
    for (int64_t row = int64_t(blockIdx.x) * per + int32_t(threadIdx.x) / tpr; row < a.T_; row += int64_t(gridDim.x) * per) {
        const int32_t* pos = a.positions + row * a.k;
        for (int32_t c = 0, v = 0; c < a.D; c += tpr * 8, ++v) {
            float y[8] = {};
            for (int32_t j0 = 0; j0 < a.k; j0 += 4) {
                Raw8<T> x[4];
                float w[4];
                bool on[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int32_t at = j0 + j < a.k ? pos[j0 + j] : -1;
                    on[j] = at >= 0 && at < a.rows;
                    if (!on[j]) continue;
                    w[j] = a.weights != nullptr ? a.weights[row * a.k + j0 + j] : 1.f;
                    load_raw8<VEC>(x[j], a.Ys + at * a.ldys, v, t, tpr, a.D);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (on[j])
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = fmaf(w[j], raw_at(x[j], i), y[i]);
            }
            if (a.R != nullptr) {
                float r[8];
                load_row8<T, VEC>(r, a.R + row * a.ldr, v, t, tpr, a.D);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] += r[i];
            }
            store_row8<T, VEC>(a.Y + row * a.ldy, y, v, t, tpr, a.D);
        }
    }
}

// X is dY, Xs is dYs.  Four choices at a time: their products with dY are summed over the group.
template <typename T, bool VEC>
__global__ void __launch_bounds__(512) moe_combine_grad_kernel(const Rows<T> a, int32_t tpr) {
    __shared__ float buf[4][32];
    ptx::griddep_wait();
    const int32_t t = int32_t(threadIdx.x) % tpr, per = int32_t(blockDim.x) / tpr;
    const int32_t total = a.Xs != nullptr ? a.offsets[a.experts] : 0;
    for (int64_t first = int64_t(blockIdx.x) * per; first < a.T_; first += int64_t(gridDim.x) * per) {
        const int64_t row = first + int32_t(threadIdx.x) / tpr;
        const bool in = row < a.T_;                     // a group past the end only keeps the barriers
        for (int32_t j0 = 0; j0 < a.k; j0 += 4) {
            int32_t at[4];
            float w[4], dot[4] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                at[j] = in && j0 + j < a.k ? a.positions[row * a.k + j0 + j] : -1;
                if (at[j] >= a.rows) at[j] = -1;
                w[j] = at[j] >= 0 ? a.weights[row * a.k + j0 + j] : 0.f;
            }
            for (int32_t c = 0, v = 0; c < a.D && in; c += tpr * 8, ++v) {
                float d[8];
                load_row8<T, VEC>(d, a.X + row * a.ldx, v, t, tpr, a.D);
                Raw8<T> y[4] = {};
                if (a.dweights != nullptr)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (at[j] >= 0) load_raw8<VEC>(y[j], a.Ys + at[j] * a.ldys, v, t, tpr, a.D);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (at[j] < 0) continue;
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (a.dweights != nullptr) dot[j] = fmaf(d[i], raw_at(y[j], i), dot[j]);
                        x[i] = w[j] * d[i];
                    }
                    if (a.Xs != nullptr) store_row8<T, VEC>(a.Xs + at[j] * a.ldxs, x, v, t, tpr, a.D);
                }
                if (a.Xs != nullptr && j0 == 0) {
                    const float zero[8] = {};
                    for (int64_t r = row * a.k > total ? row * a.k : int64_t(total); r < (row + 1) * a.k; ++r)
                        store_row8<T, VEC>(a.Xs + r * a.ldxs, zero, v, t, tpr, a.D);
                }
            }
            if (a.dweights != nullptr) {
                group_sum(dot, buf, tpr);
                if (t == 0)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (in && j0 + j < a.k) a.dweights[row * a.k + j0 + j] = at[j] >= 0 ? dot[j] : 0.f;
                if (tpr > 32) __syncthreads();          // buf, for the next choices
            }
        }
    }
}

template <typename T>
bool aligned16(const Mat& m, int64_t rows) {
    return !m || (reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && (rows <= 1 || m.ld % int64_t(16 / sizeof(T)) == 0));
}

// Threads a row and in all: the fewest warps that hold a row with one vector each, at most 512.
struct Shape {
    int32_t tpr;
    int threads;
    unsigned grid;
};
Shape shape_for(int32_t D, int32_t T, int sm_count) {
    Shape s;
    s.tpr = 32;
    while (s.tpr < 512 && s.tpr * 8 < D) s.tpr *= 2;
    s.threads = std::max(256, int(s.tpr));
    s.grid = unsigned(std::min<int64_t>(cdiv(T, s.threads / s.tpr), int64_t(sm_count) * 16));
    return s;
}

template <typename T>
int launch_rows(void* kernel, Rows<T> p, const LibCtx& c, const char* what, cudaStream_t stream) {
    Shape s = shape_for(p.D, p.T_, c.sm_count);
    void* args[] = {&p, &s.tpr};
    const cudaError_t e = launch_kernel(kernel, dim3(s.grid), s.threads, 0, 1, args, stream);
    if (e != cudaSuccess) return report_cuda(e, what);
    count_launch();
    return GBR_OK;
}

template <typename T>
int dispatch(const MoeRowsArgs& a, const LibCtx& c, cudaStream_t stream) {
    Rows<T> p = {};
    p.X = static_cast<const T*>(a.X.p), p.ldx = a.X.ld;
    p.Xs = static_cast<T*>(a.Ys.w()), p.ldxs = a.Ys.ld;
    p.positions = a.positions, p.offsets = a.offsets;
    p.T_ = a.T, p.k = a.k, p.D = a.D, p.experts = a.experts, p.rows = int64_t(a.T) * a.k;
    const bool vec = a.D % 8 == 0 && aligned16<T>(a.X, a.T) && aligned16<T>(a.Ys, p.rows);
    return launch_rows(vec ? reinterpret_cast<void*>(&moe_dispatch_kernel<T, true>)
                           : reinterpret_cast<void*>(&moe_dispatch_kernel<T, false>),
                       p, c, "launching moe_dispatch", stream);
}

template <typename T>
int combine(const MoeRowsArgs& a, int64_t rows, const LibCtx& c, cudaStream_t stream) {
    Rows<T> p = {};
    p.Ys = static_cast<const T*>(a.Ys.p), p.ldys = a.Ys.ld;
    p.R = static_cast<const T*>(a.R.p), p.ldr = a.R.ld;
    p.Y = static_cast<T*>(a.Y.w()), p.ldy = a.Y.ld;
    p.positions = a.positions, p.weights = a.weights;
    p.T_ = a.T, p.k = a.k, p.D = a.D, p.rows = rows;
    const bool vec = a.D % 8 == 0 && aligned16<T>(a.Ys, rows) && aligned16<T>(a.R, a.T) && aligned16<T>(a.Y, a.T);
    return launch_rows(vec ? reinterpret_cast<void*>(&moe_combine_rows_kernel<T, true>)
                           : reinterpret_cast<void*>(&moe_combine_rows_kernel<T, false>),
                       p, c, "launching moe_combine", stream);
}

template <typename T>
int combine_grad(const MoeCombineGradArgs& a, const LibCtx& c, cudaStream_t stream) {
    Rows<T> p = {};
    p.X = static_cast<const T*>(a.dY.p), p.ldx = a.dY.ld;
    p.Ys = static_cast<const T*>(a.Ys.p), p.ldys = a.Ys.ld;
    p.Xs = static_cast<T*>(a.dYs.w()), p.ldxs = a.dYs.ld;
    p.positions = a.positions, p.offsets = a.offsets, p.weights = a.weights, p.dweights = a.dweights;
    p.T_ = a.T, p.k = a.k, p.D = a.D, p.experts = a.experts, p.rows = int64_t(a.T) * a.k;
    const bool vec = a.D % 8 == 0 && aligned16<T>(a.dY, a.T) && aligned16<T>(a.Ys, p.rows) && aligned16<T>(a.dYs, p.rows);
    return launch_rows(vec ? reinterpret_cast<void*>(&moe_combine_grad_kernel<T, true>)
                           : reinterpret_cast<void*>(&moe_combine_grad_kernel<T, false>),
                       p, c, "launching moe_combine_backward", stream);
}

}  // namespace

int launch_moe_sort(const MoeSortArgs& a, const LibCtx& c, cudaStream_t stream) {
    SortParams p = {a.ids, a.positions, a.offsets, a.n, a.experts};
    uint32_t ctas = a.n > 8192 ? kSortCluster : 1;
    const size_t smem = (size_t(kSortWarps + 2) * size_t(a.experts) + 32) * sizeof(int32_t);
    void* kernel = reinterpret_cast<void*>(&moe_sort_kernel);
    const int r = raise_kernel_smem(kernel, smem, c.device);
    if (r != GBR_OK) return r;
    void* args[] = {&p, &ctas};
    const cudaError_t e = launch_kernel(kernel, dim3(ctas), kSortThreads, smem, int(ctas), args, stream);
    if (e != cudaSuccess) return report_cuda(e, "launching moe_sort");
    count_launch();
    return GBR_OK;
}

int launch_moe_dispatch(const MoeRowsArgs& a, const LibCtx& c, cudaStream_t stream) {
    return a.bf16 ? dispatch<__nv_bfloat16>(a, c, stream) : dispatch<float>(a, c, stream);
}
int launch_moe_combine(const MoeRowsArgs& a, int64_t rows, const LibCtx& c, cudaStream_t stream) {
    return a.bf16 ? combine<__nv_bfloat16>(a, rows, c, stream) : combine<float>(a, rows, c, stream);
}
int launch_moe_combine_grad(const MoeCombineGradArgs& a, const LibCtx& c, cudaStream_t stream) {
    return a.bf16 ? combine_grad<__nv_bfloat16>(a, c, stream) : combine_grad<float>(a, c, stream);
}

}  // namespace gbr
