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
constexpr int kSortThreads = 1024, kSortCluster = 8, kSortBatch = 8;

struct SortParams {
    const int64_t* ids;
    int32_t *positions, *offsets;
    int32_t n, experts;
};

__global__ void __launch_bounds__(kSortThreads, 1) moe_sort_kernel(const SortParams p, uint32_t ctas) {
    extern __shared__ int32_t sm[];
    const int32_t threads = int32_t(blockDim.x), warps = threads / 32;
    int32_t* count = sm;                                // [warps][experts]
    int32_t* total = count + warps * p.experts;         // [experts] of this CTA, read by the peers
    int32_t* start = total + p.experts;                 // [experts] first place of this CTA's choices
    int32_t* sums = start + p.experts;                  // [32]
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();                   // at most 8 CTAs: what comes next may set itself up
    const uint32_t rank = ctas > 1 ? ptx::cluster_ctarank() : 0u;
    const int32_t warp = int32_t(threadIdx.x) / 32, lane = int32_t(threadIdx.x) % 32, E = p.experts;
    for (int32_t i = int32_t(threadIdx.x); i < warps * E; i += threads) count[i] = 0;
    __syncthreads();
    const int64_t part = int64_t(rank) * warps + warp, parts = int64_t(ctas) * warps;
    const int32_t i0 = int32_t(p.n * part / parts), i1 = int32_t(p.n * (part + 1) / parts);
    int32_t* mine = count + warp * E;
    int32_t e[kSortBatch];
    auto load = [&](int64_t i) {
#pragma unroll
        for (int b = 0; b < kSortBatch; ++b) {
            const int64_t at = i + 32 * b + lane, id = at < i1 ? p.ids[at] : -1;
            e[b] = id >= 0 && id < E ? int32_t(id) : -1;
        }
    };
    for (int64_t i = i0; i < i1; i += 32 * kSortBatch) {
        load(i);
#pragma unroll
        for (int b = 0; b < kSortBatch; ++b) {
            if (i + 32 * b >= i1) break;
            const uint32_t same = __match_any_sync(0xffffffffu, e[b]);
            if (e[b] >= 0 && lane == __ffs(int(same)) - 1) mine[e[b]] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    // Over the warps: each warp's count becomes the number of choices of that expert before it.
    for (int32_t x = int32_t(threadIdx.x); x < E; x += threads) {
        int32_t sum = 0;
#pragma unroll 8
        for (int32_t w = 0; w < warps; ++w) {
            const int32_t c = count[w * E + x];
            count[w * E + x] = sum;
            sum += c;
        }
        total[x] = sum;
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
    const bool again = i1 - i0 > 32 * kSortBatch;       // else the ids are still in registers
    for (int64_t i = i0; i < i1; i += 32 * kSortBatch) {
        if (again) load(i);
#pragma unroll
        for (int b = 0; b < kSortBatch; ++b) {
            if (i + 32 * b >= i1) break;
            const uint32_t same = __match_any_sync(0xffffffffu, e[b]);
            int32_t place = -1;
            if (e[b] >= 0) place = start[e[b]] + mine[e[b]] + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (e[b] >= 0 && lane == __ffs(int(same)) - 1) mine[e[b]] += __popc(same);
            __syncwarp();
            if (i + 32 * b + lane < i1) p.positions[i + 32 * b + lane] = place;
        }
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

// CTAs an SM that registers let in.  One round of them is best: 4096 tokens of 4096 columns, 2 choices, with 3 / 4 / 6 / 8
// an SM of 4: combined 26.1 / 23.9 / 27.4 / 26.0 us, gradients 30.2 / 28.2 / 32.4 / 31.0.
template <typename T>
constexpr int kResident = sizeof(T) == 2 ? 4 : 3;

// A CTA takes a run of tokens, whose positions (and weights) it fetches first, so that from then on no load waits for
// another; blockDim.x / tpr tokens at a time, kV vectors of 8 columns a thread at once.  Taking a token's positions when
// its turn came: 4096 tokens of 4096 columns and 2 choices 24.8 us dispatched, 42.5 combined.  HELD false: a token is
// all that a group of threads has, and its places are read as they are wanted (301 tokens of 1000 columns and 6 choices,
// the gradient: 5.7 us held, 4.5 not); or there are more choices than the CTA holds.
constexpr int kPlaces = 256;                           // choices that a CTA holds at a time

// The CTA's tokens, in turns of as many as kPlaces choices are of.
struct TokenRun {
    int64_t begin, end;
    int32_t turn;
};
template <typename T>
__device__ __forceinline__ TokenRun token_run(const Rows<T>& a) {
    return {int64_t(a.T_) * blockIdx.x / gridDim.x, int64_t(a.T_) * (blockIdx.x + 1) / gridDim.x,
            a.k > 0 && a.k < kPlaces ? kPlaces / a.k : 1};
}

// Positions (-1 where there is no row) and weights of the choices from (token, j0) on into shared memory.
template <typename T>
__device__ __forceinline__ void fetch_places(const Rows<T>& a, int64_t first, int32_t n, int32_t* at, float* w) {
    __syncthreads();                                    // the last turn's have been read
    for (int32_t i = int32_t(threadIdx.x); i < n; i += int32_t(blockDim.x)) {
        const int32_t p = a.positions[first + i];
        at[i] = p >= 0 && p < a.rows ? p : -1;
        if (w != nullptr) w[i] = a.weights != nullptr ? a.weights[first + i] : 1.f;
    }
    __syncthreads();
}

template <typename T, int A, int kV, bool HELD>
__global__ void __launch_bounds__(256, kResident<T>) moe_dispatch_kernel(const Rows<T> a, int32_t tpr) {
    __shared__ int32_t at[kPlaces];
    ptx::griddep_wait();
    const int32_t t = int32_t(threadIdx.x) % tpr, group = int32_t(threadIdx.x) / tpr, per = int32_t(blockDim.x) / tpr;
    const TokenRun run = token_run(a);
    const int64_t total = a.offsets[a.experts];
    const float zero[8] = {};
    for (int64_t first = run.begin; first < run.end; first += run.turn) {
        const int32_t tokens = int32_t(run.end - first < run.turn ? run.end - first : run.turn);
        // More choices than the CTA holds: one token, part by part.
        for (int32_t j0 = 0; j0 < a.k; j0 += kPlaces) {
            const int32_t k = a.k - j0 < kPlaces ? a.k - j0 : kPlaces;
            // A piece: kV vectors of a token.  The next one is loaded before this one is stored, the first before the
            // places are there.
            const int32_t pieces = (a.D + tpr * 8 * kV - 1) / (tpr * 8 * kV);
            auto load = [&](Raw8<T> (&x)[kV], int32_t i, int32_t v0) {
#pragma unroll
                for (int v = 0; v < kV; ++v)
                    load_raw8<A>(x[v], a.X + (first + i) * a.ldx, v0 + v, t, tpr, i < tokens ? a.D : 0);
            };
            Raw8<T> next[kV];
            load(next, group, 0);
            if (HELD) fetch_places(a, first * a.k + j0, tokens * k, at, nullptr);
            for (int32_t i = group; i < tokens; i += per) {
                const int32_t* pos = HELD ? at + i * k : a.positions + (first + i) * a.k + j0;
                for (int32_t piece = 0; piece < pieces; ++piece) {
                    const int32_t v0 = piece * kV;
                    Raw8<T> x[kV];
#pragma unroll
                    for (int v = 0; v < kV; ++v) x[v] = next[v];
                    if (piece + 1 < pieces) load(next, i, v0 + kV);
                    else load(next, i + per, 0);
                    if (row_col(v0, t & ~31, tpr) >= a.D) continue;     // the warp has no columns
                    for (int32_t j = 0; j < k; ++j) {
                        const int32_t to = pos[j];
                        if (to < 0 || (!HELD && to >= a.rows)) continue;
#pragma unroll
                        for (int v = 0; v < kV; ++v) store_raw8<A>(a.Xs + to * a.ldxs, x[v], v0 + v, t, tpr, a.D);
                    }
                    // The token's k choices stand for k rows of Xs as well: those behind the last expert's are zeroed.
                    const int64_t r0 = (first + i) * a.k + j0;
                    for (int64_t r = r0 > total ? r0 : total; r < r0 + k; ++r)
#pragma unroll
                        for (int v = 0; v < kV; ++v) store_row8<T, A>(a.Xs + r * a.ldxs, zero, v0 + v, t, tpr, a.D);
                }
            }
        }
    }
}

// kJ choices at once.
template <typename T, int A, int kV, int kJ, bool HELD>
__global__ void __launch_bounds__(256, kResident<T>) moe_combine_rows_kernel(const Rows<T> a, int32_t tpr) {
    __shared__ int32_t at[kPlaces];
    __shared__ float weight[kPlaces];
    ptx::griddep_wait();
    const int32_t t = int32_t(threadIdx.x) % tpr, group = int32_t(threadIdx.x) / tpr, per = int32_t(blockDim.x) / tpr;
    const TokenRun run = token_run(a);
    for (int64_t first = run.begin; first < run.end; first += run.turn) {
        const int32_t tokens = int32_t(run.end - first < run.turn ? run.end - first : run.turn);
        if (HELD) fetch_places(a, first * a.k, tokens * a.k, at, weight);
        for (int32_t i = group; i < tokens; i += per) {
            const int64_t row = first + i;
            for (int32_t v0 = 0; row_col(v0, t & ~31, tpr) < a.D; v0 += kV) {        // while the warp has columns
                float y[kV][8] = {};
                Raw8<T> r[kV];
                if (a.R != nullptr)
#pragma unroll
                    for (int v = 0; v < kV; ++v) load_raw8<A>(r[v], a.R + row * a.ldr, v0 + v, t, tpr, a.D);
                for (int32_t j0 = 0; j0 < a.k; j0 += kJ) {
                    Raw8<T> x[kJ][kV];
                    float w[kJ];
                    bool on[kJ];
#pragma unroll
                    for (int j = 0; j < kJ; ++j) {
                        int32_t p = -1;
                        if (j0 + j < a.k) {
                            const int64_t c = row * a.k + j0 + j;
                            p = HELD ? at[i * a.k + j0 + j] : a.positions[c];
                            w[j] = HELD ? weight[i * a.k + j0 + j] : a.weights != nullptr ? a.weights[c] : 1.f;
                        }
                        on[j] = p >= 0 && p < a.rows;
                        if (!on[j]) continue;
#pragma unroll
                        for (int v = 0; v < kV; ++v) load_raw8<A>(x[j][v], a.Ys + p * a.ldys, v0 + v, t, tpr, a.D);
                    }
#pragma unroll
                    for (int j = 0; j < kJ; ++j) {
                        if (!on[j]) continue;
#pragma unroll
                        for (int v = 0; v < kV; ++v)
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[v][e] = fmaf(w[j], raw_at(x[j][v], e), y[v][e]);
                    }
                }
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    if (a.R != nullptr)
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[v][e] += raw_at(r[v], e);
                    store_row8<T, A>(a.Y + row * a.ldy, y[v], v0 + v, t, tpr, a.D);
                }
            }
        }
    }
}

// X is dY, Xs is dYs.  kJ choices at once: their products with dY are summed over the token's threads.
template <typename T, int A, int kV, int kJ, bool HELD>
__global__ void __launch_bounds__(256, kResident<T>) moe_combine_grad_kernel(const Rows<T> a, int32_t tpr) {
    __shared__ int32_t at[kPlaces];
    __shared__ float weight[kPlaces];
    __shared__ float buf[kJ][32];
    ptx::griddep_wait();
    const int32_t t = int32_t(threadIdx.x) % tpr, group = int32_t(threadIdx.x) / tpr, per = int32_t(blockDim.x) / tpr;
    const TokenRun run = token_run(a);
    const int64_t total = a.Xs != nullptr ? a.offsets[a.experts] : 0;
    const bool dots = a.dweights != nullptr, rows_out = a.Xs != nullptr;
    const float zero[8] = {};
    for (int64_t first = run.begin; first < run.end; first += run.turn) {
        const int32_t tokens = int32_t(run.end - first < run.turn ? run.end - first : run.turn);
        if (HELD) fetch_places(a, first * a.k, tokens * a.k, at, weight);
        for (int32_t i0 = 0; i0 < tokens; i0 += per) {
            const int32_t i = i0 + group, cols = i < tokens ? a.D : 0;   // a group past the end only keeps the barriers
            const int64_t row = first + i;
            for (int32_t j0 = 0; j0 < a.k; j0 += kJ) {
                int32_t p[kJ];
                float w[kJ], dot[kJ];
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    p[j] = -1, w[j] = dot[j] = 0.f;
                    if (i < tokens && j0 + j < a.k) {
                        const int64_t c = row * a.k + j0 + j;
                        p[j] = HELD ? at[i * a.k + j0 + j] : a.positions[c];
                        if (p[j] >= a.rows) p[j] = -1;
                        if (p[j] >= 0) w[j] = HELD ? weight[i * a.k + j0 + j] : a.weights[c];
                    }
                }
                for (int32_t v0 = 0; row_col(v0, t & ~31, tpr) < cols; v0 += kV) {   // while the warp has columns
                    Raw8<T> d[kV], y[kJ][kV];
#pragma unroll
                    for (int v = 0; v < kV; ++v) load_raw8<A>(d[v], a.X + row * a.ldx, v0 + v, t, tpr, cols);
                    if (dots)
#pragma unroll
                        for (int j = 0; j < kJ; ++j)
#pragma unroll
                            for (int v = 0; v < kV; ++v)
                                if (p[j] >= 0) load_raw8<A>(y[j][v], a.Ys + p[j] * a.ldys, v0 + v, t, tpr, cols);
#pragma unroll
                    for (int j = 0; j < kJ; ++j) {
                        if (p[j] < 0) continue;
#pragma unroll
                        for (int v = 0; v < kV; ++v) {
                            float x[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                if (dots) dot[j] = fmaf(raw_at(d[v], e), raw_at(y[j][v], e), dot[j]);
                                x[e] = w[j] * raw_at(d[v], e);
                            }
                            if (rows_out) store_row8<T, A>(a.Xs + p[j] * a.ldxs, x, v0 + v, t, tpr, cols);
                        }
                    }
                    if (rows_out && j0 == 0)
                        for (int64_t r = row * a.k > total ? row * a.k : total; r < (row + 1) * a.k; ++r)
#pragma unroll
                            for (int v = 0; v < kV; ++v) store_row8<T, A>(a.Xs + r * a.ldxs, zero, v0 + v, t, tpr, cols);
                }
                if (!dots) continue;
                group_sum(dot, buf, tpr, group);
                if (t == 0)
#pragma unroll
                    for (int j = 0; j < kJ; ++j)
                        if (i < tokens && j0 + j < a.k) a.dweights[row * a.k + j0 + j] = p[j] >= 0 ? dot[j] : 0.f;
                if (tpr > 32) __syncthreads();          // buf, for the next choices
            }
        }
    }
}

template <typename T>
bool aligned16(const Mat& m, int64_t rows) {
    return !m || (reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && (rows <= 1 || m.ld % int64_t(16 / sizeof(T)) == 0));
}

// Threads a row: whole warps that hold it with kV vectors each, in as few rounds as 256 of them would need.  Powers of two /
// this, us, bf16: combination of 4000 x 2560 with 2 choices 18.7 / 15.4, 2000 x 2312 with 6 23.9 / 19.7, gradients of 6000 x
// 1432 with 2 18.5 / 16.4.
int32_t threads_for(int32_t D, int kV) {
    const int64_t vectors = cdiv(D, 8 * kV), rounds = std::max<int64_t>(1, cdiv(vectors, 256));
    return int32_t(std::max<int64_t>(1, cdiv(cdiv(vectors, rounds), 32)) * 32);
}

// `kernels`: places held, places read.
template <typename T>
int launch_rows(void* const (&kernels)[2], Rows<T> p, int kV, const LibCtx& c, const char* what, cudaStream_t stream) {
    int32_t tpr = threads_for(p.D, kV);
    const int32_t groups = 256 / tpr, threads = groups * tpr;
    const int64_t turns = cdiv(p.T_, groups), grid = std::min<int64_t>(turns, int64_t(c.sm_count) * (kResident<T> * 256 / threads));
    void* args[] = {&p, &tpr};
    void* kernel = kernels[turns > grid && p.k <= kPlaces ? 0 : 1];
    const cudaError_t e = launch_kernel(kernel, dim3(unsigned(grid)), threads, 0, 1, args, stream);
    if (e != cudaSuccess) return report_cuda(e, what);
    count_launch();
    return GBR_OK;
}

#define GBR_BOTH(...) \
    {reinterpret_cast<void*>(&__VA_ARGS__, true>), reinterpret_cast<void*>(&__VA_ARGS__, false>)}

template <typename T>
int dispatch(const MoeRowsArgs& a, const LibCtx& c, cudaStream_t stream) {
    Rows<T> p = {};
    p.X = static_cast<const T*>(a.X.p), p.ldx = a.X.ld;
    p.Xs = static_cast<T*>(a.Ys.w()), p.ldxs = a.Ys.ld;
    p.positions = a.positions, p.offsets = a.offsets;
    p.T_ = a.T, p.k = a.k, p.D = a.D, p.experts = a.experts, p.rows = int64_t(a.T) * a.k;
    const bool vec = a.D % 8 == 0 && aligned16<T>(a.X, a.T) && aligned16<T>(a.Ys, p.rows);
    void* const wide[2] = GBR_BOTH(moe_dispatch_kernel<T, kVec, 2);
    void* const any[2] = GBR_BOTH(moe_dispatch_kernel<T, kShifted, 1);
    return launch_rows(vec ? wide : any, p, vec ? 2 : 1, c, "launching moe_dispatch", stream);
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
    // One or two choices: two vectors a thread; more: one, and four choices at once (eight spill registers: 2000 tokens of
    // 2048 columns and 6 choices, bf16, 16.7 us with four, 23.8 with eight; fp32 spills 16 to 44 bytes with four, its
    // gradients 124 to 156).
    const bool few = vec && a.k <= 2;
    void* const two[2] = GBR_BOTH(moe_combine_rows_kernel<T, kVec, 2, 2);
    void* const four[2] = GBR_BOTH(moe_combine_rows_kernel<T, kVec, 1, 4);
    void* const any[2] = GBR_BOTH(moe_combine_rows_kernel<T, kShifted, 1, 4);
    return launch_rows(!vec ? any : few ? two : four, p, few ? 2 : 1, c, "launching moe_combine", stream);
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
    const bool few = vec && a.k <= 2;
    void* const two[2] = GBR_BOTH(moe_combine_grad_kernel<T, kVec, 2, 2);
    void* const four[2] = GBR_BOTH(moe_combine_grad_kernel<T, kVec, 1, 4);
    void* const any[2] = GBR_BOTH(moe_combine_grad_kernel<T, kShifted, 1, 4);
    return launch_rows(!vec ? any : few ? two : four, p, few ? 2 : 1, c, "launching moe_combine_backward", stream);
}

}  // namespace

int launch_moe_sort(const MoeSortArgs& a, const LibCtx& c, cudaStream_t stream) {
    SortParams p = {a.ids, a.positions, a.offsets, a.n, a.experts};
    // Few choices: 8 warps, whose counts are sooner added than those of 32 (a thread an expert, so no more experts).
    uint32_t ctas = a.n > 4096 ? kSortCluster : 1;
    const int threads = a.n <= 2048 && a.experts <= 256 ? 256 : kSortThreads;
    const size_t smem = (size_t(threads / 32 + 2) * size_t(a.experts) + 32) * sizeof(int32_t);
    void* kernel = reinterpret_cast<void*>(&moe_sort_kernel);
    const int r = raise_kernel_smem(kernel, smem, c.device);
    if (r != GBR_OK) return r;
    void* args[] = {&p, &ctas};
    const cudaError_t e = launch_kernel(kernel, dim3(ctas), threads, smem, int(ctas), args, stream);
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
