// residual_norm.cu -- the norms before and after a block with its gate and the
// residual, and their gradients.
//
//   y = X q post,  q = 1 / sqrt(mean X^2 + eps)      (no post: y = X)
//   S = R + scale gate y
//   H = S r pre,   r = 1 / sqrt(mean S^2 + eps)
//
//   u = dH pre;  ds = dS + r (u - S r^2 mean(u S))    dR = ds, dpre = sum dH S r
//   dy = scale gate ds                                dgate = sum scale y ds
//   v = dy post; dX = q (v - X q^2 mean(v X))         dpost = sum dy X q
//
// No square or cube of a root is formed alone: of a row's mean m, r m comes first, which is about as large as u, then
// r (r m).  r^3 is subnormal for rows of 10^13 and more and infinite for rows below 10^-13.
//
// Bound by memory: every operand is read once and every output written once; a
// group of threads holds its row in registers between the passes that the two
// means need.  Statistics and sums are fp32.  H comes from the sum before it is
// rounded to S.
#include "gbr.h"
#include "operators.h"
#include "row8.cuh"

#include <algorithm>
#include <cfloat>
#include <cstdint>

namespace gbr {
namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename T>
struct Args {
    const T *X, *R, *G;
    const float *post, *pre;
    T *S, *H;
    int64_t ldx, ldr, ldg, lds, ldh, ld_odd;            // ld_odd: of the rows, whole aligned pieces left out
    int32_t rows, cols, per_gate;      // rows that share a row of G
    float scale, eps, inv_cols;
};

__device__ __forceinline__ float root(float sum, float inv_cols, float eps) { return rsqrtf(fmaf(sum, inv_cols, eps)); }

// ------------------------------------------------------------ forward
// blockDim.x / tpr rows a CTA, V * 8 columns a thread.  (Four vectors, rows of more than 16384 columns, spill: 400 to 460 bytes
// on 16 bytes, 1900 to 2100 elsewhere, at 32 registers a thread.)
template <typename T, int V, bool VEC>
__global__ void __launch_bounds__(1024) residual_norm_kernel(const Args<T> a, int32_t tpr) {
    __shared__ float buf[2][1][32];
    ptx::griddep_wait();
    const int32_t t = int32_t(threadIdx.x) % tpr, group = int32_t(threadIdx.x) / tpr;
    const int64_t row = int64_t(blockIdx.x) * (int32_t(blockDim.x) / tpr) + group;
    const int32_t cols = row < a.rows ? a.cols : 0;    // a group past the end only keeps the barriers
    float s[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) load_row8<T, VEC>(s[v], a.X + row * a.ldx, v, t, tpr, cols);
    if (a.R != nullptr || a.G != nullptr || a.post != nullptr || a.scale != 1.f) {
        Raw8<T> r[V] = {}, g[V];
        if (a.R != nullptr)
#pragma unroll
            for (int v = 0; v < V; ++v) load_raw8<VEC>(r[v], a.R + row * a.ldr, v, t, tpr, cols);
        if (a.G != nullptr)
#pragma unroll
            for (int v = 0; v < V; ++v) load_raw8<VEC>(g[v], a.G + row / a.per_gate * a.ldg, v, t, tpr, cols);
        float q = 1.f;
        if (a.post != nullptr) {
            float sum[1] = {};
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[0] = fmaf(s[v][j], s[v][j], sum[0]);
            group_sum(sum, buf[0], tpr, group);
            q = root(sum[0], a.inv_cols, a.eps);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float w[8];
            if (a.post != nullptr) load_row8<float, VEC>(w, a.post, v, t, tpr, cols);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float y = s[v][j];
                if (a.post != nullptr) y = y * q * w[j];
                if (a.G != nullptr) y *= raw_at(g[v], j);
                s[v][j] = fmaf(a.scale, y, raw_at(r[v], j));
            }
        }
    }
    if (a.S != nullptr)
#pragma unroll
        for (int v = 0; v < V; ++v) store_row8<T, VEC>(a.S + row * a.lds, s[v], v, t, tpr, cols);
    if (a.H == nullptr) return;
    float sum[1] = {};
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[0] = fmaf(s[v][j], s[v][j], sum[0]);
    group_sum(sum, buf[1], tpr, group);
    const float q = root(sum[0], a.inv_cols, a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float w[8];
        load_row8<float, VEC>(w, a.pre, v, t, tpr, cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = s[v][j] * q * w[j];
        store_row8<T, VEC>(a.H + row * a.ldh, w, v, t, tpr, cols);
    }
}

// Many rows: CTAs that stay, blockDim.x / tpr rows a turn, the weights in registers and the next kAhead turns' X, R and
// gate on their way into shared memory, each thread its own 16 bytes, so that nobody waits for another's copy.  A gate
// per channel is in the weights.  row_bytes: of a row in shared memory; step: of a turn's rows of all inputs.
// ODD: rows start off 16 bytes, all operands' alike.  A CTA's are eight apart, so that they too start alike; its threads'
// pieces begin at the aligned address in front of a row, and only a row's ends go element by element.
// 16384 x 4096 bf16 with all but row gates: a row a CTA 131 us, this 84 (6.4 TB/s).  More on their way is slower, HBM
// reading and writing at once: three CTAs an SM and three turns ahead 97, two and three 84 to 88, two and five 95.
template <typename T, int V, int kAhead, int kMost, bool ODD>
__global__ void __launch_bounds__(kMost, kMost == 512 ? 1 : 2) residual_norm_stream_kernel(const Args<T> a, int32_t tpr,
                                                                                       uint32_t row_bytes, uint32_t step) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float buf[2][1][32];
    ptx::griddep_wait();
    const int32_t t = int32_t(threadIdx.x) % tpr, group = int32_t(threadIdx.x) / tpr, groups = int32_t(blockDim.x) / tpr;
    // ODD: the elements between the aligned address in front of a row and the row, the same for all rows of this CTA.
    constexpr int32_t kStep = ODD ? 8 : 1;
    int64_t first = ODD ? int64_t(blockIdx.x / 8) * groups * 8 + blockIdx.x % 8 : int64_t(blockIdx.x) * groups;
    const int32_t off = ODD ? int32_t(first * a.ld_odd % int32_t(16 / sizeof(T))) : 0, cols = a.cols + off;
    const bool has_r = a.R != nullptr, one_gate = a.G != nullptr && a.per_gate == a.rows, gates = a.G != nullptr && !one_gate;
    const uint32_t base = ptx::smem_addr(ring) + uint32_t(group) * row_bytes, wide = row_bytes * uint32_t(groups);
    auto copy = [&](uint32_t to, const T* from, int v) {
        if (ODD) copy_row8_from(to, from - off, v, t, tpr, cols);
        else copy_row8(to, from, v, t, tpr, cols);
    };
    auto take = [&](Raw8<T>& x, uint32_t from, int v) {
        take_row8(x, from, v, t, tpr);
        if (ODD && v == 0 && t == 0) clear_front(x, off);
    };
    auto load = [&](F2 (&x)[4], const auto* from, int v) {
        if constexpr (ODD) load_pairs_from(x, from, v, t, tpr, off, cols);
        else load_pairs<std::remove_cv_t<std::remove_pointer_t<decltype(from)>>, kVec>(x, from, v, t, tpr, cols);
    };
    auto store = [&](T* to, const F2 (&x)[4], int v, bool in) {
        if (ODD) store_pairs_from(to - off, x, v, t, tpr, off, in ? cols : 0);
        else store_pairs<T, kVec>(to, x, v, t, tpr, in ? cols : 0);
    };
    auto fetch = [&](int64_t row, uint32_t slot) {
        if (row < a.rows) {
            uint32_t to = base + slot * step;
#pragma unroll
            for (int v = 0; v < V; ++v) copy(to, a.X + row * a.ldx, v);
            if (has_r) {
                to += wide;
#pragma unroll
                for (int v = 0; v < V; ++v) copy(to, a.R + row * a.ldr, v);
            }
            if (gates) {
                to += wide;
#pragma unroll
                for (int v = 0; v < V; ++v) copy(to, a.G + row / a.per_gate * a.ldg, v);
            }
        }
        copy_async_commit();
    };
    // What X / root is multiplied by: scale, weight and a gate that is the same for all rows.
    F2 w[V][4], wpre[V][4];
    const bool post = a.post != nullptr;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        F2 g[4];
        if (post) load(w[v], a.post, v);
        if (a.pre != nullptr) load(wpre[v], a.pre, v);
        if (one_gate) load(g, a.G, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[v][i] = post ? mul2(w[v][i], f2(a.scale)) : f2(a.scale);
            if (one_gate) w[v][i] = mul2(w[v][i], g[i]);
        }
    }
    clear_past<T, V>(ptx::smem_addr(ring), kAhead * step / row_bytes, row_bytes, t, tpr, cols);
    const int64_t turn = int64_t(gridDim.x) * groups;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(first + group * kStep + i * turn, uint32_t(i));
    for (uint32_t slot = 0; first < a.rows; first += turn, slot = slot + 1 == kAhead ? 0 : slot + 1) {
        const int64_t row = first + group * kStep;
        const bool in = row < a.rows;                   // a group past the end only keeps the barriers
        copy_async_wait<kAhead - 1>();
        const uint32_t from = base + slot * step;
        Raw8<T> x[V], r[V] = {}, g[V] = {};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            take(x[v], from, v);
            if (has_r) take(r[v], from + wide, v);
            if (gates) take(g[v], from + (has_r ? 2u : 1u) * wide, v);
        }
        float q = 1.f;
        if (post) {
            F2 xx = f2(0.f);
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 4; ++i) xx = fma2(raw_pair(x[v], i), raw_pair(x[v], i), xx);
            float sum[1] = {sum_pair(xx)};
            group_sum(sum, buf[0], tpr, group);
            q = root(sum[0], a.inv_cols, a.eps);
        }
        F2 s[V][4], ss = f2(0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[v][i] = mul2(raw_pair(x[v], i), f2(q));
                if (gates) s[v][i] = mul2(s[v][i], raw_pair(g[v], i));
                s[v][i] = fma2(s[v][i], w[v][i], raw_pair(r[v], i));
                ss = fma2(s[v][i], s[v][i], ss);
            }
            if (a.S != nullptr) store(a.S + row * a.lds, s[v], v, in);
        }
        float sum[1] = {sum_pair(ss)};
        if (a.H != nullptr) group_sum(sum, buf[1], tpr, group);
        // The slot has been read into registers that the lines above have used.
        fetch(row + kAhead * turn, slot);
        if (a.H != nullptr) {
            const F2 p = f2(root(sum[0], a.inv_cols, a.eps));
#pragma unroll
            for (int v = 0; v < V; ++v) {
                F2 h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = mul2(mul2(s[v][i], p), wpre[v][i]);
                store(a.H + row * a.ldh, h, v, in);
            }
        }
        if (tpr > 32 && (!post || a.H == nullptr)) __syncthreads();   // buf, for the next row
    }
    copy_async_wait<0>();
}

// Rows that no CTA can hold: a CTA a row, read again for each mean.  A thread has up to 2^20 terms of a sum, each addition
// off by up to 2^-24 of it (4096 equal terms one after another: 2^-15).  So kRun terms are added as they come, and the runs
// with what each addition lost handed on to the next one (Kahan's compensated summation: two roundings for any number).
constexpr int32_t kRun = 16;
struct LongSum {
    float sum = 0.f, lost = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float y = x - lost, t = sum + y;
        lost = fabsf(t) <= FLT_MAX ? (t - sum) - y : 0.f;     // an infinite sum stays one
        sum = t;
    }
};

template <typename F>
__device__ __forceinline__ float sum_in_runs(int32_t cols, F&& at) {
    LongSum total;
    int32_t c = int32_t(threadIdx.x);
    for (; c + (kRun - 1) * 1024 < cols; c += kRun * 1024) {
        float part = 0.f;
#pragma unroll
        for (int32_t i = 0; i < kRun; ++i) {
            const float x = at(c + i * 1024);
            part = fmaf(x, x, part);
        }
        total.add(part);
    }
    float part = 0.f;
    for (; c < cols; c += 1024) {
        const float x = at(c);
        part = fmaf(x, x, part);
    }
    total.add(part);
    return total.sum;
}

template <typename T>
__device__ __forceinline__ float sum_at(const Args<T>& a, int64_t row, float q, int32_t c) {
    float y = to_f32(a.X[row * a.ldx + c]);
    if (a.post != nullptr) y = y * q * a.post[c];
    if (a.G != nullptr) y *= to_f32(a.G[row / a.per_gate * a.ldg + c]);
    if (a.R == nullptr && a.scale == 1.f) return y;
    return fmaf(a.scale, y, a.R != nullptr ? to_f32(a.R[row * a.ldr + c]) : 0.f);
}

template <typename T>
__global__ void __launch_bounds__(1024, 1) residual_norm_long_kernel(const Args<T> a) {
    __shared__ float buf[2][1][32];
    ptx::griddep_wait();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float sum[1], q = 1.f;
        if (a.post != nullptr) {
            sum[0] = sum_in_runs(a.cols, [&](int32_t c) { return to_f32(a.X[row * a.ldx + c]); });
            group_sum(sum, buf[0], 1024, 0);
            q = root(sum[0], a.inv_cols, a.eps);
        }
        float r = 0.f;
        if (a.H != nullptr) {
            sum[0] = sum_in_runs(a.cols, [&](int32_t c) { return sum_at(a, row, q, c); });
            group_sum(sum, buf[1], 1024, 0);
            r = root(sum[0], a.inv_cols, a.eps);
        }
        for (int32_t c = int32_t(threadIdx.x); c < a.cols; c += 1024) {
            const float s = sum_at(a, row, q, c);
            if (a.S != nullptr) from_f32(s, a.S + row * a.lds + c);
            if (a.H != nullptr) from_f32(s * r * a.pre[c], a.H + row * a.ldh + c);
        }
        __syncthreads();                                // buf, for the next row
    }
}

// ------------------------------------------------------------ gradients
template <typename T>
struct GradArgs {
    const T *dS, *dH, *X, *S, *G;
    const float *post, *pre;
    T *dX, *dR, *dG;
    int64_t ldds, lddh, ldx, lds, ldg, lddx, lddr, lddg, ld_odd;      // ld_odd: of the rows, whole aligned pieces left out
    int32_t rows, cols, per_gate;
    float scale, eps, inv_cols;
    // Sums over rows: `items` runs of rows, `segments` of them to a gate; each CTA takes a
    // contiguous share of the items.  part: per CTA [post][pre] rows of cols, or null; gate_part:
    // per item, where a gate has several segments (one segment: dG itself).
    int32_t items, segments, span;     // span: rows of a gate (all rows where the items are one run)
    float *post_part, *pre_part, *gate_part;
    bool want_post, want_pre, want_gate;
    int32_t parts, each;               // rows cut over a cluster's CTAs, columns for each
};

// The rows of a CTA's items, `groups` at a time.
template <typename T>
struct RowWalk {
    int32_t item, last;
    int64_t first, end;                                 // rows of the turn: from `first`, below `end`

    __device__ __forceinline__ void enter(const GradArgs<T>& a) {
        const int64_t base = int64_t(item / a.segments) * a.span, seg = item % a.segments;
        first = base + a.span * seg / a.segments;
        end = base + a.span * (seg + 1) / a.segments;
    }
    // Past rows that are none; false after the last item.
    __device__ __forceinline__ bool settle(const GradArgs<T>& a) {
        while (first >= end) {
            if (++item >= last) return false;
            enter(a);
        }
        return true;
    }
};

// How rows lie: on 16 bytes; starting anywhere, as ODD above; cut over the CTAs of a cluster.
enum Lie : int { kWhole, kOdd, kCut };

// One CTA: its items' rows, blockDim.x / tpr at a time.  Thread t of each group keeps the sums of
// its columns; groups are joined in order through shared memory.  kAhead > 0 (rows on 16 bytes, or ODD as above): that many
// turns' rows of all inputs are on their way into shared memory, each thread its own 16 bytes, so that nobody
// waits for another's copy; 0: they are loaded in their turn, any alignment.
// CUT: rows of more columns than a CTA holds with FULL, a.each for each of a cluster's a.parts CTAs; two exchanges of sums a
// row, about 0.7 us each.
// FULL: a training step's call, with both norms, dS and all of dX, dR, dpost and dpre, without a gate an element.  What
// is there need not be asked then (4096 x 4096: 631 instructions a warp and row of 8 columns a thread if it is, 447 not),
// and the registers are kept for the row: the weights lie in shared memory, each thread's where it alone reads them, and
// dpost's sum in its place in scratch, added to after a gate's rows.
template <typename T, int V, int kAhead, bool FULL, int M>
__global__ void __launch_bounds__(512) residual_norm_grad_kernel(const GradArgs<T> a, int32_t tpr, uint32_t row_bytes,
                                                                 uint32_t step) {
    static_assert(M == kWhole || kAhead > 0);
    constexpr bool ODD = M == kOdd, CUT = M == kCut;
    constexpr int A = kAhead > 0 ? kVec : kStrided;
    __shared__ float buf[2][3][32], slots[2][4][4];
    // The ring; behind it, where groups > 1, [groups][8][tpr] floats.
    extern __shared__ __align__(16) uint8_t ring[];
    ptx::griddep_wait();
    const int32_t t = int32_t(threadIdx.x) % tpr, group = int32_t(threadIdx.x) / tpr;
    const int32_t groups = int32_t(blockDim.x) / tpr;
    const uint32_t parts = CUT ? uint32_t(a.parts) : 1u, rank = CUT ? ptx::cluster_ctarank() : 0u;
    const uint32_t cta = blockIdx.x / parts, ctas = gridDim.x / parts;
    const int32_t i0 = int32_t(int64_t(a.items) * cta / ctas), i1 = int32_t(int64_t(a.items) * (cta + 1) / ctas);
    // ODD: CTA b has rows 8 (b / 8 groups + group) + b % 8 and on, the same number of elements, `off`, behind an aligned
    // address; columns go from there to `all_cols`.
    constexpr int32_t kStep = ODD ? 8 : 1;
    const int64_t odd_row = int64_t(blockIdx.x / 8) * groups * 8 + blockIdx.x % 8;
    const int64_t turn = ODD ? int64_t(gridDim.x) * groups : groups;
    const int32_t off = ODD ? int32_t(odd_row * a.ld_odd % int32_t(16 / sizeof(T))) : 0, c0 = CUT ? int32_t(rank) * a.each : 0;
    const int32_t all_cols = CUT ? min(a.each, a.cols - c0) : a.cols + off;
    auto load = [&](F2 (&x)[4], const auto* from, int v) {
        if constexpr (ODD) load_pairs_from(x, from, v, t, tpr, off, all_cols);
        else load_pairs<std::remove_cv_t<std::remove_pointer_t<decltype(from)>>, A>(x, from + c0, v, t, tpr, all_cols);
    };
    auto store = [&](T* to, const F2 (&x)[4], int v, int32_t cols) {
        if constexpr (ODD) store_pairs_from(to - off, x, v, t, tpr, off, cols);
        else store_pairs<T, A>(to + c0, x, v, t, tpr, cols);
    };
    auto store_sums = [&](auto* to, const F2 (&x)[4], int v) {
        if constexpr (ODD) store_pairs_from(to - off, x, v, t, tpr, off, all_cols, true);
        else store_pairs<std::remove_pointer_t<decltype(to)>, A>(to + c0, x, v, t, tpr, all_cols);
    };
    auto copy = [&](uint32_t to, const T* from, int v) {
        if constexpr (ODD) copy_row8_from(to, from - off, v, t, tpr, all_cols);
        else copy_row8(to, from + c0, v, t, tpr, all_cols);
    };
    auto take = [&](Raw8<T>& x, uint32_t from, int v) {
        take_row8(x, from, v, t, tpr);
        if (ODD && v == 0 && t == 0) clear_front(x, off);
    };
    const bool post = FULL || a.post != nullptr, pre = FULL || a.pre != nullptr, has_x = FULL || a.X != nullptr;
    const bool has_ds = FULL || a.dS != nullptr, want_x = FULL || a.dX != nullptr, want_r = FULL || a.dR != nullptr;
    const bool want_post = FULL || a.want_post, want_pre = FULL || a.want_pre;
    const bool gate_rows = !FULL && a.G != nullptr && a.per_gate == 1;      // a gate an element: dG row by row, nothing to add
    const bool run_gate = a.G != nullptr && !gate_rows;            // one for all rows of an item
    const bool want_run = !gate_rows && (want_post || a.want_gate), weighted = post || a.G != nullptr;
    // Weights, and sums: dpre and dpost over all rows, ds X q over an item's.  dgate and dpost of rows that share a gate
    // are that last sum times what does not change with the row.
    F2 wpost[V][4], wpre[V][4], spost[V][4], spre[V][4], srun[V][4];
    // FULL: this thread's part of the weights, then of gate times weight.
    const uint32_t own = ptx::smem_addr(ring) + kAhead * step + (groups > 1 ? 32u * blockDim.x : 0u) + 16u * threadIdx.x;
    const uint32_t own_gw = own + 32u * V * blockDim.x;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (gate_rows && post) load(wpost[v], a.post, v);
        if (pre) load(wpre[v], a.pre, v);
        if (FULL) put_pairs(own + uint32_t(v) * 32u * blockDim.x, wpre[v]);
#pragma unroll
        for (int i = 0; i < 4; ++i) spost[v][i] = spre[v][i] = srun[v][i] = f2(0.f);
    }
    // Adds the groups' sums in order, a vector at a time; the result is in group 0.
    float* joined = reinterpret_cast<float*>(ring) + kAhead * step / sizeof(float);
    auto join = [&](F2 (&s)[V][4]) {
        if (groups == 1) return;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i)
                split2(s[v][i], joined[(group * 8 + 2 * i) * tpr + t], joined[(group * 8 + 2 * i + 1) * tpr + t]);
            __syncthreads();
            if (group != 0) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                for (int32_t g = 1; g < groups; ++g)
                    s[v][i] = add2(s[v][i], f2(joined[(g * 8 + 2 * i) * tpr + t], joined[(g * 8 + 2 * i + 1) * tpr + t]));
        }
    };
    // The inputs of a row in the ring, in this order: dH and S, X, dS, the gate.
    const uint32_t ring0 = ptx::smem_addr(ring) + uint32_t(group) * row_bytes, at_x = pre ? 2 : 0;
    const uint32_t at_ds = at_x + (has_x ? 1 : 0), at_g = at_ds + (has_ds ? 1 : 0), wide = row_bytes * groups;
    RowWalk<T> ahead = {i0, i1, 0, 0};
    if (ODD) ahead.first = odd_row, ahead.end = a.rows;
    else ahead.enter(a);
    bool more = ahead.settle(a);
    auto fetch = [&](uint32_t slot) {
        const int64_t row = ahead.first + group * kStep;
        if (more && row < ahead.end) {
            const uint32_t to = ring0 + slot * step;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (pre) {
                    copy(to, a.dH + row * a.lddh, v);
                    copy(to + wide, a.S + row * a.lds, v);
                }
                if (has_x) copy(to + at_x * wide, a.X + row * a.ldx, v);
                if (has_ds) copy(to + at_ds * wide, a.dS + row * a.ldds, v);
                if (gate_rows) copy(to + at_g * wide, a.G + row * a.ldg, v);
            }
        }
        copy_async_commit();
        if (more) {
            ahead.first += turn;
            more = ahead.settle(a);
        }
    };
    if (kAhead > 0) clear_past<T, V>(ptx::smem_addr(ring), kAhead * step / row_bytes, row_bytes, t, tpr, all_cols);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(uint32_t(i));
    uint32_t slot = 0;
    int which = 0;
    if (CUT) ptx::cluster_sync_all();                   // the others' slots are there
    for (int32_t item = i0; item < i1; ++item) {
        const int32_t g = item / a.segments, seg = item % a.segments;
        const int64_t base = int64_t(g) * a.span;
        const int64_t r0 = ODD ? odd_row : base + int64_t(a.span) * seg / a.segments;
        const int64_t r1 = ODD ? a.rows : base + int64_t(a.span) * (seg + 1) / a.segments;
        const T* gate = run_gate ? a.G + g * a.ldg : nullptr;
        F2 gw[V][4];                                    // gate times weight
        if (!gate_rows && weighted)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                F2 w[4];
                if (post) load(gw[v], a.post, v);
                if (run_gate) load(w, gate, v);
#pragma unroll
                for (int i = 0; i < 4; ++i) gw[v][i] = !run_gate ? gw[v][i] : post ? mul2(gw[v][i], w[i]) : w[i];
                if (FULL) put_pairs(own_gw + uint32_t(v) * 32u * blockDim.x, gw[v]);
            }
        for (int64_t first = r0; first < r1; first += turn) {
            const int64_t row = first + group * kStep;
            const bool in = row < r1;
            const int32_t cols = in ? all_cols : 0;
            Raw8<T> x[V] = {}, s[V] = {}, dh[V] = {}, ds[V] = {}, gt[V] = {};
            if (kAhead > 0) {
                copy_async_wait<(kAhead > 0 ? kAhead : 1) - 1>();
                const uint32_t from = ring0 + slot * step;
                if (in)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        if (pre) {
                            take(dh[v], from, v);
                            take(s[v], from + wide, v);
                        }
                        if (has_x) take(x[v], from + at_x * wide, v);
                        if (has_ds) take(ds[v], from + at_ds * wide, v);
                        if (gate_rows) take(gt[v], from + at_g * wide, v);
                    }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (has_x) load_raw8<A>(x[v], a.X + row * a.ldx, v, t, tpr, cols);
                    if (pre) {
                        load_raw8<A>(s[v], a.S + row * a.lds, v, t, tpr, cols);
                        load_raw8<A>(dh[v], a.dH + row * a.lddh, v, t, tpr, cols);
                    }
                    if (has_ds) load_raw8<A>(ds[v], a.dS + row * a.ldds, v, t, tpr, cols);
                    if (gate_rows) load_raw8<A>(gt[v], a.G + row * a.ldg, v, t, tpr, cols);
                }
            }
            F2 ss = f2(0.f), us = f2(0.f), xx = f2(0.f);
            if (pre)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (FULL) get_pairs(wpre[v], own + uint32_t(v) * 32u * blockDim.x);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const F2 S = raw_pair(s[v], i);
                        ss = fma2(S, S, ss);
                        us = fma2(mul2(raw_pair(dh[v], i), wpre[v][i]), S, us);
                    }
                }
            if (post)
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const F2 X = raw_pair(x[v], i);
                        xx = fma2(X, X, xx);
                    }
            float sum[3] = {sum_pair(ss), sum_pair(us), sum_pair(xx)};
            if (pre || post) group_sum(sum, buf[0], tpr, group);
            if (CUT) cluster_sum(sum, slots[which], parts, rank), which ^= 1;
            // A group without a row adds zeros.
            const float r = in ? root(sum[0], a.inv_cols, a.eps) : 0.f, rm = r * (r * sum[1] * a.inv_cols);
            const float q = !post ? 1.f : in ? root(sum[2], a.inv_cols, a.eps) : 0.f;
            F2 d[V][4], dot = f2(0.f);
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 4; ++i) d[v][i] = raw_pair(ds[v], i);
            if (pre) {
                const F2 r2 = f2(r), m2 = f2(-rm);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (FULL) get_pairs(wpre[v], own + uint32_t(v) * 32u * blockDim.x);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const F2 S = raw_pair(s[v], i), H = raw_pair(dh[v], i);
                        const F2 n = mul2(S, r2);
                        d[v][i] = fma2(n, m2, fma2(r2, mul2(H, wpre[v][i]), d[v][i]));
                        spre[v][i] = fma2(H, n, spre[v][i]);
                    }
                }
            }
            if (want_r)
#pragma unroll
                for (int v = 0; v < V; ++v) store(a.dR + row * a.lddr, d[v], v, cols);
            const F2 q2 = f2(q);
            if (gate_rows) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    F2 dg[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const F2 X = raw_pair(x[v], i), n = mul2(X, q2), y = post ? mul2(n, wpost[v][i]) : n;
                        dg[i] = mul2(mul2(f2(a.scale), d[v][i]), y);
                        d[v][i] = mul2(d[v][i], raw_pair(gt[v], i));
                        if (post) {
                            spost[v][i] = fma2(mul2(f2(a.scale), d[v][i]), n, spost[v][i]);
                            d[v][i] = mul2(d[v][i], wpost[v][i]);
                            dot = fma2(d[v][i], X, dot);
                        }
                    }
                    if (a.want_gate) store(a.dG + row * a.lddg, dg, v, cols);
                }
            } else if (weighted) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (FULL) get_pairs(gw[v], own_gw + uint32_t(v) * 32u * blockDim.x);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const F2 X = raw_pair(x[v], i);
                        if (want_run) srun[v][i] = fma2(d[v][i], mul2(X, q2), srun[v][i]);
                        d[v][i] = mul2(d[v][i], gw[v][i]);
                        dot = fma2(d[v][i], X, dot);
                    }
                }
            }
            // The slot has been read into registers that the lines above have used.
            if (kAhead > 0) {
                fetch(slot);
                slot = slot + 1 == uint32_t(kAhead) ? 0 : slot + 1;
            }
            if (want_x) {
                F2 m2 = f2(0.f);
                if (post) {
                    float sums[1] = {sum_pair(dot)};
                    group_sum(sums, buf[1], tpr, group);
                    if (CUT) cluster_sum(sums, slots[which], parts, rank), which ^= 1;
                    m2 = f2(-q * (q * sums[0] * a.inv_cols));
                }
                const F2 k2 = f2(a.scale * q);
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (post) d[v][i] = fma2(raw_pair(x[v], i), m2, d[v][i]);
                        d[v][i] = mul2(d[v][i], k2);
                    }
                    store(a.dX + row * a.lddx, d[v], v, cols);
                }
            }
            if (tpr > 32 && (!want_x || !post)) __syncthreads();   // buf[0], for the next rows
        }
        if (want_run) {
            // dpost gains scale gate sum, dgate is scale weight sum.
            if (FULL) join(srun);
            if (want_post && (!FULL || group == 0))
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    F2 w[4];
                    float* sum = a.post_part + int64_t(cta) * a.cols;
                    if (run_gate) load(w, gate, v);
                    if (FULL && item > i0) load(spost[v], sum, v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const F2 k = run_gate ? mul2(f2(a.scale), w[i]) : f2(a.scale);
                        spost[v][i] = fma2(srun[v][i], k, spost[v][i]);
                    }
                    if (FULL) {
                        store_sums(sum, spost[v], v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) spost[v][i] = f2(0.f);
                    }
                }
            if (a.want_gate) {
                if (!FULL) join(srun);
                if (group == 0)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        F2 w[4];
                        if (post) load(w, a.post, v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            srun[v][i] = mul2(srun[v][i], f2(a.scale));
                            if (post) srun[v][i] = mul2(srun[v][i], w[i]);
                        }
                        if (a.segments > 1)
                            store_sums(a.gate_part + int64_t(item) * a.cols, srun[v], v);
                        else
                            store_sums(a.dG + g * a.lddg, srun[v], v);
                    }
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 4; ++i) srun[v][i] = f2(0.f);
        }
    }
    if (kAhead > 0) copy_async_wait<0>();
    if (want_post && !FULL) {
        join(spost);
        if (group == 0)
#pragma unroll
            for (int v = 0; v < V; ++v)
                store_sums(a.post_part + int64_t(cta) * a.cols, spost[v], v);
    }
    if (want_pre) {
        join(spre);
        if (group == 0)
#pragma unroll
            for (int v = 0; v < V; ++v)
                store_sums(a.pre_part + int64_t(cta) * a.cols, spre[v], v);
    }
    if (CUT) ptx::cluster_sync_all();                   // no CTA leaves while another writes its slots
}

// Rows that no CTA holds with what goes with them: their means first (a CTA a row), then everything else column by
// column, 8 of them a thread.
constexpr int kLongThreads = 256;

// stats[row] = {r, r^2 mean(u S), q, q^2 mean(v X)}.  Sums as in the forward pass's long rows, in runs
// of four pieces (16 terms).
constexpr int32_t kRunPieces = 4;
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024, 1) residual_norm_stats_kernel(const GradArgs<T> a, float4* stats) {
    __shared__ float buf[2][3][32];
    ptx::griddep_wait();
    const bool pre = a.pre != nullptr, post = a.post != nullptr;
    const int32_t t = int32_t(threadIdx.x), pieces = (a.cols + 8191) / 8192;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        LongSum all_ss, all_us, all_xx, all_vx;
        for (int32_t p0 = 0; p0 < pieces; p0 += kRunPieces) {
            F2 ss = f2(0.f), us = f2(0.f), xx = f2(0.f);
#pragma unroll
            for (int32_t p = p0; p < p0 + kRunPieces; ++p) {
                if (p >= pieces) break;
                Raw8<T> s, dh, x;
                F2 w[4];
                if (pre) {
                    load_raw8<VEC>(s, a.S + row * a.lds, p, t, 1024, a.cols);
                    load_raw8<VEC>(dh, a.dH + row * a.lddh, p, t, 1024, a.cols);
                    load_pairs<float, VEC>(w, a.pre, p, t, 1024, a.cols);
                }
                if (post) load_raw8<VEC>(x, a.X + row * a.ldx, p, t, 1024, a.cols);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (pre) {
                        ss = fma2(raw_pair(s, i), raw_pair(s, i), ss);
                        us = fma2(mul2(raw_pair(dh, i), w[i]), raw_pair(s, i), us);
                    }
                    if (post) xx = fma2(raw_pair(x, i), raw_pair(x, i), xx);
                }
            }
            all_ss.add(sum_pair(ss)), all_us.add(sum_pair(us)), all_xx.add(sum_pair(xx));
        }
        float sum[3] = {all_ss.sum, all_us.sum, all_xx.sum};
        group_sum(sum, buf[0], 1024, 0);
        const float r = root(sum[0], a.inv_cols, a.eps), rm = r * (r * sum[1] * a.inv_cols);
        const float q = post ? root(sum[2], a.inv_cols, a.eps) : 1.f;
        if (post)
            for (int32_t p0 = 0; p0 < pieces; p0 += kRunPieces) {
                F2 vx = f2(0.f);
#pragma unroll
                for (int32_t p = p0; p < p0 + kRunPieces; ++p) {
                    if (p >= pieces) break;
                    Raw8<T> s, dh, x, ds = {}, g;
                    F2 w[4], wp[4];
                    if (pre) {
                        load_raw8<VEC>(s, a.S + row * a.lds, p, t, 1024, a.cols);
                        load_raw8<VEC>(dh, a.dH + row * a.lddh, p, t, 1024, a.cols);
                        load_pairs<float, VEC>(w, a.pre, p, t, 1024, a.cols);
                    }
                    load_raw8<VEC>(x, a.X + row * a.ldx, p, t, 1024, a.cols);
                    load_pairs<float, VEC>(wp, a.post, p, t, 1024, a.cols);
                    if (a.dS != nullptr) load_raw8<VEC>(ds, a.dS + row * a.ldds, p, t, 1024, a.cols);
                    if (a.G != nullptr) load_raw8<VEC>(g, a.G + row / a.per_gate * a.ldg, p, t, 1024, a.cols);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        F2 e = raw_pair(ds, i);
                        if (pre) e = fma2(f2(r), fma2(raw_pair(s, i), f2(-rm), mul2(raw_pair(dh, i), w[i])), e);
                        if (a.G != nullptr) e = mul2(e, raw_pair(g, i));
                        vx = fma2(mul2(e, wp[i]), raw_pair(x, i), vx);
                    }
                }
                all_vx.add(sum_pair(vx));
            }
        float dot[1] = {all_vx.sum};
        group_sum(dot, buf[1], 1024, 0);
        if (threadIdx.x == 0) stats[row] = make_float4(r, rm, q, a.scale * (q * (q * dot[0] * a.inv_cols)));
    }
}

// blockIdx.x: the columns; blockIdx.y: the share of the items.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kLongThreads, 2) residual_norm_grad_long_kernel(const GradArgs<T> a, const float4* stats) {
    ptx::griddep_wait();
    // Eight columns of the CTA's 2048 a thread.
    const int32_t c0 = int32_t(blockIdx.x) * kLongThreads * 8, t = int32_t(threadIdx.x), tpr = kLongThreads, cols = a.cols - c0;
    const int32_t i0 = int32_t(int64_t(a.items) * blockIdx.y / gridDim.y);
    const int32_t i1 = int32_t(int64_t(a.items) * (blockIdx.y + 1) / gridDim.y);
    const bool pre = a.pre != nullptr, post = a.post != nullptr, gate_rows = a.G != nullptr && a.per_gate == 1;
    const bool run_gate = a.G != nullptr && !gate_rows;
    F2 wpost[4], wpre[4], spost[4], spre[4];
    if (post) load_pairs<float, VEC>(wpost, a.post + c0, 0, t, tpr, cols);
    if (pre) load_pairs<float, VEC>(wpre, a.pre + c0, 0, t, tpr, cols);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        spost[i] = spre[i] = f2(0.f);
        if (!post) wpost[i] = f2(1.f);
    }
    for (int32_t item = i0; item < i1; ++item) {
        const int32_t g = item / a.segments, seg = item % a.segments;
        const int64_t base = int64_t(g) * a.span;
        const int64_t r0 = base + int64_t(a.span) * seg / a.segments, r1 = base + int64_t(a.span) * (seg + 1) / a.segments;
        F2 srun[4], gate[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) srun[i] = f2(0.f), gate[i] = f2(1.f);
        if (run_gate) load_pairs<T, VEC>(gate, a.G + g * a.ldg + c0, 0, t, tpr, cols);
#pragma unroll 2
        for (int64_t row = r0; row < r1; ++row) {
            const float4 st = stats[row];
            Raw8<T> s, dh, x = {}, ds = {};
            if (pre) {
                load_raw8<VEC>(s, a.S + row * a.lds + c0, 0, t, tpr, cols);
                load_raw8<VEC>(dh, a.dH + row * a.lddh + c0, 0, t, tpr, cols);
            }
            if (a.X != nullptr) load_raw8<VEC>(x, a.X + row * a.ldx + c0, 0, t, tpr, cols);
            if (a.dS != nullptr) load_raw8<VEC>(ds, a.dS + row * a.ldds + c0, 0, t, tpr, cols);
            if (gate_rows) load_pairs<T, VEC>(gate, a.G + row * a.ldg + c0, 0, t, tpr, cols);
            F2 e[4], dg[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e[i] = raw_pair(ds, i);
                if (pre) {
                    const F2 S = raw_pair(s, i), H = raw_pair(dh, i);
                    e[i] = fma2(f2(st.x), fma2(S, f2(-st.y), mul2(H, wpre[i])), e[i]);
                    spre[i] = fma2(H, mul2(S, f2(st.x)), spre[i]);
                }
            }
            if (a.dR != nullptr) store_pairs<T, VEC>(a.dR + row * a.lddr + c0, e, 0, t, tpr, cols);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F2 X = raw_pair(x, i), n = mul2(X, f2(st.z));
                e[i] = mul2(e[i], f2(a.scale));
                dg[i] = mul2(e[i], mul2(n, wpost[i]));
                srun[i] = add2(srun[i], dg[i]);
                e[i] = mul2(e[i], gate[i]);
                spost[i] = fma2(e[i], n, spost[i]);
                e[i] = mul2(e[i], wpost[i]);
                if (post) e[i] = fma2(X, f2(-st.w), e[i]);
                e[i] = mul2(e[i], f2(st.z));
            }
            if (a.want_gate && gate_rows) store_pairs<T, VEC>(a.dG + row * a.lddg + c0, dg, 0, t, tpr, cols);
            if (a.dX != nullptr) store_pairs<T, VEC>(a.dX + row * a.lddx + c0, e, 0, t, tpr, cols);
        }
        if (a.want_gate && !gate_rows) {
            if (a.segments > 1)
                store_pairs<float, VEC>(a.gate_part + int64_t(item) * a.cols + c0, srun, 0, t, tpr, cols);
            else
                store_pairs<T, VEC>(a.dG + g * a.lddg + c0, srun, 0, t, tpr, cols);
        }
    }
    if (a.want_post) store_pairs<float, VEC>(a.post_part + int64_t(blockIdx.y) * a.cols + c0, spost, 0, t, tpr, cols);
    if (a.want_pre) store_pairs<float, VEC>(a.pre_part + int64_t(blockIdx.y) * a.cols + c0, spre, 0, t, tpr, cols);
}

// Sums of runs of `count` rows of a [runs * count, cols] fp32 matrix, 32 columns a CTA: the rows dealt to
// 16 warps, then the warps' sums added in order.  blockIdx.y: which of the up to three outputs' runs.
struct PartSums {
    struct Of {
        const float* in;
        void* out;
        int64_t ldo;
        int32_t runs, count;
        bool bf16;
    } of[3];
    int32_t n, cols;
};

__global__ void __launch_bounds__(512) norm_sums_kernel(const __grid_constant__ PartSums p) {
    __shared__ float part[16][32];
    ptx::griddep_wait();
    int32_t run = int32_t(blockIdx.y), i = 0;
    while (i + 1 < p.n && run >= p.of[i].runs) run -= p.of[i++].runs;
    const PartSums::Of& o = p.of[i];
    const int32_t lane = int32_t(threadIdx.x) % 32, warp = int32_t(threadIdx.x) / 32, count = o.count;
    const int32_t c = int32_t(blockIdx.x) * 32 + lane;
    const float* in = o.in + int64_t(run) * count * p.cols + c;
    float s = 0.f;
    if (c < p.cols)
#pragma unroll 10
        for (int32_t k = warp; k < count; k += 16) s += in[int64_t(k) * p.cols];
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || c >= p.cols) return;
#pragma unroll
    for (int w = 1; w < 16; ++w) s += part[w][lane];
    if (o.bf16)
        static_cast<__nv_bfloat16*>(o.out)[run * o.ldo + c] = __float2bfloat16_rn(s);
    else
        static_cast<float*>(o.out)[run * o.ldo + c] = s;
}

// ------------------------------------------------------------ launches
// Rows on 16 bytes; a single row's pitch does not matter.
template <typename T>
bool aligned16(const void* p, int64_t ld, int64_t rows) {
    return p == nullptr ||
           (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld % int64_t(16 / sizeof(T)) == 0));
}

// Rows of all the matrices start alike, seen from the aligned address in front of them: each *ld_odd elements on from the last,
// but for whole pieces of 16 bytes.
template <typename T, int N>
bool start_alike(const Mat* const (&mats)[N], int64_t* ld_odd) {
    constexpr int64_t kPiece = 16 / sizeof(T);
    int64_t ld = -1;
    for (const Mat* m : mats) {
        if (m->p == nullptr) continue;
        if (reinterpret_cast<uintptr_t>(m->p) % 16 != 0 || (ld >= 0 && m->ld % kPiece != ld)) return false;
        ld = m->ld % kPiece;
    }
    *ld_odd = ld;
    return true;
}

// Threads a row that hold it with V vectors each: a power of two below a warp, else as many warps as it takes (a row a CTA,
// us, against powers of two of warps: 700 x 5120 bf16 9.7 / 15.3, 4096 x 8200 92 / 109).
int threads_for(int64_t cols, int V) {
    if (cols > 32 * 8 * V) return int(cdiv(cols, 32 * 8 * V)) * 32;
    int tpr = 4;
    while (int64_t(tpr) * 8 * V < cols) tpr *= 2;
    return tpr;
}

template <typename T, int V>
void* forward_kernel(bool vec) {
    return vec ? reinterpret_cast<void*>(&residual_norm_kernel<T, V, true>)
               : reinterpret_cast<void*>(&residual_norm_kernel<T, V, false>);
}

template <typename T, int kAhead, int kMost>
void* stream_kernel(bool odd) {
    return odd ? reinterpret_cast<void*>(&residual_norm_stream_kernel<T, 2, kAhead, kMost, true>)
               : reinterpret_cast<void*>(&residual_norm_stream_kernel<T, 2, kAhead, kMost, false>);
}

struct StreamPlan {
    int32_t tpr;
    int threads, ctas, ahead;                           // ctas: an SM
    size_t step;
};
// `cols`: with what may lie between an aligned address and a row.
// An SM's registers hold 640 threads (bf16; up to 102 registers a thread), 512 (fp32).  Against warps in powers of two and
// at most two CTAs, us, bf16: 8192 x 5120 53 / 76, 16384 x 2560 55 / 70, 16384 x 1536 34 / 39.
StreamPlan stream_plan(const ResidualNormArgs& s, int32_t cols, size_t esize) {
    StreamPlan p;
    const int inputs = 1 + (s.R.p ? 1 : 0) + (s.G.p && s.gates > 1 ? 1 : 0), most = esize == 2 ? 640 : 512;
    p.tpr = threads_for(cols, 2);
    p.threads = std::max(1, 256 / p.tpr) * p.tpr, p.ctas = most / p.threads;
    p.step = size_t(p.threads) * 16 * esize * size_t(inputs);
    p.ahead = p.ctas == 1 && 3 * p.step <= 216 * 1024 ? 3 : 2;
    return p;
}
// Rows of up to 8192 columns, and enough of them for CTAs that stay: eight turns of all.
bool streams(const ResidualNormArgs& s, int32_t cols, size_t esize, int sm_count) {
    if (cols > 8192) return false;
    const StreamPlan p = stream_plan(s, cols, esize);
    return s.rows >= int64_t(8) * sm_count * (p.threads / p.tpr) && size_t(p.ahead) * p.step <= 216 * 1024;
}

template <typename T>
int run_forward(const ResidualNormArgs& s, const LibCtx& c, cudaStream_t stream) {
    Args<T> a = {static_cast<const T*>(s.X.p), static_cast<const T*>(s.R.p), static_cast<const T*>(s.G.p), s.post, s.pre,
                 static_cast<T*>(s.S.w()), static_cast<T*>(s.H.w()), s.X.ld, s.R.ld, s.G.ld, s.S.ld, s.H.ld, 0,
                 s.rows, s.cols, s.per_gate, s.scale, s.eps, float(1.0 / double(s.cols))};
    bool vec = s.cols % 8 == 0 && aligned16<float>(s.post, 0, 1) && aligned16<float>(s.pre, 0, 1) &&
               aligned16<T>(s.G.p, s.G.ld, s.gates);
    for (const Mat* m : {&s.X, &s.R, &s.S, &s.H}) vec = vec && aligned16<T>(m->p, m->ld, s.rows);
    // Rows that start anywhere can be streamed where those of all operands start alike, as contiguous tensors' do: us, bf16,
    // 16384 rows, strided / streamed: 4095 columns 264 / 109, 3001 244 / 76, 1001 64 / 31.
    const Mat none = {};
    const bool runs = s.G.p && s.gates > 1 && s.gates < s.rows;
    const bool odd = !vec && !runs && start_alike<T>({&s.X, &s.R, &s.S, &s.H, s.gates > 1 ? &s.G : &none}, &a.ld_odd);
    constexpr int32_t kPiece = 16 / sizeof(T);
    const int32_t wide = odd && a.ld_odd != 0 ? s.cols + kPiece - 1 : s.cols;
    cudaError_t e;
    if (s.cols > 1024 * 32) {
        void* args[] = {&a};
        e = launch_kernel(reinterpret_cast<void*>(&residual_norm_long_kernel<T>),
                          dim3(unsigned(std::min<int64_t>(s.rows, 2 * c.sm_count))), 1024, 0, 1, args, stream);
    } else if ((vec || odd) && streams(s, wide, sizeof(T), c.sm_count)) {
        const StreamPlan p = stream_plan(s, wide, sizeof(T));
        int32_t tpr = p.tpr;
        uint32_t row_bytes = uint32_t(p.tpr * 16 * sizeof(T)), step = uint32_t(p.step);
        void* kernel = p.ctas > 1     ? stream_kernel<T, 2, sizeof(T) == 2 ? 320 : 256>(odd)
                       : p.ahead == 3 ? stream_kernel<T, 3, 512>(odd)
                                      : stream_kernel<T, 2, 512>(odd);
        const size_t smem = size_t(p.ahead) * p.step;
        const int r = raise_kernel_smem(kernel, smem, c.device);
        if (r != GBR_OK) return r;
        void* args[] = {&a, &tpr, &row_bytes, &step};
        int64_t grid = c.sm_count * std::min<int64_t>(p.ctas, 216 * 1024 / smem);
        if (odd) grid = std::max<int64_t>(8, grid / 8 * 8);     // eight CTAs' rows start in eight ways
        e = launch_kernel(kernel, dim3(unsigned(grid)), p.threads, smem, 1, args, stream);
    } else {
        const int V = s.cols > 1024 * 16 ? 4 : s.cols > 1024 * 8 ? 2 : 1;
        int32_t tpr = threads_for(s.cols, V);
        const int threads = std::max(1, 256 / tpr) * tpr;
        void* kernel = V == 4 ? forward_kernel<T, 4>(vec) : V == 2 ? forward_kernel<T, 2>(vec) : forward_kernel<T, 1>(vec);
        void* args[] = {&a, &tpr};
        e = launch_kernel(kernel, dim3(unsigned(cdiv(s.rows, threads / tpr))), threads, 0, 1, args, stream);
    }
    if (e != cudaSuccess) return report_cuda(e, "launching residual_norm");
    count_launch();
    return GBR_OK;
}

// Columns for each of `parts` CTAs, and the clusters of them that fit at once, a CTA an SM (of fours, 144 of 152 SMs' worth).
int32_t part_cols(int64_t cols, int parts) { return int32_t(cdiv(cdiv(cols, parts), 8) * 8); }
int64_t clusters_for(int parts, int sms) { return parts == 4 ? sms * 18 / 19 / 4 : sms / parts; }

template <typename T, int V>
void* grad_kernel(int ahead, bool full, bool odd) {
    if (odd) return full ? reinterpret_cast<void*>(&residual_norm_grad_kernel<T, V, 2, true, kOdd>)
                         : reinterpret_cast<void*>(&residual_norm_grad_kernel<T, 1, 2, false, kOdd>);
    switch (ahead) {
        case 3: return full ? reinterpret_cast<void*>(&residual_norm_grad_kernel<T, V, 3, true, kWhole>)
                            : reinterpret_cast<void*>(&residual_norm_grad_kernel<T, 1, 3, false, kWhole>);
        case 2: return full ? reinterpret_cast<void*>(&residual_norm_grad_kernel<T, V, 2, true, kWhole>)
                            : reinterpret_cast<void*>(&residual_norm_grad_kernel<T, 1, 2, false, kWhole>);
        default: return reinterpret_cast<void*>(&residual_norm_grad_kernel<T, 1, 0, false, kWhole>);
    }
}

// Cuts the rows into items and the items into at most `ctas` shares: without a gate that several
// rows share one run of equal pieces; else so many segments a gate that the largest share is the
// smallest (an item's sums cost about as much as two rows).
template <typename T>
int64_t cut_rows(GradArgs<T>* a, int32_t gates, int64_t ctas, int32_t groups) {
    const int64_t turns = cdiv(a->rows, groups);
    if (gates == 0 || a->per_gate == 1) {
        a->items = a->segments = int32_t(std::max<int64_t>(1, std::min(turns, ctas)));
        a->span = a->rows;
        return a->items;
    }
    a->span = a->per_gate;
    int64_t best = INT64_MAX;
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(a->per_gate, 4 * ctas / gates));
    for (int64_t s = 1; s <= most; ++s) {
        const int64_t cost = cdiv(gates * s, ctas) * (cdiv(cdiv(a->per_gate, s), groups) + 2);
        if (cost < best) best = cost, a->segments = int32_t(s);
    }
    a->items = gates * a->segments;
    return std::min<int64_t>(a->items, ctas);
}

int launch_sums(PartSums sums, int32_t runs, cudaStream_t stream) {
    void* args[] = {&sums};
    const cudaError_t e = launch_kernel(reinterpret_cast<void*>(&norm_sums_kernel),
                                        dim3(unsigned(cdiv(sums.cols, 32)), unsigned(runs)), 512, 0, 1, args, stream);
    if (e != cudaSuccess) return report_cuda(e, "launching the sums of residual_norm_backward");
    count_launch();
    return GBR_OK;
}

// Sums over no rows: zeros, whatever weights and gates hold (factors that the kernels above apply to sums).
int no_rows(const ResidualNormGradArgs& s, cudaStream_t stream) {
    constexpr int64_t kGates = 65533;                   // of a launch, whose grid has 65535 runs at most
    for (int64_t first = 0; first == 0 || first < s.gates; first += kGates) {
        PartSums sums = {};
        sums.cols = s.cols;
        int32_t runs = 0;
        if (first == 0)
            for (float* out : {s.dpost, s.dpre})
                if (out != nullptr) sums.of[sums.n++] = {nullptr, out, 0, 1, 0, false}, ++runs;
        const int32_t n = s.dG.p ? int32_t(std::min<int64_t>(kGates, s.gates - first)) : 0;
        if (n > 0) {
            uint8_t* out = static_cast<uint8_t*>(s.dG.w()) + first * s.dG.ld * (s.bf16 ? 2 : 4);
            sums.of[sums.n++] = {nullptr, out, s.dG.ld, n, 0, s.bf16}, runs += n;
        }
        const int r = runs > 0 ? launch_sums(sums, runs, stream) : GBR_OK;
        if (r != GBR_OK) return r;
    }
    return GBR_OK;
}

template <typename T>
int run_backward(const ResidualNormGradArgs& s, const LibCtx& c, cudaStream_t stream) {
    GradArgs<T> a = {};
    a.dS = static_cast<const T*>(s.dS.p), a.dH = static_cast<const T*>(s.dH.p), a.X = static_cast<const T*>(s.X.p);
    a.S = static_cast<const T*>(s.S.p), a.G = static_cast<const T*>(s.G.p);
    a.post = s.post, a.pre = s.pre;
    a.dX = static_cast<T*>(s.dX.w()), a.dR = static_cast<T*>(s.dR.w()), a.dG = static_cast<T*>(s.dG.w());
    a.ldds = s.dS.ld, a.lddh = s.dH.ld, a.ldx = s.X.ld, a.lds = s.S.ld, a.ldg = s.G.ld;
    a.lddx = s.dX.ld, a.lddr = s.dR.ld, a.lddg = s.dG.ld;
    a.rows = s.rows, a.cols = s.cols, a.per_gate = s.per_gate;
    a.scale = s.scale, a.eps = s.eps, a.inv_cols = float(1.0 / double(s.cols));
    a.want_post = s.dpost != nullptr, a.want_pre = s.dpre != nullptr, a.want_gate = s.dG.p != nullptr && s.gates > 0;
    bool vec = s.cols % 8 == 0 && aligned16<T>(s.G.p, s.G.ld, s.gates) && aligned16<T>(s.dG.p, s.dG.ld, s.gates);
    for (const Mat* m : {&s.dS, &s.dH, &s.X, &s.S, &s.dX, &s.dR}) vec = vec && aligned16<T>(m->p, m->ld, s.rows);
    for (const float* w : {s.post, s.pre, static_cast<const float*>(s.dpost), static_cast<const float*>(s.dpre)})
        vec = vec && aligned16<float>(w, 0, 1);
    const bool gate_rows = s.G.p && s.per_gate == 1;
    // Rows that start anywhere, as in the forward pass, if there is one for each SM: us, bf16, strided / streamed: 4096 x 4001
    // 160 / 61, 4096 x 1001 46 / 27, 301 x 1001 13.6 / 11.9, but 37 x 4001 11.8 / 13.6.
    constexpr int32_t kPiece = 16 / sizeof(T);
    const Mat none = {}, &g = gate_rows ? s.G : none, &dg = gate_rows ? s.dG : none;
    const bool odd = !vec && s.rows >= c.sm_count && (s.gates <= 1 || gate_rows) &&
                     start_alike<T>({&s.dS, &s.dH, &s.X, &s.S, &s.dX, &s.dR, &g, &dg}, &a.ld_odd);
    int32_t wide = odd && a.ld_odd != 0 ? s.cols + kPiece - 1 : s.cols;
    const bool full = (vec || odd) && s.post && s.pre && s.dS.p && s.dX.p && s.dR.p && a.want_post && a.want_pre && !gate_rows;
    const int inputs = (s.pre ? 2 : 0) + (s.X.p ? 1 : 0) + (s.dS.p ? 1 : 0) + (gate_rows ? 1 : 0);
    // V vectors a thread.  Two where the rows go round (the fewer warps a row, the less of what is done once a warp) and
    // two turns of them fit; rows that do not fit at all have their means taken first (as rows of fp32 of 8192 columns).
    struct Plan {
        int V, threads, groups, ctas, ahead;
        int32_t tpr;
        size_t step, join;
    } plan = {};
    auto lay_out = [&](int V, int most_ctas = 16) {
        plan.V = V, plan.tpr = std::max(32, threads_for(wide, V));
        plan.groups = std::max(1, 256 / plan.tpr), plan.threads = plan.groups * plan.tpr;
        // An SM: 128 registers a thread.  Against warps in powers of two, at most two CTAs, us, bf16: 4096 x 5120 61 / 71,
        // 4096 x 2560 33 / 40.
        plan.ctas = std::min(most_ctas, std::max(1, 512 / plan.threads));
        const size_t mine = size_t(plan.threads) * 8 * sizeof(float);
        plan.join = (plan.groups > 1 ? mine : 0) + (full ? 2 * mine * V : 0);
        plan.step = vec || odd ? size_t(plan.threads) * 8 * V * sizeof(T) * size_t(inputs) : 0;
        const size_t most = size_t(220 / plan.ctas) * 1024 - plan.join;
        plan.ahead = !vec && !odd ? 0 : !odd && 3 * plan.step <= most ? 3 : 2 * plan.step <= most ? 2 : 0;
    };
    const bool many = s.rows >= int64_t(c.sm_count) * 8 * std::max(1, 4096 / s.cols);
    if (wide <= 8192) lay_out(full && (many || wide > 4096) ? 2 : 1);
    if (plan.V == 2 && plan.ahead == 0 && wide <= 4096) lay_out(1);
    bool long_rows = wide > 8192 || plan.tpr > 512 || (plan.V == 2 && plan.ahead == 0);
    // FULL: such rows are cut over two or four CTAs, if their ring fits, and read once then: us, means taken first / cut, 4096 x
    // 16384 bf16 349 / 235, 2048 x 8192 fp32 223 / 136, 400 x 11008 fp32 80 / 48, 5 x 8344 bf16 11.7 / 11.9.  (Forwards, where
    // rows of 16384 columns fit on a CTA, it loses: 4096 x 16384 131 / 152.)
    a.parts = 1;
    for (int parts = 2; parts <= 4 && long_rows && vec && full; parts *= 2) {
        a.each = part_cols(s.cols, parts);
        if (a.each > 8192) continue;
        wide = a.each;
        lay_out(2, 1);
        if (plan.ahead > 0 && plan.groups == 1) a.parts = parts, plan.ahead = 2, long_rows = false;
    }
    const int64_t col_ctas = cdiv(s.cols, kLongThreads * 8);
    // One CTA (or cluster) takes two turns of rows by itself, one without a ring, and writes its sums as they are wanted: us,
    // bf16, two kernels / one, 1 x 2048 6.2 / 4.4, 2 x 2048 6.2 / 5.2, 3 x 2048 6.2 / 6.2; element by element 3 x 2047 8.6 / 13.
    const int64_t turns = s.gates > 1 && !gate_rows ? s.gates * cdiv(s.per_gate, plan.groups) : cdiv(s.rows, plan.groups);
    const bool few = !long_rows && turns <= (plan.ahead > 0 ? 2 : 1);
    const int64_t ctas = few ? 1 : a.parts > 1 ? clusters_for(a.parts, c.sm_count) : long_rows ? std::max<int64_t>(1, 4 * c.sm_count / col_ctas)
                                   : c.sm_count * plan.ctas;
    const bool stream_odd = odd && !long_rows && plan.ahead > 0;
    int64_t grid;
    if (stream_odd) {                                   // eight CTAs' rows start in eight ways
        grid = std::max<int64_t>(8, std::min(ctas, cdiv(s.rows, plan.groups) + 7) / 8 * 8);
        a.items = a.segments = int32_t(grid), a.span = s.rows;
    } else {
        grid = cut_rows(&a, s.gates, ctas, long_rows ? 1 : plan.groups);
    }
    // Scratch of the sums over rows and of the rows' statistics, in one block.
    PartSums sums = {};
    sums.cols = s.cols;
    int32_t runs = 0;
    size_t floats = 0;
    auto part = [&](bool want, int64_t n, int64_t count, void* out, int64_t ldo, bool bf16) -> int {
        if (!want) return -1;
        sums.of[sums.n] = {reinterpret_cast<const float*>(floats), out, ldo, int32_t(n), int32_t(count), bf16};
        floats += (size_t(n * count) * size_t(s.cols) + 3) / 4 * 4;
        runs += int32_t(n);
        return sums.n++;
    };
    const bool direct = grid == 1 && !long_rows;
    const int i_post = part(a.want_post && !direct, 1, grid, s.dpost, 0, false), i_pre = part(a.want_pre && !direct, 1, grid, s.dpre, 0, false);
    const int i_gate = part(a.want_gate && a.per_gate != 1 && a.segments > 1, s.gates, a.segments, s.dG.w(), s.dG.ld, s.bf16);
    const size_t stats_at = floats;
    if (long_rows) floats += size_t(s.rows) * 4;
    Scratch ws(c, stream);
    void* q = nullptr;
    int r;
    if (floats > 0 && (r = ws.take(floats * sizeof(float), "cudaMallocFromPoolAsync(sums over rows)", &q)) != GBR_OK) return r;
    float* base = static_cast<float*>(q);
    for (int i = 0; i < sums.n; ++i) sums.of[i].in = base + reinterpret_cast<size_t>(sums.of[i].in);
    auto of = [&](int i) { return i < 0 ? nullptr : const_cast<float*>(sums.of[i].in); };
    a.post_part = direct ? s.dpost : of(i_post), a.pre_part = direct ? s.dpre : of(i_pre), a.gate_part = of(i_gate);
    cudaError_t e;
    if (long_rows) {
        float4* stats = reinterpret_cast<float4*>(base + stats_at);
        void* args[] = {&a, &stats};
        e = launch_kernel(vec ? reinterpret_cast<void*>(&residual_norm_stats_kernel<T, true>)
                              : reinterpret_cast<void*>(&residual_norm_stats_kernel<T, false>),
                          dim3(unsigned(std::max<int64_t>(1, std::min<int64_t>(s.rows, 2 * c.sm_count)))), 1024, 0, 1, args,
                          stream);
        if (e != cudaSuccess) return report_cuda(e, "launching residual_norm_backward");
        count_launch();
        e = launch_kernel(vec ? reinterpret_cast<void*>(&residual_norm_grad_long_kernel<T, true>)
                              : reinterpret_cast<void*>(&residual_norm_grad_long_kernel<T, false>),
                          dim3(unsigned(col_ctas), unsigned(grid)), kLongThreads, 0, 1, args, stream);
    } else {
        uint32_t row_bytes = uint32_t(plan.tpr * 8 * plan.V * sizeof(T)), step = plan.ahead > 0 ? uint32_t(plan.step) : 0;
        // Without a ring: not FULL.
        void* kernel = a.parts > 1 ? reinterpret_cast<void*>(&residual_norm_grad_kernel<T, 2, 2, true, kCut>)
                       : plan.V == 2 ? grad_kernel<T, 2>(plan.ahead, full, stream_odd) : grad_kernel<T, 1>(plan.ahead, full, stream_odd);
        const size_t smem = plan.join + size_t(plan.ahead) * step;
        if ((r = raise_kernel_smem(kernel, smem, c.device)) != GBR_OK) return r;
        void* args[] = {&a, &plan.tpr, &row_bytes, &step};
        e = launch_kernel(kernel, dim3(unsigned(grid * a.parts)), plan.threads, smem, a.parts, args, stream);
    }
    if (e != cudaSuccess) return report_cuda(e, "launching residual_norm_backward");
    count_launch();
    return runs == 0 ? GBR_OK : launch_sums(sums, runs, stream);
}

}  // namespace

int launch_residual_norm(const ResidualNormArgs& a, const LibCtx& c, cudaStream_t stream) {
    return a.bf16 ? run_forward<__nv_bfloat16>(a, c, stream) : run_forward<float>(a, c, stream);
}

int launch_residual_norm_grad(const ResidualNormGradArgs& a, const LibCtx& c, cudaStream_t stream) {
    if (a.rows == 0) return no_rows(a, stream);
    return a.bf16 ? run_backward<__nv_bfloat16>(a, c, stream) : run_backward<float>(a, c, stream);
}

}  // namespace gbr
