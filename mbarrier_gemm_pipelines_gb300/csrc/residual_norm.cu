// residual_norm.cu -- the norms before and after a block with its gate and the
// residual, and their gradients.
//
//   y = X q post,  q = 1 / sqrt(mean X^2 + eps)      (no post: y = X)
//   S = R + scale gate y
//   H = S r pre,   r = 1 / sqrt(mean S^2 + eps)
//
//   u = dH pre;  ds = dS + r u - S r^3 mean(u S)      dR = ds, dpre = sum dH S r
//   dy = scale gate ds                                dgate = sum scale y ds
//   v = dy post; dX = q v - X q^3 mean(v X)           dpost = sum dy X q
//
// Bound by memory: every operand is read once and every output written once; a
// group of threads holds its row in registers between the passes that the two
// means need.  Statistics and sums are fp32.  H comes from the sum before it is
// rounded to S.
#include "gbr.h"
#include "operators.h"
#include "row8.cuh"

#include <algorithm>
#include <cstdint>

namespace gbr {
namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename T>
struct Args {
    const T *X, *R, *G;
    const float *post, *pre;
    T *S, *H;
    int64_t ldx, ldr, ldg, lds, ldh;
    int32_t rows, cols, per_gate;      // rows that share a row of G
    float scale, eps, inv_cols;
};

__device__ __forceinline__ float root(float sum, float inv_cols, float eps) { return rsqrtf(fmaf(sum, inv_cols, eps)); }

// ------------------------------------------------------------ forward
// blockDim.x / tpr rows a CTA, V * 8 columns a thread.
template <typename T, int V, bool VEC>
__global__ void __launch_bounds__(1024) residual_norm_kernel(const Args<T> a, int32_t tpr) {
    __shared__ float buf[2][1][32];
    ptx::griddep_wait();
    const int32_t t = int32_t(threadIdx.x) % tpr;
    const int64_t row = int64_t(blockIdx.x) * (int32_t(blockDim.x) / tpr) + int32_t(threadIdx.x) / tpr;
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
            group_sum(sum, buf[0], tpr);
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
    group_sum(sum, buf[1], tpr);
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
// 16384 x 4096 bf16 with all but row gates: a row a CTA 131 us, this 84 (6.4 TB/s).  More on their way is slower, HBM
// reading and writing at once: three CTAs an SM and three turns ahead 97, two and three 84 to 88, two and five 95.
template <typename T, int V, int kAhead, int kMost>
__global__ void __launch_bounds__(kMost, kMost == 256 ? 2 : 1) residual_norm_stream_kernel(const Args<T> a, int32_t tpr,
                                                                                       uint32_t row_bytes, uint32_t step) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float buf[2][1][32];
    ptx::griddep_wait();
    const int32_t t = int32_t(threadIdx.x) % tpr, group = int32_t(threadIdx.x) / tpr, groups = int32_t(blockDim.x) / tpr;
    const int32_t cols = a.cols;
    const bool has_r = a.R != nullptr, one_gate = a.G != nullptr && a.per_gate == a.rows, gates = a.G != nullptr && !one_gate;
    const uint32_t base = ptx::smem_addr(ring) + uint32_t(group) * row_bytes, wide = row_bytes * uint32_t(groups);
    auto fetch = [&](int64_t row, uint32_t slot) {
        if (row < a.rows) {
            uint32_t to = base + slot * step;
#pragma unroll
            for (int v = 0; v < V; ++v) copy_row8(to, a.X + row * a.ldx, v, t, tpr, cols);
            if (has_r) {
                to += wide;
#pragma unroll
                for (int v = 0; v < V; ++v) copy_row8(to, a.R + row * a.ldr, v, t, tpr, cols);
            }
            if (gates) {
                to += wide;
#pragma unroll
                for (int v = 0; v < V; ++v) copy_row8(to, a.G + row / a.per_gate * a.ldg, v, t, tpr, cols);
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
        if (post) load_pairs<float, true>(w[v], a.post, v, t, tpr, cols);
        if (a.pre != nullptr) load_pairs<float, true>(wpre[v], a.pre, v, t, tpr, cols);
        if (one_gate) load_pairs<T, true>(g, a.G, v, t, tpr, cols);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[v][i] = post ? mul2(w[v][i], f2(a.scale)) : f2(a.scale);
            if (one_gate) w[v][i] = mul2(w[v][i], g[i]);
        }
    }
    clear_past<T, V>(ptx::smem_addr(ring), kAhead * step / row_bytes, row_bytes, t, tpr, cols);
    const int64_t turn = int64_t(gridDim.x) * groups;
    int64_t first = int64_t(blockIdx.x) * groups;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(first + group + i * turn, uint32_t(i));
    for (uint32_t slot = 0; first < a.rows; first += turn, slot = slot + 1 == kAhead ? 0 : slot + 1) {
        const int64_t row = first + group;
        const int32_t out = row < a.rows ? cols : 0;    // a group past the end only keeps the barriers
        copy_async_wait<kAhead - 1>();
        const uint32_t from = base + slot * step;
        Raw8<T> x[V], r[V] = {}, g[V] = {};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            take_row8(x[v], from, v, t, tpr);
            if (has_r) take_row8(r[v], from + wide, v, t, tpr);
            if (gates) take_row8(g[v], from + (has_r ? 2u : 1u) * wide, v, t, tpr);
        }
        float q = 1.f;
        if (post) {
            F2 xx = f2(0.f);
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 4; ++i) xx = fma2(raw_pair(x[v], i), raw_pair(x[v], i), xx);
            float sum[1] = {sum_pair(xx)};
            group_sum(sum, buf[0], tpr);
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
            if (a.S != nullptr) store_pairs<T, true>(a.S + row * a.lds, s[v], v, t, tpr, out);
        }
        float sum[1] = {sum_pair(ss)};
        if (a.H != nullptr) group_sum(sum, buf[1], tpr);
        // The slot has been read into registers that the lines above have used.
        fetch(row + kAhead * turn, slot);
        if (a.H != nullptr) {
            const F2 p = f2(root(sum[0], a.inv_cols, a.eps));
#pragma unroll
            for (int v = 0; v < V; ++v) {
                F2 h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = mul2(mul2(s[v][i], p), wpre[v][i]);
                store_pairs<T, true>(a.H + row * a.ldh, h, v, t, tpr, out);
            }
        }
        if (tpr > 32 && (!post || a.H == nullptr)) __syncthreads();   // buf, for the next row
    }
    copy_async_wait<0>();
}

// Rows that no CTA can hold: a CTA a row, read again for each mean.
template <typename T>
__device__ __forceinline__ float sum_at(const Args<T>& a, int64_t row, float q, int32_t c) {
    float y = to_f32(a.X[row * a.ldx + c]);
    if (a.post != nullptr) y = y * q * a.post[c];
    if (a.G != nullptr) y *= to_f32(a.G[row / a.per_gate * a.ldg + c]);
    if (a.R == nullptr && a.scale == 1.f) return y;
    return fmaf(a.scale, y, a.R != nullptr ? to_f32(a.R[row * a.ldr + c]) : 0.f);
}

template <typename T>
__global__ void __launch_bounds__(1024) residual_norm_long_kernel(const Args<T> a) {
    __shared__ float buf[2][1][32];
    ptx::griddep_wait();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float sum[1] = {}, q = 1.f;
        if (a.post != nullptr) {
            for (int32_t c = int32_t(threadIdx.x); c < a.cols; c += 1024) {
                const float x = to_f32(a.X[row * a.ldx + c]);
                sum[0] = fmaf(x, x, sum[0]);
            }
            group_sum(sum, buf[0], 1024);
            q = root(sum[0], a.inv_cols, a.eps);
        }
        float r = 0.f;
        if (a.H != nullptr) {
            sum[0] = 0.f;
            for (int32_t c = int32_t(threadIdx.x); c < a.cols; c += 1024) {
                const float s = sum_at(a, row, q, c);
                sum[0] = fmaf(s, s, sum[0]);
            }
            group_sum(sum, buf[1], 1024);
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
    int64_t ldds, lddh, ldx, lds, ldg, lddx, lddr, lddg;
    int32_t rows, cols, per_gate;
    float scale, eps, inv_cols;
    // Sums over rows: `items` runs of rows, `segments` of them to a gate; each CTA takes a
    // contiguous share of the items.  part: per CTA [post][pre] rows of cols, or null; gate_part:
    // per item, where a gate has several segments (one segment: dG itself).
    int32_t items, segments, span;     // span: rows of a gate (all rows where the items are one run)
    float *post_part, *pre_part, *gate_part;
    bool want_post, want_pre, want_gate;
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

// One CTA: its items' rows, blockDim.x / tpr at a time.  Thread t of each group keeps the sums of
// its columns; groups are joined in order through shared memory.  kAhead > 0 (rows on 16 bytes): that many
// turns' rows of all inputs are on their way into shared memory, each thread its own 16 bytes, so that nobody
// waits for another's copy; 0: they are loaded in their turn, any alignment.
// FULL: a training step's call, with both norms, dS and all of dX, dR, dpost and dpre, without a gate an element.  What
// is there need not be asked then (4096 x 4096: 631 instructions a warp and row of 8 columns a thread if it is, 447 not),
// and the registers are kept for the row: the weights lie in shared memory, each thread's where it alone reads them, and
// dpost's sum in its place in scratch, added to after a gate's rows.
template <typename T, int V, int kAhead, bool FULL>
__global__ void __launch_bounds__(512) residual_norm_grad_kernel(const GradArgs<T> a, int32_t tpr, uint32_t row_bytes,
                                                                 uint32_t step) {
    constexpr bool VEC = kAhead > 0;
    __shared__ float buf[2][3][32];
    // The ring; behind it, where groups > 1, [groups][8][tpr] floats.
    extern __shared__ __align__(16) uint8_t ring[];
    ptx::griddep_wait();
    const int32_t t = int32_t(threadIdx.x) % tpr, group = int32_t(threadIdx.x) / tpr;
    const int32_t groups = int32_t(blockDim.x) / tpr;
    const int32_t i0 = int32_t(int64_t(a.items) * blockIdx.x / gridDim.x);
    const int32_t i1 = int32_t(int64_t(a.items) * (blockIdx.x + 1) / gridDim.x);
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
        if (gate_rows && post) load_pairs<float, VEC>(wpost[v], a.post, v, t, tpr, a.cols);
        if (pre) load_pairs<float, VEC>(wpre[v], a.pre, v, t, tpr, a.cols);
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
    ahead.enter(a);
    bool more = ahead.settle(a);
    auto fetch = [&](uint32_t slot) {
        const int64_t row = ahead.first + group;
        if (more && row < ahead.end) {
            const uint32_t to = ring0 + slot * step;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (pre) {
                    copy_row8(to, a.dH + row * a.lddh, v, t, tpr, a.cols);
                    copy_row8(to + wide, a.S + row * a.lds, v, t, tpr, a.cols);
                }
                if (has_x) copy_row8(to + at_x * wide, a.X + row * a.ldx, v, t, tpr, a.cols);
                if (has_ds) copy_row8(to + at_ds * wide, a.dS + row * a.ldds, v, t, tpr, a.cols);
                if (gate_rows) copy_row8(to + at_g * wide, a.G + row * a.ldg, v, t, tpr, a.cols);
            }
        }
        copy_async_commit();
        if (more) {
            ahead.first += groups;
            more = ahead.settle(a);
        }
    };
    if (kAhead > 0) clear_past<T, V>(ptx::smem_addr(ring), kAhead * step / row_bytes, row_bytes, t, tpr, a.cols);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(uint32_t(i));
    uint32_t slot = 0;
    for (int32_t item = i0; item < i1; ++item) {
        const int32_t g = item / a.segments, seg = item % a.segments;
        const int64_t base = int64_t(g) * a.span;
        const int64_t r0 = base + int64_t(a.span) * seg / a.segments, r1 = base + int64_t(a.span) * (seg + 1) / a.segments;
        const T* gate = run_gate ? a.G + g * a.ldg : nullptr;
        F2 gw[V][4];                                    // gate times weight
        if (!gate_rows && weighted)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                F2 w[4];
                if (post) load_pairs<float, VEC>(gw[v], a.post, v, t, tpr, a.cols);
                if (run_gate) load_pairs<T, VEC>(w, gate, v, t, tpr, a.cols);
#pragma unroll
                for (int i = 0; i < 4; ++i) gw[v][i] = !run_gate ? gw[v][i] : post ? mul2(gw[v][i], w[i]) : w[i];
                if (FULL) put_pairs(own_gw + uint32_t(v) * 32u * blockDim.x, gw[v]);
            }
        for (int64_t first = r0; first < r1; first += groups) {
            const int64_t row = first + group;
            const bool in = row < r1;
            const int32_t cols = in ? a.cols : 0;
            Raw8<T> x[V] = {}, s[V] = {}, dh[V] = {}, ds[V] = {}, gt[V] = {};
            if (kAhead > 0) {
                copy_async_wait<(kAhead > 0 ? kAhead : 1) - 1>();
                const uint32_t from = ring0 + slot * step;
                if (in)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        if (pre) {
                            take_row8(dh[v], from, v, t, tpr);
                            take_row8(s[v], from + wide, v, t, tpr);
                        }
                        if (has_x) take_row8(x[v], from + at_x * wide, v, t, tpr);
                        if (has_ds) take_row8(ds[v], from + at_ds * wide, v, t, tpr);
                        if (gate_rows) take_row8(gt[v], from + at_g * wide, v, t, tpr);
                    }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (has_x) load_raw8<VEC>(x[v], a.X + row * a.ldx, v, t, tpr, cols);
                    if (pre) {
                        load_raw8<VEC>(s[v], a.S + row * a.lds, v, t, tpr, cols);
                        load_raw8<VEC>(dh[v], a.dH + row * a.lddh, v, t, tpr, cols);
                    }
                    if (has_ds) load_raw8<VEC>(ds[v], a.dS + row * a.ldds, v, t, tpr, cols);
                    if (gate_rows) load_raw8<VEC>(gt[v], a.G + row * a.ldg, v, t, tpr, cols);
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
            if (pre || post) group_sum(sum, buf[0], tpr);
            // A group without a row adds zeros.
            const float r = in ? root(sum[0], a.inv_cols, a.eps) : 0.f, rc = r * r * r * sum[1] * a.inv_cols;
            const float q = !post ? 1.f : in ? root(sum[2], a.inv_cols, a.eps) : 0.f;
            F2 d[V][4], dot = f2(0.f);
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 4; ++i) d[v][i] = raw_pair(ds[v], i);
            if (pre) {
                const F2 r2 = f2(r), m2 = f2(-rc);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (FULL) get_pairs(wpre[v], own + uint32_t(v) * 32u * blockDim.x);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const F2 S = raw_pair(s[v], i), H = raw_pair(dh[v], i);
                        d[v][i] = fma2(S, m2, fma2(r2, mul2(H, wpre[v][i]), d[v][i]));
                        spre[v][i] = fma2(H, mul2(S, r2), spre[v][i]);
                    }
                }
            }
            if (want_r)
#pragma unroll
                for (int v = 0; v < V; ++v) store_pairs<T, VEC>(a.dR + row * a.lddr, d[v], v, t, tpr, cols);
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
                    if (a.want_gate) store_pairs<T, VEC>(a.dG + row * a.lddg, dg, v, t, tpr, cols);
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
                    group_sum(sums, buf[1], tpr);
                    m2 = f2(-a.scale * (q * q * q * sums[0] * a.inv_cols));
                }
                const F2 k2 = f2(a.scale * q);
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        d[v][i] = mul2(d[v][i], k2);
                        if (post) d[v][i] = fma2(raw_pair(x[v], i), m2, d[v][i]);
                    }
                    store_pairs<T, VEC>(a.dX + row * a.lddx, d[v], v, t, tpr, cols);
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
                    float* sum = a.post_part + int64_t(blockIdx.x) * a.cols;
                    if (run_gate) load_pairs<T, VEC>(w, gate, v, t, tpr, a.cols);
                    if (FULL && item > i0) load_pairs<float, VEC>(spost[v], sum, v, t, tpr, a.cols);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const F2 k = run_gate ? mul2(f2(a.scale), w[i]) : f2(a.scale);
                        spost[v][i] = fma2(srun[v][i], k, spost[v][i]);
                    }
                    if (FULL) {
                        store_pairs<float, VEC>(sum, spost[v], v, t, tpr, a.cols);
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
                        if (post) load_pairs<float, VEC>(w, a.post, v, t, tpr, a.cols);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            srun[v][i] = mul2(srun[v][i], f2(a.scale));
                            if (post) srun[v][i] = mul2(srun[v][i], w[i]);
                        }
                        if (a.segments > 1)
                            store_pairs<float, VEC>(a.gate_part + int64_t(item) * a.cols, srun[v], v, t, tpr, a.cols);
                        else
                            store_pairs<T, VEC>(a.dG + g * a.lddg, srun[v], v, t, tpr, a.cols);
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
                store_pairs<float, VEC>(a.post_part + int64_t(blockIdx.x) * a.cols, spost[v], v, t, tpr, a.cols);
    }
    if (want_pre) {
        join(spre);
        if (group == 0)
#pragma unroll
            for (int v = 0; v < V; ++v)
                store_pairs<float, VEC>(a.pre_part + int64_t(blockIdx.x) * a.cols, spre[v], v, t, tpr, a.cols);
    }
}

// Rows that no CTA holds with what goes with them: their means first (a CTA a row), then everything else column by
// column, 8 of them a thread.
constexpr int kLongThreads = 256;

// stats[row] = {r, r^3 mean(u S), q, q^3 mean(v X)}
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024, 1) residual_norm_stats_kernel(const GradArgs<T> a, float4* stats) {
    __shared__ float buf[2][3][32];
    ptx::griddep_wait();
    const bool pre = a.pre != nullptr, post = a.post != nullptr;
    const int32_t t = int32_t(threadIdx.x), pieces = (a.cols + 8191) / 8192;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        F2 ss = f2(0.f), us = f2(0.f), xx = f2(0.f), vx = f2(0.f);
        for (int32_t p = 0; p < pieces; ++p) {
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
        float sum[3] = {sum_pair(ss), sum_pair(us), sum_pair(xx)};
        group_sum(sum, buf[0], 1024);
        const float r = root(sum[0], a.inv_cols, a.eps), rc = r * r * r * sum[1] * a.inv_cols;
        const float q = post ? root(sum[2], a.inv_cols, a.eps) : 1.f;
        if (post)
            for (int32_t p = 0; p < pieces; ++p) {
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
                    if (pre) e = fma2(raw_pair(s, i), f2(-rc), fma2(f2(r), mul2(raw_pair(dh, i), w[i]), e));
                    if (a.G != nullptr) e = mul2(e, raw_pair(g, i));
                    vx = fma2(mul2(e, wp[i]), raw_pair(x, i), vx);
                }
            }
        float dot[1] = {sum_pair(vx)};
        group_sum(dot, buf[1], 1024);
        if (threadIdx.x == 0) stats[row] = make_float4(r, rc, q, a.scale * (q * q * q * dot[0] * a.inv_cols));
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
                    e[i] = fma2(S, f2(-st.y), fma2(f2(st.x), mul2(H, wpre[i]), e[i]));
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
                e[i] = mul2(mul2(e[i], wpost[i]), f2(st.z));
                if (post) e[i] = fma2(X, f2(-st.w), e[i]);
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

// Threads a row: the fewest warps (or less, as `least` lets them) that hold it with V vectors each.
int threads_for(int64_t cols, int V, int least = 32) {
    int tpr = least;
    while (int64_t(tpr) * 8 * V < cols) tpr *= 2;
    return tpr;
}

template <typename T, int V>
void* forward_kernel(bool vec) {
    return vec ? reinterpret_cast<void*>(&residual_norm_kernel<T, V, true>)
               : reinterpret_cast<void*>(&residual_norm_kernel<T, V, false>);
}

template <typename T, int kAhead, int kMost>
void* stream_kernel() {
    return reinterpret_cast<void*>(&residual_norm_stream_kernel<T, 2, kAhead, kMost>);
}

struct StreamPlan {
    int32_t tpr;
    int threads, ctas, ahead;                           // ctas: an SM, by registers
    size_t step;
};
StreamPlan stream_plan(const ResidualNormArgs& s, size_t esize) {
    StreamPlan p;
    const int inputs = 1 + (s.R.p ? 1 : 0) + (s.G.p && s.gates > 1 ? 1 : 0);
    p.tpr = threads_for(s.cols, 2, 4);
    p.threads = std::max(256, int(p.tpr)), p.ctas = p.threads > 256 ? 1 : 2;
    p.step = size_t(p.threads) * 16 * esize * size_t(inputs);
    p.ahead = p.threads > 256 && 3 * p.step <= 216 * 1024 ? 3 : 2;
    return p;
}
// Rows of up to 8192 columns, and enough of them for CTAs that stay: eight turns of all.
bool streams(const ResidualNormArgs& s, size_t esize, int sm_count) {
    if (s.cols > 8192) return false;
    const StreamPlan p = stream_plan(s, esize);
    return s.rows >= int64_t(8) * sm_count * (p.threads / p.tpr) && size_t(p.ahead) * p.step <= 216 * 1024;
}

template <typename T>
int run_forward(const ResidualNormArgs& s, const LibCtx& c, cudaStream_t stream) {
    Args<T> a = {static_cast<const T*>(s.X.p), static_cast<const T*>(s.R.p), static_cast<const T*>(s.G.p), s.post, s.pre,
                 static_cast<T*>(s.S.w()), static_cast<T*>(s.H.w()), s.X.ld, s.R.ld, s.G.ld, s.S.ld, s.H.ld, s.rows,
                 s.cols, s.per_gate, s.scale, s.eps, float(1.0 / double(s.cols))};
    bool vec = s.cols % 8 == 0 && aligned16<float>(s.post, 0, 1) && aligned16<float>(s.pre, 0, 1) &&
               aligned16<T>(s.G.p, s.G.ld, s.gates);
    for (const Mat* m : {&s.X, &s.R, &s.S, &s.H}) vec = vec && aligned16<T>(m->p, m->ld, s.rows);
    cudaError_t e;
    if (s.cols > 1024 * 32) {
        void* args[] = {&a};
        e = launch_kernel(reinterpret_cast<void*>(&residual_norm_long_kernel<T>),
                          dim3(unsigned(std::min<int64_t>(s.rows, 2 * c.sm_count))), 1024, 0, 1, args, stream);
    } else if (vec && streams(s, sizeof(T), c.sm_count)) {
        const StreamPlan p = stream_plan(s, sizeof(T));
        int32_t tpr = p.tpr;
        uint32_t row_bytes = uint32_t(p.tpr * 16 * sizeof(T)), step = uint32_t(p.step);
        void* kernel = p.threads <= 256 ? stream_kernel<T, 2, 256>()
                       : p.ahead == 3   ? stream_kernel<T, 3, 512>()
                                        : stream_kernel<T, 2, 512>();
        const size_t smem = size_t(p.ahead) * p.step;
        const int r = raise_kernel_smem(kernel, smem, c.device);
        if (r != GBR_OK) return r;
        void* args[] = {&a, &tpr, &row_bytes, &step};
        e = launch_kernel(kernel, dim3(unsigned(c.sm_count * std::min<int64_t>(p.ctas, 216 * 1024 / smem))), p.threads, smem,
                          1, args, stream);
    } else {
        const int V = s.cols > 1024 * 16 ? 4 : s.cols > 1024 * 8 ? 2 : 1;
        int32_t tpr = threads_for(s.cols, V, 4);
        const int threads = std::max(256, int(tpr));
        void* kernel = V == 4 ? forward_kernel<T, 4>(vec) : V == 2 ? forward_kernel<T, 2>(vec) : forward_kernel<T, 1>(vec);
        void* args[] = {&a, &tpr};
        e = launch_kernel(kernel, dim3(unsigned(cdiv(s.rows, threads / tpr))), threads, 0, 1, args, stream);
    }
    if (e != cudaSuccess) return report_cuda(e, "launching residual_norm");
    count_launch();
    return GBR_OK;
}

template <typename T, int V>
void* grad_kernel(int ahead, bool full) {
    switch (ahead) {
        case 3: return full ? reinterpret_cast<void*>(&residual_norm_grad_kernel<T, V, 3, true>)
                            : reinterpret_cast<void*>(&residual_norm_grad_kernel<T, 1, 3, false>);
        case 2: return full ? reinterpret_cast<void*>(&residual_norm_grad_kernel<T, V, 2, true>)
                            : reinterpret_cast<void*>(&residual_norm_grad_kernel<T, 1, 2, false>);
        default: return reinterpret_cast<void*>(&residual_norm_grad_kernel<T, 1, 0, false>);
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
    const bool full = vec && s.post && s.pre && s.dS.p && s.dX.p && s.dR.p && a.want_post && a.want_pre && !gate_rows;
    const int inputs = (s.pre ? 2 : 0) + (s.X.p ? 1 : 0) + (s.dS.p ? 1 : 0) + (gate_rows ? 1 : 0);
    // V vectors a thread.  Two where the rows go round (the fewer warps a row, the less of what is done once a warp) and
    // two turns of them fit; rows that do not fit at all have their means taken first (as rows of fp32 of 8192 columns).
    struct Plan {
        int V, threads, groups, ahead;
        int32_t tpr;
        size_t step, join;
    } plan = {};
    auto lay_out = [&](int V) {
        plan.V = V, plan.tpr = threads_for(s.cols, V), plan.threads = std::max(256, int(plan.tpr));
        plan.groups = plan.threads / plan.tpr;
        const size_t mine = size_t(plan.threads) * 8 * sizeof(float);
        plan.join = (plan.groups > 1 ? mine : 0) + (full ? 2 * mine * V : 0);
        plan.step = vec ? size_t(plan.threads) * 8 * V * sizeof(T) * size_t(inputs) : 0;
        const size_t most = size_t(plan.threads > 256 ? 220 : 111) * 1024 - plan.join;
        plan.ahead = !vec ? 0 : 3 * plan.step <= most ? 3 : 2 * plan.step <= most ? 2 : 0;
    };
    const bool many = s.rows >= int64_t(c.sm_count) * 8 * std::max(1, 4096 / s.cols);
    if (s.cols <= 8192) lay_out(full && (many || s.cols > 4096) ? 2 : 1);
    if (plan.V == 2 && plan.ahead == 0 && s.cols <= 4096) lay_out(1);
    const bool long_rows = s.cols > 8192 || plan.tpr > 512 || (plan.V == 2 && plan.ahead == 0);
    const int64_t col_ctas = cdiv(s.cols, kLongThreads * 8);
    const int64_t ctas = long_rows ? std::max<int64_t>(1, 4 * c.sm_count / col_ctas)
                                   : c.sm_count * (plan.threads > 256 ? 1 : 2);
    const int64_t grid = cut_rows(&a, s.gates, ctas, long_rows ? 1 : plan.groups);
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
    const int i_post = part(a.want_post, 1, grid, s.dpost, 0, false), i_pre = part(a.want_pre, 1, grid, s.dpre, 0, false);
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
    a.post_part = of(i_post), a.pre_part = of(i_pre), a.gate_part = of(i_gate);
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
        void* kernel = plan.V == 2 ? grad_kernel<T, 2>(plan.ahead, full) : grad_kernel<T, 1>(plan.ahead, full);
        const size_t smem = plan.join + size_t(plan.ahead) * step;
        if ((r = raise_kernel_smem(kernel, smem, c.device)) != GBR_OK) return r;
        void* args[] = {&a, &plan.tpr, &row_bytes, &step};
        e = launch_kernel(kernel, dim3(unsigned(grid)), plan.threads, smem, 1, args, stream);
    }
    if (e != cudaSuccess) return report_cuda(e, "launching residual_norm_backward");
    count_launch();
    if (runs == 0) return GBR_OK;
    void* args[] = {&sums};
    e = launch_kernel(reinterpret_cast<void*>(&norm_sums_kernel), dim3(unsigned(cdiv(s.cols, 32)), unsigned(runs)), 512,
                      0, 1, args, stream);
    if (e != cudaSuccess) return report_cuda(e, "launching the sums of residual_norm_backward");
    count_launch();
    return GBR_OK;
}

}  // namespace

int launch_residual_norm(const ResidualNormArgs& a, const LibCtx& c, cudaStream_t stream) {
    return a.bf16 ? run_forward<__nv_bfloat16>(a, c, stream) : run_forward<float>(a, c, stream);
}

int launch_residual_norm_grad(const ResidualNormGradArgs& a, const LibCtx& c, cudaStream_t stream) {
    return a.bf16 ? run_backward<__nv_bfloat16>(a, c, stream) : run_backward<float>(a, c, stream);
}

}  // namespace gbr
