// moe_layer.cu -- a whole mixture-of-experts layer for a few tokens.
//
//   logits = X Wr; per token the top_k largest and the softmax over them;
//   h_te = act(x_t W1_e + b1_e) (gated: act(gate) * up);
//   y_t  = sum over its experts e of w_te (h_te W2_e + b2_e)
//
// Bound by the chosen experts' weights, each read once: one token through 2 of
// 8 experts of 4096 x 14336 needs 470 MB.  Three launches that overlap
// (programmatic dependent launch):
//
// moe_router_kernel   a cluster of 8 CTAs for each group of tokens, each CTA
//     one eighth of the logits' sums; parts added over distributed shared
//     memory in rank order; one warp a token picks the top_k.
//
// moe_expert_kernel   one persistent CTA an SM.  The hidden columns of all
//     chosen experts, in units of 64, are one list that is cut into equal
//     parts.  A part computes its hidden columns for every token (transposed:
//     128 hidden columns are the MMA's M, the tokens its N of 16..64, so no
//     token is gathered: an expert's tokens are picked when results are
//     written), keeps them in shared memory as bf16, and multiplies them at
//     once with its rows of W2: W1's columns and W2's rows of a part belong
//     together, so nothing waits for another CTA and one ring of TMA loads
//     runs through both products without a break.  What comes out is an fp32
//     part of y for the expert's tokens, written to scratch.
//
// moe_combine_kernel  adds the parts of each token's experts in order, times
//     the router's weights.  No atomics: a result depends on the routing alone.
//
// Measured: that token 80 us, of which about 10 pass before the first weights
// arrive (the router, the tables, the first load) and 4 after the last, and 67
// stream the 470 MB at 7.0 TB/s; 64 tokens on all 8 experts, 1.9 GB, 310 us;
// 19 tokens through 6 of 64 gated experts of 2048 x 1000 131 us (rows of 4000
// bytes: HBM reads 812 MB for the 665 that are asked for).
//
// Roles of the expert kernel (192 threads):
//   warps 0-3  TMEM -> hidden values (bias, activation, bf16, swizzled shared
//              memory) and TMEM -> parts
//   warp 4     TMA producer (one lane)
//   warp 5     TMEM allocation, MMA issue (one lane)
#include "gbr.h"
#include "gemm_umma.cuh"
#include "mma_issue.cuh"
#include "moe_cut.cuh"
#include "operators.h"

#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

namespace gbr {
namespace {

using namespace moe;
using bf16 = __nv_bfloat16;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ------------------------------------------------------------ router
constexpr int kRouterThreads = 1024, kRouterCluster = 8, kRouterTokens = 4;

// Orders logits: a NaN below everything, +0 = -0; 0 is below any logit's key.
__device__ __forceinline__ uint32_t logit_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return isnan(x) ? 1u : (u >> 31) ? ~u : u | 0x80000000u;
}

// TB tokens a cluster.  Thread (ty, tx) sums rows ty, ty + ny, ... of this
// CTA's eighth of Wr for experts 4 tx .. 4 tx + 3 (VEC: rows of Wr start on 16
// bytes; 2^shift threads along the experts); one read of Wr serves TB tokens.
// Sums over ty: shuffles within a warp, then over the warps, then over the
// CTAs in rank order, all in a fixed order.
template <int TB, bool VEC>
__global__ void __launch_bounds__(kRouterThreads) moe_router_kernel(const MoeArgs a, int32_t shift) {
    constexpr int kWarps = kRouterThreads / 32;
    extern __shared__ __align__(16) float router_mem[];
    const int wide = 4 << shift;                        // experts, rounded up
    float* red = router_mem;                            // [TB][kWarps][wide]: a warp's sums
    float* sums = red + TB * kWarps * wide;             // of rank 0: [CTA][TB][wide]
    ptx::cluster_arrive();              // this CTA has started
    ptx::griddep_launch_dependents();   // the expert kernel's set-up overlaps this one
    ptx::griddep_wait();
    const uint32_t rank = ptx::cluster_ctarank();
    const int t0 = int(blockIdx.x / kRouterCluster) * TB, tid = int(threadIdx.x), lane = tid % 32, warp = tid / 32;
    const int lanes = 1 << shift, e = (tid & (lanes - 1)) * 4, ty = tid >> shift, ny = kRouterThreads >> shift;
    const int d0 = int(rank) * (a.D / kRouterCluster), d1 = d0 + a.D / kRouterCluster;
    const bf16* x = static_cast<const bf16*>(a.X) + int64_t(t0) * a.D;
    const int tokens = min(TB, a.T - t0), left = a.E - e;
    float acc[TB][4] = {};
    if (left > 0) {
#pragma unroll 4
        for (int d = d0 + ty; d < d1; d += ny) {
            const float* wp = a.Wr + int64_t(d) * a.E + e;
            float w[4] = {};
            if (VEC) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(wp));
                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < left) w[j] = __ldg(wp + j);
            }
#pragma unroll
            for (int i = 0; i < TB; ++i)
                if (i < tokens) {
                    const float xv = __bfloat162float(x[int64_t(i) * a.D + d]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xv, w[j], acc[i][j]);
                }
        }
    }
    // Lanes with the same experts lie `lanes` apart (fewer than 32 lanes), or
    // the warp's lanes all have different ones.
    for (int o = 16; o >= lanes; o /= 2)
#pragma unroll
        for (int i = 0; i < TB; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] += __shfl_xor_sync(0xffffffffu, acc[i][j], o);
    if (lane < lanes)
#pragma unroll
        for (int i = 0; i < TB; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < left) red[(i * kWarps + warp) * wide + e + j] = acc[i][j];
    __syncthreads();
    ptx::cluster_wait();                // rank 0 has started: its memory may be written
    // Of 64 threads along the experts a warp has one half: its row holds those.
    const int stride = lanes > 32 ? lanes / 32 : 1;
    for (int q = warp; q < TB * a.E; q += kWarps) {
        const int i = q / a.E, ee = q % a.E;
        const int first = lanes > 32 ? ee / 128 : 0;    // the warps whose lanes have expert ee
        const int row = first + lane * stride;
        float v = row < kWarps ? red[(i * kWarps + row) * wide + ee] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) {
            const uint32_t at = ptx::smem_addr(sums + (rank * TB + uint32_t(i)) * uint32_t(wide) + uint32_t(ee));
            ptx::st_shared_cluster_u32(ptx::mapa_shared(at, 0), __float_as_uint(v));
        }
    }
    ptx::cluster_sync_all();            // every CTA's sums are in rank 0
    const int i = warp;
    if (rank != 0 || i >= tokens) return;
    float logit[kMoeMaxExperts / 32];
    uint32_t key[kMoeMaxExperts / 32];
#pragma unroll
    for (int c = 0; c < kMoeMaxExperts / 32; ++c) {
        logit[c] = 0.f;
        key[c] = 0u;
        if (32 * c < a.E && lane + 32 * c < a.E) {
#pragma unroll
            for (int r = 0; r < kRouterCluster; ++r) logit[c] += sums[(r * TB + i) * wide + lane + 32 * c];
            key[c] = logit_key(logit[c]);
        }
    }
    int mine = 0;                                       // lane k keeps the k-th choice
    float value = 0.f, top = 0.f;
    for (int k = 0; k < a.top_k; ++k) {
        uint32_t best = 0;
        int at = kMoeMaxExperts;
#pragma unroll
        for (int c = 0; c < kMoeMaxExperts / 32; ++c)
            if (32 * c < a.E && key[c] > best) best = key[c], at = lane + 32 * c;
        const uint32_t most = __reduce_max_sync(0xffffffffu, best);
        const int pick = __reduce_min_sync(0xffffffffu, best == most ? at : kMoeMaxExperts);
        float v = 0.f;
#pragma unroll
        for (int c = 0; c < kMoeMaxExperts / 32; ++c)
            if (pick == lane + 32 * c) {
                key[c] = 0;
                v = logit[c];
            }
        v = __shfl_sync(0xffffffffu, v, pick % 32);
        if (k == 0) top = v;
        if (lane == k) mine = pick, value = v;
    }
    const float w = lane < a.top_k ? expf(value - top) : 0.f;
    float sum = 0.f;
    for (int k = 0; k < a.top_k; ++k) sum += __shfl_sync(0xffffffffu, w, k);
    if (lane < a.top_k) {
        a.ids[int64_t(t0 + i) * a.top_k + lane] = mine;
        a.weights[int64_t(t0 + i) * a.top_k + lane] = w / sum;
    }
}

// ------------------------------------------------------------ experts
constexpr int kThreads = 192;
// 128-column tiles that are accumulated side by side: the tokens' tile of a
// k step is loaded once for all of them, and a row of W1 or W2 is read 1 KiB
// at a time (four tiles' panels one after the other).
constexpr int kWide = 4;

// A position in a ring of n slots.
struct Ring {
    uint32_t slot = 0, phase = 0, count = 0;
    __device__ __forceinline__ void step(uint32_t n) {
        ++count;
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// Where the parts of one (token, choice) lie: rows row0, row0 + step, ...
// (count of them) of the parts' buffer.
struct PairParts {
    int32_t row0, step, count, expert;
};

struct ExpertParams {
    CUtensorMap mapX, mapW1, mapW2, mapW2half;          // W boxes: 64 ksub rows (half: 64)
    MoeArgs a;
    float* parts;                                       // [rows][D] fp32
    PairParts* pairs;                                   // [T * top_k]
    int32_t t_pad;                                      // tokens, rounded up to 16
    CutSizes sizes;
    int32_t stages;
    int32_t ksub;                                       // 64-row slices of a stage, 1 or 2
    KernelCtl ctl;
    FaultInjection inject;                              // self test only
};

struct alignas(16) Tables {
    uint64_t mask[kMoeMaxExperts];                      // tokens of expert e
    int32_t active[kMoeMaxExperts];                     // a-th chosen expert
    int32_t base[kMoeMaxExperts];                       // first row of its parts
    int32_t first[kMoeMaxExperts];                      // its first part
    int32_t num_active;
};

// Exclusive sum over the warp's lanes.
__device__ __forceinline__ int32_t warp_exclusive(int32_t v, uint32_t lane, int32_t& total) {
    int32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (int(lane) >= o) x += y;
    }
    total = __shfl_sync(0xffffffffu, x, 31);
    return x - v;
}

// Builds the tables from the router's choice (all threads of the CTA; the
// masks are zero already).
__device__ __forceinline__ void build_tables(const ExpertParams& P, Tables& tb) {
    const MoeArgs& a = P.a;
    for (int i = int(threadIdx.x); i < a.T * a.top_k; i += kThreads) {
        const int e = int(__ldcg(a.ids + i));
        atomicOr(reinterpret_cast<unsigned long long*>(&tb.mask[e]), 1ull << (i / a.top_k));
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const uint32_t lane = threadIdx.x;
        int32_t active = 0;
        for (int32_t e0 = 0; e0 < a.E; e0 += 32) {      // in the order of the experts
            const bool on = e0 + int32_t(lane) < kMoeMaxExperts && tb.mask[e0 + lane] != 0;
            const uint32_t b = __ballot_sync(0xffffffffu, on);
            if (on) tb.active[active + __popc(b & ((1u << lane) - 1u))] = e0 + int32_t(lane);
            active += __popc(b);
        }
        if (lane == 0) tb.num_active = active;
        __syncwarp();
        const Cut cut = make_cut(P.sizes, active);
        int32_t base = 0;
        for (int32_t x0 = 0; x0 < active; x0 += 32) {
            const int32_t x = x0 + int32_t(lane);
            int32_t rows = 0, sum;
            if (x < active) {
                tb.first[x] = cut.first(x);
                rows = cut.count(x) * __popcll(tb.mask[tb.active[x]]);
            }
            const int32_t before = warp_exclusive(rows, lane, sum);
            if (x < active) tb.base[x] = base + before;
            base += sum;
        }
    }
    __syncthreads();
}

// NG: 1, or 2 when gated: of the first product's kWide tiles, which are then
// gate and up columns in turn.
template <int ACT, int NG>
__global__ void __launch_bounds__(kThreads, 1) moe_expert_kernel(const __grid_constant__ ExpertParams P) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Tables tb;
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], x_full[kXStages], x_empty[kXStages], acc_full[2],
        acc_empty[2], h_full, h_empty, drain;
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    const MoeArgs& a = P.a;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
    const uint32_t S = uint32_t(P.stages), t_pad = uint32_t(P.t_pad), ksub = uint32_t(P.ksub);
    const uint32_t h_block = t_pad * 128u;              // 64 hidden columns of every token
    const uint32_t x_bytes = ksub * h_block;            // 64 ksub columns of X of every token
    const uint32_t panel = ksub * kSliceBytes, stage_bytes = 2 * panel;
    uint8_t* h_mem = align_1024(smem_raw);
    const uint32_t h_base = ptx::smem_addr(h_mem);
    const uint32_t x_base = h_base + uint32_t(P.sizes.max_units) * h_block;
    const uint32_t ring_base = x_base + kXStages * x_bytes;
    // Two accumulators of kWide tiles: a power of two of columns, at most 512.
    const uint32_t tmem_cols = t_pad > 32 ? 512u : 8u * t_pad;
    constexpr int32_t kUnitsPass = 2 * kWide / NG;      // units accumulated side by side

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < S; ++i) {
            ptx::mbar_init(ptx::smem_addr(full + i), 1);
            ptx::mbar_init(ptx::smem_addr(empty + i), 1);
        }
        for (uint32_t i = 0; i < kXStages; ++i) {
            ptx::mbar_init(ptx::smem_addr(x_full + i), 1);
            ptx::mbar_init(ptx::smem_addr(x_empty + i), 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_addr(acc_full + i), 1);
            ptx::mbar_init(ptx::smem_addr(acc_empty + i), 4);
        }
        ptx::mbar_init(ptx::smem_addr(&h_full), 4);
        ptx::mbar_init(ptx::smem_addr(&h_empty), 1);
        ptx::mbar_init(ptx::smem_addr(&drain), 1);
        abort_word = 0;
        ptx::fence_barrier_init();
    } else if (threadIdx.x == 128) {
        ptx::prefetch_tensormap(&P.mapX);
        ptx::prefetch_tensormap(&P.mapW1);
        ptx::prefetch_tensormap(&P.mapW2);
    }
    if (warp == 5) {
        ptx::tmem_alloc(ptx::smem_addr(&tmem_holder), tmem_cols);
        ptx::tmem_relinquish_alloc_permit();
    }
    for (int e = int(threadIdx.x); e < kMoeMaxExperts; e += kThreads) tb.mask[e] = 0;
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = tmem_holder;
    ptx::griddep_wait();
    build_tables(P, tb);
    const Cut cut = make_cut(P.sizes, tb.num_active);
    const int32_t kstep = 64 * int32_t(ksub);
    Ring ring, xring;                                   // of the producer; of the MMA lane

    if (warp == 4 && lane == 0) {
        // ------------------------------------------------------ producer
        bool ok = true;
        const uint64_t once = ptx::l2_policy_evict_first();
        auto stage = [&](uint32_t bytes) -> uint32_t {
            ok = mbar_wait(ptx::smem_addr(empty + ring.slot), ring.phase ^ 1u, P.ctl, abort_flag,
                           kSiteProducerEmpty, ring.count);
            if (ok) ptx::mbar_arrive_expect_tx(ptx::smem_addr(full + ring.slot), bytes);
            return ring_base + ring.slot * stage_bytes;
        };
        Segment s;
        for (Walk w(cut, int32_t(blockIdx.x), P.sizes.sms); ok && w.next(cut, P.sizes.units, s);) {
            const int32_t expert = tb.active[s.index];
            for (int32_t g0 = 0; ok && g0 < s.n; g0 += kUnitsPass) {
                const int32_t g1 = min(g0 + kUnitsPass, s.n);
                for (int32_t k = 0; ok && k < a.D; k += kstep) {
                    if (!(ok = mbar_wait(ptx::smem_addr(x_empty + xring.slot), xring.phase ^ 1u, P.ctl, abort_flag,
                                         kSiteProducerEmpty, xring.count)))
                        break;
                    const uint32_t xbar = ptx::smem_addr(x_full + xring.slot), xdst = x_base + xring.slot * x_bytes;
                    ptx::mbar_arrive_expect_tx(xbar, x_bytes);
                    for (uint32_t h = 0; h < ksub; ++h)
                        ptx::tma_load_2d(xdst + h * h_block, &P.mapX, xbar, k + int32_t(h) * 64, 0);
                    xring.step(kXStages);
                    for (int32_t u = g0; ok && u < g1; u += 2) {
                        const bool two = u + 1 < g1;
#pragma unroll
                        for (int32_t g = 0; g < NG; ++g) {
                            const uint32_t dst = stage(two ? stage_bytes : panel);
                            if (!ok) break;
                            const uint32_t bar = ptx::smem_addr(full + ring.slot);
                            const int32_t col = g * a.F + (s.u0 + u) * kUnit;
                            const bool skip = inject_skip(P.inject, ring.count);
                            if (!skip) ptx::tma_load_3d_hint(dst, &P.mapW1, bar, col, k, expert, once);
                            if (two && !skip)
                                ptx::tma_load_3d_hint(dst + panel, &P.mapW1, bar, col + kUnit, k, expert, once);
                            ring.step(S);
                        }
                    }
                }
            }
            for (int32_t d0 = 0; ok && d0 < a.D; d0 += 128 * kWide)
                for (int32_t b = 0; ok && b < s.n; b += int32_t(ksub)) {
                    const bool half = b + int32_t(ksub) > s.n;   // 64 rows are left, of 128
                    const CUtensorMap* map = half ? &P.mapW2half : &P.mapW2;
                    for (int32_t d = d0; d < min(d0 + 128 * kWide, a.D); d += 128) {
                        const uint32_t dst = stage(half ? 2 * kSliceBytes : stage_bytes);
                        if (!ok) break;
                        const uint32_t bar = ptx::smem_addr(full + ring.slot);
                        if (!inject_skip(P.inject, ring.count)) {
                            ptx::tma_load_3d_hint(dst, map, bar, d, (s.u0 + b) * kUnit, expert, once);
                            ptx::tma_load_3d_hint(dst + panel, map, bar, d + 64, (s.u0 + b) * kUnit, expert, once);
                        }
                        ring.step(S);
                    }
                }
        }
        ptx::griddep_launch_dependents();
    } else if (warp == 5 && lane == 0) {
        // ------------------------------------------------------ MMA issuer
        // fp32 += bf16 x bf16, the wide operand MN-major, M = 128, N = t_pad.
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | ((t_pad >> 3) << 17) |
                               ((128u >> 4) << 24);
        uint32_t tl = 0, hn = 0;
        bool ok = true;
        auto acc_take = [&]() -> uint32_t {
            const uint32_t b = tl & 1u;
            ok = mbar_wait(ptx::smem_addr(acc_empty + b), ((tl >> 1) & 1u) ^ 1u, P.ctl, abort_flag,
                           kSiteMmaAccEmpty, tl);
            ptx::tc_fence_after_sync();
            return tmem + b * kWide * t_pad;
        };
        auto acc_give = [&]() {
            ptx::mma_commit(ptx::smem_addr(acc_full + (tl & 1u)));
            ++tl;
        };
        // One stage into accumulator acc: `slices` (1 or 2) of 64 k; addresses in
        // descriptor units, the tokens' slices x_next apart.
        constexpr uint32_t hi = desc_hi(1024);
        const uint32_t w_first = desc_lo(ring_base, panel), x_next = h_block / 16;
        const uint32_t full0 = ptx::smem_addr(full), to_empty = ptx::smem_addr(empty) - full0;
        const uint32_t bar_end = full0 + 8u * S;
        uint32_t w_lo = w_first, bar = full0, phase = 0;
        // Whether the next stage is full is asked before the present one's MMAs are
        // issued, so that the answer is there when it is needed.
        bool ready = false;
        auto k_step = [&](int32_t tiles, uint32_t acc, uint32_t x_lo, uint32_t slices, uint32_t accumulate) {
#pragma unroll
            for (int32_t j = 0; j < kWide; ++j) {
                if (j >= tiles) break;
                if (!ready && !(ok = mbar_wait(bar, phase, P.ctl, abort_flag, kSiteMmaFull, tl))) break;
                ptx::tc_fence_after_sync();
                const uint32_t give = bar + to_empty, from = w_lo;
                bar += 8;
                w_lo += stage_bytes / 16;
                if (bar == bar_end) {
                    bar = full0;
                    w_lo = w_first;
                    phase ^= 1u;
                }
                ready = mbar_test<false>(bar, phase);
                mma_slice<kStepMN, kStepK>(acc, from, x_lo, hi, idesc, accumulate);
                if (slices == 2)
                    mma_slice<kStepMN, kStepK>(acc, from + kSliceBytes / 16, x_lo + x_next, hi, idesc, 1u);
                ptx::mma_commit(give);
                acc += t_pad;
            }
        };
        Segment s;
        for (Walk w(cut, int32_t(blockIdx.x), P.sizes.sms); ok && w.next(cut, P.sizes.units, s); ++hn) {
            for (int32_t g0 = 0; ok && g0 < s.n; g0 += kUnitsPass) {
                const int32_t tiles = (min(kUnitsPass, s.n - g0) + 1) / 2 * NG;
                const uint32_t acc = acc_take();
                for (int32_t k = 0; ok && k < a.D; k += kstep) {
                    if (!(ok = mbar_wait(ptx::smem_addr(x_full + xring.slot), xring.phase, P.ctl, abort_flag,
                                         kSiteMmaFull, xring.count)))
                        break;
                    const uint32_t x_lo = desc_lo(x_base + xring.slot * x_bytes, 16);
                    k_step(tiles, acc, x_lo, ksub, uint32_t(k));
                    ptx::mma_commit(ptx::smem_addr(x_empty + xring.slot));
                    xring.step(kXStages);
                }
                if (ok) acc_give();
            }
            if (!ok || !(ok = mbar_wait(ptx::smem_addr(&h_full), hn & 1u, P.ctl, abort_flag, kSiteMmaHidden, hn)))
                break;
            ptx::tc_fence_after_sync();
            for (int32_t d0 = 0; ok && d0 < a.D; d0 += 128 * kWide) {
                const int32_t tiles = min(kWide, (a.D - d0 + 127) / 128);
                const uint32_t acc = acc_take();
                for (int32_t b = 0; ok && b < s.n; b += int32_t(ksub)) {
                    const uint32_t x_lo = desc_lo(h_base + uint32_t(b) * h_block, 16);
                    const uint32_t slices = uint32_t(min(int32_t(ksub), s.n - b));
                    k_step(tiles, acc, x_lo, slices, uint32_t(b));
                }
                if (ok) acc_give();
            }
            if (ok) ptx::mma_commit(ptx::smem_addr(&h_empty));
        }
        // No MMA may still be running when TMEM is released.
        ptx::mma_commit(ptx::smem_addr(&drain));
        mbar_wait_drain(ptx::smem_addr(&drain), 0, P.ctl.timeout_ns);
    } else if (warp < 4) {
        // ------------------------------------------------------ epilogue
        // Where the combination finds the parts.
        if (blockIdx.x == 0) {
            for (int i = int(threadIdx.x); i < a.T * a.top_k; i += 128) {
                const int e = int(a.ids[i]), t = i / a.top_k;
                int x = 0;                                  // e's place among the chosen
                for (int lo = 0, hi = tb.num_active; lo < hi;) {
                    x = (lo + hi) / 2;
                    if (tb.active[x] == e) break;
                    if (tb.active[x] < e) lo = x + 1;
                    else hi = x;
                }
                PairParts q;
                q.row0 = tb.base[x] + __popcll(tb.mask[e] & ((1ull << t) - 1));
                q.step = __popcll(tb.mask[e]);
                q.count = cut.count(x);
                q.expert = e;
                P.pairs[i] = q;
            }
        }
        uint32_t tl = 0, hn = 0;
        bool ok = true;
        auto acc_wait = [&]() -> uint32_t {
            const uint32_t b = tl & 1u;
            ok = mbar_wait_warp(ptx::smem_addr(acc_full + b), (tl >> 1) & 1u, P.ctl, abort_flag, kSiteEpiAccFull, tl);
            ptx::tc_fence_after_sync();
            return tmem + ((warp * 32u) << 16) + b * kWide * t_pad;
        };
        auto acc_done = [&]() {
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(acc_empty + (tl & 1u)));
            ++tl;
        };
        Segment s;
        for (Walk w(cut, int32_t(blockIdx.x), P.sizes.sms); ok && w.next(cut, P.sizes.units, s); ++hn) {
            // The previous segment's second product has read the hidden values.
            if (hn > 0 && !(ok = mbar_wait_warp(ptx::smem_addr(&h_empty), (hn - 1u) & 1u, P.ctl, abort_flag,
                                                kSiteEpiHidden, hn)))
                break;
            const int32_t expert = tb.active[s.index];
            const uint64_t mask = tb.mask[expert];
            for (int32_t g0 = 0; ok && g0 < s.n; g0 += kUnitsPass) {
                const uint32_t acc0 = acc_wait();
                if (!ok) break;
                for (int32_t u = g0; u < min(g0 + kUnitsPass, s.n); u += 2) {
                    const int32_t col = int32_t(warp * 32u + lane), f = (s.u0 + u) * kUnit + col;
                    if (col >= 64 && u + 1 >= s.n) continue;   // uniform over the warp
                    const bool inside = f < a.F;
                    float b_gate = 0.f, b_up = 0.f;
                    if (inside && a.b1 != nullptr) {
                        const float* b1 = a.b1 + int64_t(expert) * a.F * NG;
                        b_gate = __ldg(b1 + f);
                        if (NG == 2) b_up = __ldg(b1 + a.F + f);
                    }
                    const uint32_t acc = acc0 + uint32_t(u - g0) / 2u * NG * t_pad;
                    // Row t of the 64-column block: 16-byte chunks swizzled by t % 8.
                    const uint32_t blk = h_base + uint32_t(u + col / 64) * h_block, c8 = uint32_t(col % 64) / 8u;
                    for (uint32_t t = 0; t < t_pad; t += 16) {
                        uint32_t r[16], r2[16];
                        ptx::tmem_ld_32x32b_x16(acc + t, r);
                        if (NG == 2) ptx::tmem_ld_32x32b_x16(acc + t_pad + t, r2);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (uint32_t i = 0; i < 16; i += 2) {
                            float z0 = __uint_as_float(r[i]) + b_gate, z1 = __uint_as_float(r[i + 1]) + b_gate;
                            act_value2<ACT>(z0, z1);
                            r[i] = __float_as_uint(z0);
                            r[i + 1] = __float_as_uint(z1);
                        }
#pragma unroll
                        for (uint32_t i = 0; i < 16; ++i) {
                            float z = __uint_as_float(r[i]);
                            if (NG == 2) z *= __uint_as_float(r2[i]) + b_up;
                            // Columns past F meet zero rows of W2: they must be finite.
                            const bf16 v = __float2bfloat16_rn(inside ? z : 0.f);
                            ptx::st_shared_u16(blk + (t + i) * 128u + ((c8 ^ ((t + i) & 7u)) << 4) +
                                                   uint32_t(col % 8) * 2u,
                                               __bfloat16_as_ushort(v));
                        }
                    }
                }
                acc_done();
            }
            if (!ok) break;
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&h_full));
            // Parts of y: lane = output column, TMEM column = token.
            const int32_t count = __popcll(mask);
            float* out = P.parts + (int64_t(tb.base[s.index]) + int64_t(s.part - tb.first[s.index]) * count) * a.D;
            for (int32_t d0 = 0; ok && d0 < a.D; d0 += 128 * kWide) {
                const uint32_t acc = acc_wait();
                if (!ok) break;
#pragma unroll
                for (int g = 0; g < kWide; ++g) {
                    const int32_t d = d0 + g * 128 + int32_t(warp * 32u + lane);
                    if (d0 + g * 128 >= a.D) break;
                    float* o = out + d;
                    for (uint32_t t = 0; t < t_pad; t += 16) {
                        const uint32_t bits = uint32_t(mask >> t) & 0xFFFFu;
                        if (bits == 0) continue;
                        uint32_t r[16];
                        ptx::tmem_ld_32x32b_x16(acc + uint32_t(g) * t_pad + t, r);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (uint32_t i = 0; i < 16; ++i) {
                            const uint32_t on = (bits >> i) & 1u;
                            if (on != 0 && d < a.D) *o = __uint_as_float(r[i]);
                            o += on * uint32_t(a.D);
                        }
                    }
                }
                acc_done();
            }
        }
    }

    __syncwarp();
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (*abort_flag && warp == 4 && lane == 0) {
        // Stages registered but not consumed: their loads have to land first.
        for (uint32_t j = ring.count > S ? ring.count - S : 0u; j < ring.count; ++j)
            if (!inject_skip(P.inject, j))
                mbar_wait_drain(ptx::smem_addr(full + j % S), (j / S) & 1u, P.ctl.timeout_ns);
        for (uint32_t j = xring.count > kXStages ? xring.count - kXStages : 0u; j < xring.count; ++j)
            mbar_wait_drain(ptx::smem_addr(x_full + j % kXStages), (j / kXStages) & 1u, P.ctl.timeout_ns);
    }
    __syncthreads();
    if (warp == 5) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, tmem_cols);
    }
}

// ------------------------------------------------------------ combination
// 128 columns of one token a CTA; L warps share the parts, whose sums are then
// added in order.  With few tokens L is 32: a token's parts (about 150 of a
// lone token's) are all under way at once.
template <int L>
__global__ void __launch_bounds__(32 * L)
    moe_combine_kernel(const MoeArgs a, const float* parts, const PairParts* pairs) {
    __shared__ float4 red[L][32];
    ptx::griddep_wait();
    const int t = int(blockIdx.y), quad = int(threadIdx.x) % 32, sl = int(threadIdx.x) / 32;
    const int d = (int(blockIdx.x) * 32 + quad) * 4;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (d < a.D) {
        int skip = sl;                                  // this warp's first part of the next choice
        for (int k = 0; k < a.top_k; ++k) {
            const PairParts q = pairs[t * a.top_k + k];
            const float w = a.weights[t * a.top_k + k];
            const float* p = parts + int64_t(q.row0) * a.D + d;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (skip == 0 && a.b2 != nullptr)
                v = __ldg(reinterpret_cast<const float4*>(a.b2 + int64_t(q.expert) * a.D + d));
            int i = skip;
#pragma unroll 4
            for (; i < q.count; i += L) {
                const float4 x = __ldcg(reinterpret_cast<const float4*>(p + int64_t(i) * q.step * a.D));
                v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
            }
            skip = i - q.count;
            y.x = fmaf(w, v.x, y.x), y.y = fmaf(w, v.y, y.y), y.z = fmaf(w, v.z, y.z), y.w = fmaf(w, v.w, y.w);
        }
    }
    red[sl][quad] = y;
    __syncthreads();
    if (sl == 0 && d < a.D) {
#pragma unroll
        for (int i = 1; i < L; ++i) {
            const float4 x = red[i][quad];
            y.x += x.x, y.y += x.y, y.z += x.z, y.w += x.w;
        }
        const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
        uint2 v;
        v.x = *reinterpret_cast<const uint32_t*>(&lo);
        v.y = *reinterpret_cast<const uint32_t*>(&hi);
        *reinterpret_cast<uint2*>(static_cast<bf16*>(a.Y) + int64_t(t) * a.D + d) = v;
    }
}

// ------------------------------------------------------------ host side
template <int NG>
void* expert_kernel(int act) {
    switch (act) {
        case kActRelu: return reinterpret_cast<void*>(&moe_expert_kernel<kActRelu, NG>);
        case kActGelu: return reinterpret_cast<void*>(&moe_expert_kernel<kActGelu, NG>);
        case kActGeluTanh: return reinterpret_cast<void*>(&moe_expert_kernel<kActGeluTanh, NG>);
        case kActSilu: return reinterpret_cast<void*>(&moe_expert_kernel<kActSilu, NG>);
        default: return reinterpret_cast<void*>(&moe_expert_kernel<kActNone, NG>);
    }
}

size_t router_smem_bytes(int tb, int32_t shift) {
    return size_t(tb) * size_t(kRouterThreads / 32 + kRouterCluster) * (size_t(4) << shift) * sizeof(float);
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

template <class... Args>
cudaError_t launch_overlapped(void (*kernel)(Args...), dim3 grid, int threads, int cluster, cudaStream_t stream,
                              Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = unsigned(cluster);
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    n += unsigned(programmatic_launch_attr(attr + n));
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

size_t moe_scratch_bytes(const MoeArgs& a, const LibCtx& c) {
    const ExpertPlan p = plan_experts(a, c.sm_count, c.smem_optin);
    const int64_t rows = most_part_rows(a, {p.units, p.max_units, c.sm_count});
    return up256(size_t(a.T) * a.top_k * sizeof(PairParts)) + size_t(rows) * size_t(a.D) * sizeof(float);
}

int launch_moe(const MoeArgs& a, void* scratch, const LibCtx& c, cudaStream_t stream) {
    const ExpertPlan plan = plan_experts(a, c.sm_count, c.smem_optin);
    ExpertParams P;
    memset(&P, 0, sizeof(P));
    const int64_t F1 = a.gated ? 2 * int64_t(a.F) : a.F;
    const uint64_t xd[2] = {uint64_t(a.D), uint64_t(a.T)}, xs[1] = {uint64_t(a.D) * 2};
    const uint64_t d1[3] = {uint64_t(F1), uint64_t(a.D), uint64_t(a.E)};
    const uint64_t s1[2] = {uint64_t(F1) * 2, uint64_t(F1) * uint64_t(a.D) * 2};
    const uint64_t d2[3] = {uint64_t(a.D), uint64_t(a.F), uint64_t(a.E)};
    const uint64_t s2[2] = {uint64_t(a.D) * 2, uint64_t(a.F) * uint64_t(a.D) * 2};
    const uint32_t bx[2] = {64, uint32_t(plan.t_pad)}, bw[3] = {64, 64u * uint32_t(plan.ksub), 1},
                   bh[3] = {64, 64, 1};
    const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
    // A 128-byte row of a box is fetched with its 256-byte neighbourhood only
    // where that is the next panel's row, not where every row starts elsewhere
    // (1000 gated columns: 163 us with, 155 without).
    auto promotion = [](uint64_t pitch) {
        return pitch % 256 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
    };
    // Gated, W1's panels stand alone (gate and up columns lie F apart): where its
    // rows do not start on 128 bytes, the least that HBM gives, 64 bytes, brings
    // less that nobody asked for (us, 128 / 64 bytes: 19 tokens, 6 of 64 experts
    // of 2048 x 1000 145 / 141, 16 tokens, 4 of 32 of 2008 x 2008 156 / 153, 2
    // tokens, 3 of 8 of 3440 x 5704 131 / 132; not gated up to 2 % slower).
    const auto p1 = a.gated && s1[0] % 128 != 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B : promotion(s1[0]);
    const auto p2 = promotion(s2[0]);
    int r;
    if ((r = encode_tensor_map(&P.mapX, bf, 2, a.X, xd, xs, bx, sw, "X")) != GBR_OK ||
        (r = encode_tensor_map(&P.mapW1, bf, 3, a.W1, d1, s1, bw, sw, "W1", p1)) != GBR_OK ||
        (r = encode_tensor_map(&P.mapW2, bf, 3, a.W2, d2, s2, bw, sw, "W2", p2)) != GBR_OK ||
        (r = encode_tensor_map(&P.mapW2half, bf, 3, a.W2, d2, s2, bh, sw, "W2", p2)) != GBR_OK)
        return r;
    P.a = a;
    P.pairs = static_cast<PairParts*>(scratch);
    P.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) +
                                       up256(size_t(a.T) * a.top_k * sizeof(PairParts)));
    P.t_pad = plan.t_pad, P.sizes = {plan.units, plan.max_units, c.sm_count};
    P.stages = plan.stages, P.ksub = plan.ksub;
    P.ctl = c.ctl;
    P.inject = c.inject;

    int32_t shift = 0;
    while ((4 << shift) < a.E) ++shift;
    // Few tokens: a cluster each, for latency; more share the reads of Wr.
    const int tb = a.T * kRouterCluster <= c.sm_count ? 1 : kRouterTokens;
    const bool vec = a.E % 4 == 0;
    void (*router)(const MoeArgs, int32_t) =
        tb == 1 ? (vec ? moe_router_kernel<1, true> : moe_router_kernel<1, false>)
                : (vec ? moe_router_kernel<kRouterTokens, true> : moe_router_kernel<kRouterTokens, false>);
    const size_t router_smem = router_smem_bytes(tb, shift);
    if ((r = raise_kernel_smem(reinterpret_cast<void*>(router), router_smem, c.device)) != GBR_OK) return r;
    void* rargs[] = {const_cast<MoeArgs*>(&a), &shift};
    cudaError_t e = launch_kernel(reinterpret_cast<void*>(router), dim3(unsigned(cdiv(a.T, tb)) * kRouterCluster),
                                  kRouterThreads, router_smem, kRouterCluster, rargs, stream);
    if (e != cudaSuccess) return report_cuda(e, "launching the router");
    count_launch();

    void* kernel = a.gated ? expert_kernel<2>(a.act) : expert_kernel<1>(a.act);
    if ((r = raise_kernel_smem(kernel, plan.smem, c.device)) != GBR_OK) return r;
    void* args[] = {&P};
    if ((e = launch_kernel(kernel, dim3(unsigned(c.sm_count)), kThreads, plan.smem, 1, args, stream)) != cudaSuccess)
        return report_cuda(e, "launching the experts");
    count_launch();
    const dim3 cg(unsigned(cdiv(a.D, 128)), unsigned(a.T));
    const float* parts = P.parts;
    const PairParts* pairs = P.pairs;
    e = a.T <= 8 ? launch_overlapped(moe_combine_kernel<32>, cg, 32 * 32, 1, stream, a, parts, pairs)
                 : launch_overlapped(moe_combine_kernel<8>, cg, 32 * 8, 1, stream, a, parts, pairs);
    if (e != cudaSuccess) return report_cuda(e, "launching the combination");
    count_launch();
    return GBR_OK;
}

}  // namespace gbr
