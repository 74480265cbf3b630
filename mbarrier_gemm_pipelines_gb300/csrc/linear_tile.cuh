// linear_tile.cuh -- the fused linear layer and its gradients' products where
// the output has too few 256 x 256 tiles to fill the GPU: few rows (down to one
// token), or a small output with a long contraction.
//
// The tile is transposed: 128 output COLUMNS are the MMA's M (TMEM lanes) and
// BT output ROWS its N (TMEM columns, 16 to 256), so a single token costs an
// MMA of N = 16 and the weights stream through the tensor core as its wide
// operand.  One CTA per tile and K range, not persistent: a cluster of S CTAs
// (1, 2, 4 or 8) shares a tile, each multiplies its own run of 64-k slices,
// leaves its fp32 part in shared memory, and then every CTA of the cluster
// finishes an equal share of the tile, adding the S parts over distributed
// shared memory in rank order: the result does not depend on timing.
//
//   warps 0-3  TMEM -> shared memory; all warps: sum of parts and epilogue
//   warp 4     TMA producer (one lane)
//   warp 5     TMEM allocation, MMA issue (one lane)
//
// Bound: with few rows, the weights' bytes (each read once); several CTAs an
// SM and a ring of 64-k stages keep the loads in flight.  The parts alias the
// ring, which is idle by then.  Measured, calls back to back: one row of 4096 x
// 4096 7.4 us (34 MB, kept in L2 from call to call) or 9.8 (from HBM, 3.4 TB/s), 37
// rows of 4096 x 14336 23 either way (117 MB at 5.1 TB/s), 512 rows of 4096 x 4096
// 19.4, 301 x 520 x 1000 6.4.
//
// Shared-memory stage: 128 columns of the wide operand, 16 KiB (one K-major
// box or two MN-major panels), then BT rows of the narrow one, BT x 128 bytes
// (one K-major box, or BT / 64 MN-major panels).
#pragma once
#include "gemm_umma.cuh"
#include "mma_issue.cuh"
#include "operators.h"
#include "vec8.cuh"

namespace gbr {
namespace linear {

constexpr uint32_t kTileThreads = 192;
constexpr uint32_t kWideBytes = 128 * 128;
constexpr uint32_t kTileBarBytes = 256;                // barriers and words, before the ring
constexpr uint32_t kTileMaxStages = 12;

struct TileParams {
    CUtensorMap mapW, mapX;
    const float* bias;
    const __nv_bfloat16* R;
    __nv_bfloat16 *C, *Z;
    int64_t ldr, ldc, ldz;
    int32_t I, J;                                      // output rows and columns
    int32_t bt, t_tiles;                               // rows per tile, tiles along the rows
    int32_t num_ks, split;                             // 64-k slices, CTAs sharing a tile
    int32_t stages;
    uint32_t tmem_cols;
    uint32_t vec;                                      // 16-byte accesses to R, C and Z are aligned
    Dropout drop;
    KernelCtl ctl;
    FaultInjection inject;                             // self test only
};

__host__ __device__ constexpr uint32_t tile_stage_bytes(int32_t bt) { return kWideBytes + uint32_t(bt) * 128u; }
// Ring and parts share their memory.  Never below 108 KiB, so that such a CTA
// shares no SM with one of a CTA-pair kernel (120 KiB or more of the 228): a
// cluster whose CTAs wait for Tensor Memory that a pair holds, while the pair
// waits for what another CTA of that cluster holds, would not get on.
__host__ __device__ constexpr size_t tile_smem_bytes(int32_t bt, int32_t stages) {
    const size_t ring = size_t(stages) * tile_stage_bytes(bt), part = size_t(bt) * 512u;
    const size_t need = 1024 + kTileBarBytes + 1024 + (ring > part ? ring : part);
    return need > 108 * 1024 ? need : 108 * 1024;
}

// Eight neighbouring outputs: v holds A B summed over K.
template <int ACT, bool PLAIN>
__device__ __forceinline__ void finish8(const TileParams& P, int32_t i, int32_t j, float (&v)[8]) {
    const int32_t left = P.J - j;                      // >= 1 columns inside
    const bool whole = P.vec != 0 && left >= 8;
    if (!PLAIN) {
        if (P.bias != nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) v[e] += __ldg(P.bias + j + e);
        }
        if (P.Z != nullptr) {
            __nv_bfloat16* z = P.Z + int64_t(i) * P.ldz + j;
            if (whole) {
                store8(z, v);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < left) z[e] = __float2bfloat16_rn(v[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) act_value2<ACT>(v[e], v[e + 1]);
        if (P.drop.threshold != 0) {
            const uint4 bits = dropout_bits(P.drop, uint32_t(i), uint32_t(j) / 8u);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = dropout_keep(P.drop, bits, e) ? v[e] * P.drop.scale : 0.f;
        }
        if (P.R != nullptr) {
            const __nv_bfloat16* r = P.R + int64_t(i) * P.ldr + j;
            if (whole) {
                float w[8];
                load8(r, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += w[e];
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < left) v[e] += __bfloat162float(r[e]);
            }
        }
    }
    __nv_bfloat16* c = P.C + int64_t(i) * P.ldc + j;
    if (whole) {
        store8(c, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left) c[e] = __float2bfloat16_rn(v[e]);
    }
}

// One CTA: `block` among those of the product, in clusters of `cluster` CTAs, a
// multiple of P.split that divides the number of the first of them.
template <bool W_MN, bool X_MN, int ACT, bool PLAIN>
__device__ __forceinline__ void tile_cta(const TileParams& P, uint32_t block, uint32_t cluster) {
    extern __shared__ uint8_t smem_raw[];
    uint64_t* full = reinterpret_cast<uint64_t*>(align_1024(smem_raw));
    uint64_t* empty = full + kTileMaxStages;
    uint64_t* acc_full = empty + kTileMaxStages;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_full + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    uint8_t* ring = align_1024(reinterpret_cast<uint8_t*>(full) + kTileBarBytes);

    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
    const uint32_t S = uint32_t(P.split), stages = uint32_t(P.stages);
    const uint32_t tile = block / S, rank = block % S;
    const uint32_t peer0 = cluster > 1 ? ptx::cluster_ctarank() - rank : 0u;   // of those that share the tile
    const int32_t i0 = int32_t(tile % uint32_t(P.t_tiles)) * P.bt, j0 = int32_t(tile / uint32_t(P.t_tiles)) * 128;
    // A CTA past the last tile only keeps its cluster whole (unsigned: up to 2^31).
    const bool idle = tile / uint32_t(P.t_tiles) * 128u >= uint32_t(P.J);
    const int32_t num_ks = idle ? 0 : P.num_ks;
    const int32_t ks0 = int32_t(int64_t(num_ks) * rank / S), ks1 = int32_t(int64_t(num_ks) * (rank + 1) / S);
    const uint32_t stage_bytes = tile_stage_bytes(P.bt);

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < stages; ++i) {
            ptx::mbar_init(ptx::smem_addr(full + i), 1);
            ptx::mbar_init(ptx::smem_addr(empty + i), 1);
        }
        ptx::mbar_init(ptx::smem_addr(acc_full), 1);
        *abort_flag = 0;
        ptx::fence_barrier_init();
    } else if (threadIdx.x == 128 && P.num_ks > 0) {
        ptx::prefetch_tensormap(&P.mapW);
        ptx::prefetch_tensormap(&P.mapX);
    }
    if (warp == 5) {
        ptx::tmem_alloc(ptx::smem_addr(tmem_holder), P.tmem_cols);
        ptx::tmem_relinquish_alloc_permit();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = *tmem_holder;
    const uint32_t ring_base = ptx::smem_addr(ring);
    ptx::griddep_wait();

    uint32_t issued = 0;
    if (warp == 4 && lane == 0) {
        uint32_t slot = 0, ph = 0;
        for (int32_t ks = ks0; ks < ks1; ++ks, ++issued) {
            if (!mbar_wait(ptx::smem_addr(empty + slot), ph ^ 1u, P.ctl, abort_flag, kSiteProducerEmpty, issued))
                break;
            const uint32_t bar = ptx::smem_addr(full + slot), dst = ring_base + slot * stage_bytes;
            ptx::mbar_arrive_expect_tx(bar, stage_bytes);
            const int32_t k0 = ks * 64;
            if (inject_skip(P.inject, issued)) {
                // self test: the stage's loads are left out
            } else {
                if (W_MN) {
                    ptx::tma_load_2d(dst, &P.mapW, bar, j0, k0);
                    ptx::tma_load_2d(dst + 64 * 128, &P.mapW, bar, j0 + 64, k0);
                } else {
                    ptx::tma_load_2d(dst, &P.mapW, bar, k0, j0);
                }
                if (X_MN) {
                    for (int32_t b = 0; b < P.bt; b += 64)
                        ptx::tma_load_2d(dst + kWideBytes + uint32_t(b) * 128u, &P.mapX, bar, i0 + b, k0);
                } else {
                    ptx::tma_load_2d(dst + kWideBytes, &P.mapX, bar, k0, i0);
                }
            }
            if (++slot == stages) {
                slot = 0;
                ph ^= 1u;
            }
        }
        ptx::griddep_launch_dependents();
    } else if (warp == 5 && lane == 0) {
        // Instruction descriptor: fp32 += bf16 x bf16, M = 128, N = bt.
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(W_MN) << 15) |
                               (uint32_t(X_MN) << 16) | ((uint32_t(P.bt) >> 3) << 17) | ((128u >> 4) << 24);
        constexpr uint32_t hi = desc_hi(1024), lbo_w = W_MN ? 64 * 128 : 16, lbo_x = X_MN ? 64 * 128 : 16;
        const uint32_t w_first = desc_lo(ring_base, lbo_w), x_first = desc_lo(ring_base + kWideBytes, lbo_x);
        const uint32_t full0 = ptx::smem_addr(full), to_empty = ptx::smem_addr(empty) - full0;
        uint32_t at = 0, bar = full0, left = stages, ph = 0, it = 0;
        for (int32_t ks = ks0; ks < ks1; ++ks, ++it) {
            if (!mbar_wait(bar, ph, P.ctl, abort_flag, kSiteMmaFull, it)) break;
            ptx::tc_fence_after_sync();
            mma_slice<W_MN ? kStepMN : kStepK, X_MN ? kStepMN : kStepK>(tmem, w_first + at, x_first + at, hi, idesc,
                                                                        it);
            ptx::mma_commit(bar + to_empty);
            bar += 8;
            at += stage_bytes / 16;
            if (--left == 0) {
                left = stages;
                at = 0;
                bar = full0;
                ph ^= 1u;
            }
        }
        // Completes when every MMA issued has: also what the exit path waits for.
        ptx::mma_commit(ptx::smem_addr(acc_full));
    }
    __syncwarp();

    // All MMAs of this CTA are done: their operands' memory may be reused.
    const bool done = mbar_wait_warp(ptx::smem_addr(acc_full), 0, P.ctl, abort_flag, kSiteEpiAccFull, 0);
    ptx::tc_fence_after_sync();
    const int32_t rows = idle ? 0 : min(P.bt, P.I - i0);
    if (warp < 4 && done) {
        // Part of the tile: [row][128 columns] fp32.
        float* part = reinterpret_cast<float*>(ring) + warp * 32u + lane;
        for (int32_t c = 0; c < rows; c += 16) {
            uint32_t r[16];
            ptx::tmem_ld_32x32b_x16(tmem + ((warp * 32u) << 16) + uint32_t(c), r);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) part[(c + e) * 128] = ks1 > ks0 ? __uint_as_float(r[e]) : 0.f;
        }
    }
    ptx::tc_fence_before_sync();
    __syncwarp();
    if (cluster > 1)
        ptx::cluster_sync_all();
    else
        __syncthreads();
    // After an abort loads may still be in flight; no part is complete then.
    if (*abort_flag) {
        if (warp == 5 && lane == 0) mbar_wait_drain(ptx::smem_addr(acc_full), 0, P.ctl.timeout_ns);
        if (warp == 4 && lane == 0)
            umma::drain_ring<1>(full, stages, issued, 0, stage_bytes, P.inject, blockIdx.x,
                                P.ctl.timeout_ns);
    } else {
        const uint32_t part0 = ring_base;
        for (int32_t u = int32_t(rank * kTileThreads + threadIdx.x); u < rows * 16; u += int32_t(S * kTileThreads)) {
            const int32_t t = u >> 4, j = j0 + (u & 15) * 8;
            if (j >= P.J) continue;
            const uint32_t at = part0 + uint32_t(t) * 512u + uint32_t(u & 15) * 32u;
            // Every part's load is under way before the first is added: one
            // by one they cost a round trip each (128 rows shared by 8 CTAs:
            // 22 us of 4096 x 4096 against 14 us shared by 4).
            float4 a[8], b[8];
#pragma unroll
            for (uint32_t s = 0; s < 8; ++s)
                if (s < S) {
                    const uint32_t from = ptx::mapa_shared(at, peer0 + s);
                    a[s] = ptx::ld_shared_cluster_v4_f32(from);
                    b[s] = ptx::ld_shared_cluster_v4_f32(from + 16);
                }
            float v[8] = {};
#pragma unroll
            for (uint32_t s = 0; s < 8; ++s)
                if (s < S) {
                    v[0] += a[s].x, v[1] += a[s].y, v[2] += a[s].z, v[3] += a[s].w;
                    v[4] += b[s].x, v[5] += b[s].y, v[6] += b[s].z, v[7] += b[s].w;
                }
            finish8<ACT, PLAIN>(P, i0 + t, j, v);
        }
    }
    __syncwarp();
    if (cluster > 1)
        ptx::cluster_sync_all();   // no CTA leaves while a peer may read its part
    else
        __syncthreads();
    if (warp == 5) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, P.tmem_cols);
    }
}

template <bool W_MN, bool X_MN, int ACT, bool PLAIN>
__global__ void __launch_bounds__(kTileThreads)
    linear_tile_kernel(const __grid_constant__ TileParams P) {
    tile_cta<W_MN, X_MN, ACT, PLAIN>(P, blockIdx.x, uint32_t(P.split));
}

// Both products of the gradients in one grid: dA in the first `first` CTAs, dB in
// the others.
struct TileGradParams {
    TileParams da, db;
    uint32_t first, cluster;
};

}  // namespace linear
}  // namespace gbr
