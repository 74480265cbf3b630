// mxfp4_tile.cuh -- C = R + act(A B^T + bias) from microscaled 4-bit operands
// where the output has too few 256 x 256 tiles to fill the GPU: down to one row.
//
// The layout of linear_tile.cuh: 128 output COLUMNS are the MMA's M, so that the
// weights stream through the tensor core as its wide operand, BT output ROWS its
// N; a cluster of 1, 2, 4 or 8 CTAs shares a tile along K and adds its fp32
// parts in rank order over distributed shared memory.  A 128-byte slice of a row
// is 256 values here, so bytes, ring and MMAs are those of a bf16 product with a
// quarter of the contraction, and the choice of tile and split is the same.
//
// Stage: 128 columns of B (16 KiB), BT rows of A (BT x 128 bytes), the scales of
// both (1 KiB for 128 rows and 8 blocks).  The MMA's thread copies the scales to
// Tensor Memory; the tensor core runs copies and MMAs in order.  Two sets of
// columns alternate, and a stage's copies are issued in front of the MMAs of the
// stage before, so that neither waits for the other.
#pragma once
#include "linear_tile.cuh"
#include "mxfp4.cuh"

namespace gbr {
namespace mx {

using linear::kTileBarBytes;
using linear::kTileMaxStages;
using linear::kTileThreads;
using linear::kWideBytes;

constexpr uint32_t kScaleBytes = 2 * kMxTileBytes;     // 128 rows, one stage
constexpr int32_t kSliceK = 256;                       // values of a stage

struct TileParams {
    linear::TileParams t;                              // maps, epilogue, split; num_ks: stages' worth of K
    CUtensorMap mapWs, mapXs;                          // scales
    int32_t blocks;
    uint32_t prefetch;                                 // B into L2 while the launch in front still runs
};

// Row tiles of 128 whose scales a tile of BT rows needs.
__host__ __device__ constexpr uint32_t tile_row_tiles(int32_t bt) { return bt > 128 ? 2u : 1u; }
__host__ __device__ constexpr uint32_t tile_stage_bytes(int32_t bt) {
    return kWideBytes + uint32_t(bt) * 128u + kScaleBytes * (1u + tile_row_tiles(bt));
}
// Tensor Memory: the accumulator, then two sets of scales (8 columns for B, 8 or 16 for A).
__host__ __device__ constexpr uint32_t tile_scale_col(int32_t bt) { return bt < 32 ? 32u : (uint32_t(bt) + 31u) / 32u * 32u; }
__host__ __device__ constexpr uint32_t tile_tmem_cols(int32_t bt) {
    const uint32_t need = tile_scale_col(bt) + 2u * 8u * (1u + tile_row_tiles(bt));
    return need <= 64u ? 64u : need <= 128u ? 128u : need <= 256u ? 256u : 512u;
}
// As for linear_tile.cuh never below 108 KiB; tiles that take all of Tensor
// Memory never share an SM with another that waits for some.
__host__ __device__ constexpr size_t tile_smem_bytes(int32_t bt, int32_t stages) {
    const size_t ring = size_t(stages) * tile_stage_bytes(bt), part = size_t(bt) * 512u;
    const size_t need = 1024 + kTileBarBytes + 1024 + (ring > part ? ring : part);
    const size_t least = tile_tmem_cols(bt) > 256u ? 124 * 1024 : 108 * 1024;
    return need > least ? need : least;
}

// High word of the matrix descriptor of 512 bytes of scales in shared memory: 32 rows of 16 bytes, groups of 8 rows
// 128 bytes apart, no swizzle (bit layout: see sw128_desc in gemm_umma.cuh).
constexpr uint32_t kScaleDescHi = (128u >> 4) | (1u << 14);
// fp32 += e2m1 x e2m1 with E8M0 scales; `m` and `n` the MMA's shape, `pair` (0 or 1) which two of four scale bytes.
__host__ __device__ constexpr uint32_t mx_idesc(uint32_t m, uint32_t n, uint32_t pair) {
    return (pair * 2u << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (1u << 23) | ((m >> 4) << 24) |
           (pair * 2u << 29);
}

// Eight neighbouring outputs of the tile's rows t0, t0 + step, ... below `rows`, TURN rows at a time so that their loads
// are under way together; `sum` gives A B^T.  (Row by row, with the bias read for each, a tile of 128 rows took 1.5 us
// more for a bias, 1.3 for a residual: 128 x 800 x 152 with both and GELU 9.2 us, this 5.7; 256 x 8192 x 8192 27.6 / 19.1.)
template <int ACT, int TURN, typename F>
__device__ __forceinline__ void finish_rows(const linear::TileParams& P, int32_t i0, int32_t j, const float (&bias)[8],
                                            int32_t t0, int32_t rows, int32_t step, F&& sum) {
    const int32_t left = P.J - j;                      // >= 1 columns inside
    const bool whole = P.vec != 0 && left >= 8;
    for (int32_t t = t0; t < rows; t += TURN * step) {
        uint4 r[TURN];
        float v[TURN][8];
#pragma unroll
        for (int k = 0; k < TURN; ++k) {
            const int32_t u = t + k * step;
            r[k] = make_uint4(0, 0, 0, 0);
            if (u >= rows || P.R == nullptr) continue;
            const __nv_bfloat16* from = P.R + int64_t(i0 + u) * P.ldr + j;
            r[k] = whole ? *reinterpret_cast<const uint4*>(from) : load8_raw(from, left);
        }
#pragma unroll
        for (int k = 0; k < TURN; ++k)
            if (t + k * step < rows) sum(t + k * step, v[k]);
#pragma unroll
        for (int k = 0; k < TURN; ++k) {
            const int32_t u = t + k * step;
            if (u >= rows) break;
            float w[8];
            unpack8(r[k], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] += bias[e];
#pragma unroll
            for (int e = 0; e < 8; e += 2) act_value2<ACT>(v[k][e], v[k][e + 1]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] += w[e];
            __nv_bfloat16* c = P.C + int64_t(i0 + u) * P.ldc + j;
            if (whole) {
                store8(c, v[k]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < left) c[e] = __float2bfloat16_rn(v[k][e]);
            }
        }
    }
}

template <int ACT>
__global__ void __launch_bounds__(kTileThreads) mxfp4_tile_kernel(const __grid_constant__ TileParams Q) {
    extern __shared__ uint8_t smem_raw[];
    const linear::TileParams& P = Q.t;
    uint64_t* full = reinterpret_cast<uint64_t*>(align_1024(smem_raw));
    uint64_t* empty = full + kTileMaxStages;
    uint64_t* acc_full = empty + kTileMaxStages;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_full + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    uint8_t* ring = align_1024(reinterpret_cast<uint8_t*>(full) + kTileBarBytes);

    const uint32_t warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31u;
    const uint32_t S = uint32_t(P.split), stages = uint32_t(P.stages);
    const uint32_t tile = blockIdx.x / S, rank = blockIdx.x % S;
    const int32_t i0 = int32_t(tile % uint32_t(P.t_tiles)) * P.bt, j0 = int32_t(tile / uint32_t(P.t_tiles)) * 128;
    const int32_t ks0 = int32_t(int64_t(P.num_ks) * rank / S), ks1 = int32_t(int64_t(P.num_ks) * (rank + 1) / S);
    const uint32_t stage_bytes = tile_stage_bytes(P.bt), row_tiles = tile_row_tiles(P.bt);
    const uint32_t tmem_cols = tile_tmem_cols(P.bt);

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
        ptx::prefetch_tensormap(&Q.mapWs);
        ptx::prefetch_tensormap(&Q.mapXs);
    }
    // B does not come from the launch in front, as A mostly does (just quantised): its way from HBM need not wait.
    if (threadIdx.x == 128 && Q.prefetch != 0 && i0 == 0)
        for (int32_t ks = ks0; ks < ks1; ++ks) {
            ptx::tma_prefetch_2d(&P.mapW, ks * 128, j0);
            ptx::tma_prefetch_2d(&Q.mapWs, ks * 256, j0 / 128);
        }
    if (warp == 5) {
        ptx::tmem_alloc(ptx::smem_addr(tmem_holder), tmem_cols);
        ptx::tmem_relinquish_alloc_permit();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
    const uint32_t ring_base = ptx::smem_addr(ring);
    ptx::griddep_wait();

    uint32_t issued = 0;
    if (warp == 4 && lane == 0) {
        uint32_t slot = 0, ph = 0;
        for (int32_t ks = ks0; ks < ks1; ++ks, ++issued) {
            if (!mbar_wait(ptx::smem_addr(empty + slot), ph ^ 1u, P.ctl, abort_flag, kSiteProducerEmpty, issued))
                break;
            const uint32_t bar = ptx::smem_addr(full + slot), dst = ring_base + slot * stage_bytes;
            const uint32_t scales = dst + kWideBytes + uint32_t(P.bt) * 128u;
            ptx::mbar_arrive_expect_tx(bar, stage_bytes);
            if (!inject_skip(P.inject, issued)) {       // self test: the stage's loads are left out
                ptx::tma_load_2d(dst, &P.mapW, bar, ks * 128, j0);
                ptx::tma_load_2d(dst + kWideBytes, &P.mapX, bar, ks * 128, i0);
                ptx::tma_load_2d(scales, &Q.mapWs, bar, ks * 256, j0 / 128);
                ptx::tma_load_2d(scales + kScaleBytes, &Q.mapXs, bar, ks * 256, i0 / 128);
            }
            if (++slot == stages) {
                slot = 0;
                ph ^= 1u;
            }
        }
        ptx::griddep_launch_dependents();
    } else if (warp == 5) {
        const uint32_t idesc0 = mx_idesc(128, uint32_t(P.bt), 0), idesc1 = mx_idesc(128, uint32_t(P.bt), 1);
        constexpr uint32_t hi = desc_hi(1024), s_hi = kScaleDescHi;
        const uint32_t w_first = desc_lo(ring_base, 16), x_first = desc_lo(ring_base + kWideBytes, 16);
        const uint32_t s_first = desc_lo(ring_base + kWideBytes + uint32_t(P.bt) * 128u, 0);
        const uint32_t sf = tmem + tile_scale_col(P.bt), set = 8u * (1u + row_tiles), count = uint32_t(ks1 - ks0);
        const uint32_t x_col = uint32_t(i0 % 128) / 32u;   // a tile may start at row 64 of 128; an odd column faults
        auto copy_scales = [&](uint32_t slot, uint32_t it) {
            const uint32_t from = s_first + slot * (stage_bytes / 16), to = sf + (it & 1u) * set;
            if (row_tiles == 2) mx_copy_scales<1, 2>(from, s_hi, to, to + 8u);
            else mx_copy_scales<1, 1>(from, s_hi, to, to + 8u);
        };
        uint32_t slot = 0, ph = 0, copied = 0;
        for (uint32_t it = 0; it < count; ++it) {
            const bool wait = copied == it;
            if (wait && !mbar_wait_warp(ptx::smem_addr(full + slot), ph, P.ctl, abort_flag, kSiteMmaFull, it)) break;
            // The next stage's scales, if it is there, in front of this one's MMAs.
            const uint32_t next = slot + 1 == stages ? 0 : slot + 1, next_ph = next == 0 ? ph ^ 1u : ph;
            const bool ahead =
                it + 1 < count && __all_sync(0xffffffffu, mbar_test<false>(ptx::smem_addr(full + next), next_ph));
            ptx::tc_fence_after_sync();
            if (ptx::elect_one()) {
                const uint32_t at = slot * (stage_bytes / 16), sfw = sf + (it & 1u) * set, sfx = sfw + 8u + x_col;
                // Pairs of blocks that the matrix has.
                const int32_t steps = min(4, (Q.blocks - (ks0 + int32_t(it)) * 8 + 1) / 2);
                if (wait) copy_scales(slot, it);
                if (ahead) copy_scales(next, it + 1);
                if (row_tiles == 2) mx_mmas<1, 2>(steps, tmem, w_first + at, x_first + at, hi, sfw, sfx, idesc0, idesc1, it);
                else mx_mmas<1, 1>(steps, tmem, w_first + at, x_first + at, hi, sfw, sfx, idesc0, idesc1, it);
                ptx::mma_commit(ptx::smem_addr(empty + slot));
            }
            __syncwarp();
            copied = it + (ahead ? 2u : 1u);
            slot = next;
            ph = next_ph;
        }
        // Completes when every MMA issued has: also what the exit path waits for.
        if (ptx::elect_one()) ptx::mma_commit(ptx::smem_addr(acc_full));
    }
    __syncwarp();

    // Every row of the output that this thread finishes has these eight columns.
    static_assert(kTileThreads % 16 == 0);
    const int32_t j = j0 + int32_t(threadIdx.x & 15u) * 8;
    float bias[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = P.bias != nullptr && j + e < P.J ? __ldg(P.bias + j + e) : 0.f;

    // All MMAs of this CTA are done: their operands' memory may be reused.
    const bool done = mbar_wait_warp(ptx::smem_addr(acc_full), 0, P.ctl, abort_flag, kSiteEpiAccFull, 0);
    ptx::tc_fence_after_sync();
    const int32_t rows = min(P.bt, P.I - i0);
    if (warp < 4 && done) {
        // Part of the tile: [row][128 columns] fp32.
        float* part = reinterpret_cast<float*>(ring) + warp * 32u + lane;
        for (int32_t c = 0; c < rows; c += 32) {       // (the second half may be scales, which are not kept)
            uint32_t r[2][16];
            ptx::tmem_ld_32x32b_x16(tmem + ((warp * 32u) << 16) + uint32_t(c), r[0]);
            ptx::tmem_ld_32x32b_x16(tmem + ((warp * 32u) << 16) + uint32_t(c) + 16u, r[1]);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (h == 0 || c + 16 < rows)
#pragma unroll
                    for (int e = 0; e < 16; ++e) part[(c + 16 * h + e) * 128] = ks1 > ks0 ? __uint_as_float(r[h][e]) : 0.f;
        }
    }
    ptx::tc_fence_before_sync();
    __syncwarp();
    if (S > 1)
        ptx::cluster_sync_all();
    else
        __syncthreads();
    // After an abort loads may still be in flight; no part is complete then.
    if (*abort_flag) {
        if (warp == 5 && lane == 0) mbar_wait_drain(ptx::smem_addr(acc_full), 0, P.ctl.timeout_ns);
        if (warp == 4 && lane == 0)
            umma::drain_ring<1>(full, stages, issued, 0, stage_bytes, P.inject, blockIdx.x, P.ctl.timeout_ns);
    } else {
        const int32_t t0 = int32_t(rank * kTileThreads + threadIdx.x) / 16, step = int32_t(S * kTileThreads / 16);
        const uint32_t at = ring_base + (threadIdx.x & 15u) * 32u;
        if (j >= P.J) {
        } else if (S == 1) {
            finish_rows<ACT, 4>(P, i0, j, bias, t0, rows, step, [&](int32_t t, float (&v)[8]) {
                const uint4 x = ptx::ld_shared_v4(at + uint32_t(t) * 512u), y = ptx::ld_shared_v4(at + uint32_t(t) * 512u + 16u);
                v[0] = __uint_as_float(x.x), v[1] = __uint_as_float(x.y), v[2] = __uint_as_float(x.z);
                v[3] = __uint_as_float(x.w), v[4] = __uint_as_float(y.x), v[5] = __uint_as_float(y.y);
                v[6] = __uint_as_float(y.z), v[7] = __uint_as_float(y.w);
            });
        } else {
            finish_rows<ACT, 1>(P, i0, j, bias, t0, rows, step, [&](int32_t t, float (&v)[8]) {
                // Every part's load is under way before the first is added.
                float4 a[8], b[8];
#pragma unroll
                for (uint32_t s = 0; s < 8; ++s)
                    if (s < S) {
                        const uint32_t from = ptx::mapa_shared(at + uint32_t(t) * 512u, s);
                        a[s] = ptx::ld_shared_cluster_v4_f32(from);
                        b[s] = ptx::ld_shared_cluster_v4_f32(from + 16);
                    }
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll
                for (uint32_t s = 0; s < 8; ++s)
                    if (s < S) {
                        v[0] += a[s].x, v[1] += a[s].y, v[2] += a[s].z, v[3] += a[s].w;
                        v[4] += b[s].x, v[5] += b[s].y, v[6] += b[s].z, v[7] += b[s].w;
                    }
            });
        }
    }
    __syncwarp();
    if (S > 1)
        ptx::cluster_sync_all();   // no CTA leaves while a peer may read its part
    else
        __syncthreads();
    if (warp == 5) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, tmem_cols);
    }
}

}  // namespace mx
}  // namespace gbr
