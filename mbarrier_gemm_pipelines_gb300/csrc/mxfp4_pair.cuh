// mxfp4_pair.cuh -- C = R + act(A B^T + bias) from microscaled 4-bit operands on
// CTA pairs: the persistent warp-specialised tcgen05 pipeline of
// linear_pair.cuh (256 x 256 tiles, cta_group::2) with 4-bit operands and their
// scales.
//
// A 128-byte slice of a row is 256 values: a stage is 128 rows of A and of B a
// CTA (32 KiB) and the scales of this CTA's 128 rows of A (1 KiB) and of all 256
// rows of B (2 KiB, in both CTAs).  The MMA's warp copies the scales to Tensor
// Memory; the tensor core runs copies and MMAs in order.  Two sets of columns
// alternate, and a stage's copies are issued in front of the MMAs of the stage
// before.
//
// That warp runs in step and one lane issues, which leaves the operands of the
// tensor core's instructions in uniform registers.  A stage, 4096 x 16384 x 14336:
// 0.46 us from a lane on a path of its own, whatever the order of the copies, 0.32
// in step; MMAs 0.27.  What is left is bound by what an SM takes in: 35 KiB a stage
// at 64 bytes a cycle are 560 cycles, the MMAs take 512.
//
// Tensor Memory: two accumulators of 256 columns would leave nothing for the
// scales, and one would leave the tensor core idle during a tile's epilogue.  So
// the two share 64 columns: [0, 256) and [192, 448), scales in [448, 512).  The
// epilogue takes the shared columns of its tile first, and the next tile's MMAs
// wait for those alone (and for the tile before, which is done by then): 0.4 us
// from one tile's last MMA to the next one's first, of 6.2 at K = 4096.  (1.1 us
// with arrivals that release memory at cluster scope: they wait for the epilogue's
// stores.  4096 x 4096 x 14336 92 -> 84 us, GELU 99 -> 90; with the host's order of the tiles 79.5 and 88.)  Tiles of 192 columns have
// room for two accumulators, but take in more bytes for the same products: 8192^3
// 176 us with 256 columns, 196 with 192, before that.
#pragma once
#include "gemm_umma.cuh"
#include "mxfp4_tile.cuh"
#include "operators.h"

namespace gbr {
namespace mx {

constexpr uint32_t kTile = 256;
constexpr uint32_t kPairStages = 5;
constexpr uint32_t kSliceBytes = 128 * 128;            // one operand, one CTA
constexpr uint32_t kPairStageBytes = 2 * kSliceBytes + 3 * kScaleBytes;
constexpr int kPairThreads = 640;                      // 4 warps of roles, 16 of the epilogue
constexpr uint32_t kEpiWarps = 16;
constexpr uint32_t kSlotBytes = 32 * 64;               // 32 rows x 32 columns bf16
constexpr uint32_t kPairBarBytes = 512;                // 32 barriers and three words
constexpr size_t kPairSmemBytes = 1024 + kPairStages * kPairStageBytes + kEpiWarps * kSlotBytes + kPairBarBytes;
constexpr uint32_t kAccStep = 192, kScaleCol = 448, kScaleSet = 32;   // Tensor Memory columns

struct PairParams {
    CUtensorMap mapA, mapB, mapAs, mapBs, mapC, mapR;
    const float* bias;
    const __nv_bfloat16* R;
    __nv_bfloat16* C;
    int64_t ldr, ldc;
    int32_t M, N, blocks;
    int32_t m_tiles, n_tiles, num_tiles, num_ks, group_m;
    uint32_t has_r, tma_c, tma_r;                      // C and R by TMA
    uint32_t bias_vec;                                 // bias starts on 16 bytes
    KernelCtl ctl;
    FaultInjection inject;                             // self test only
};

template <int ACT>
__global__ void __launch_bounds__(kPairThreads, 1) mxfp4_pair_kernel(const __grid_constant__ PairParams P) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = align_1024(smem_raw);
    uint8_t* epi = ring + kPairStages * kPairStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(epi + kEpiWarps * kSlotBytes);
    uint64_t* empty = full + kPairStages;
    uint64_t* acc_full = empty + kPairStages;
    uint64_t* acc_empty = acc_full + 2;                // an accumulator has been read
    uint64_t* shared_empty = acc_empty + 2;            // a tile's shared columns have been read
    uint64_t* drain = shared_empty + 1;
    uint64_t* res_full = drain + 1;                    // [16 warps]
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(res_full + kEpiWarps);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    uint32_t* issued_word = tmem_holder + 2;

    const uint32_t warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31u;
    const uint32_t rank = ptx::cluster_ctarank();
    const uint32_t unit = blockIdx.x / 2, units = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kPairStages; ++i) {
            ptx::mbar_init(ptx::smem_addr(full + i), 1);
            ptx::mbar_init(ptx::smem_addr(empty + i), 1);
        }
        for (uint32_t a = 0; a < 2; ++a) {
            ptx::mbar_init(ptx::smem_addr(acc_full + a), 1);
            ptx::mbar_init(ptx::smem_addr(acc_empty + a), 2 * kEpiWarps);
        }
        ptx::mbar_init(ptx::smem_addr(shared_empty), 16);  // 8 warps a CTA hold 64 columns
        ptx::mbar_init(ptx::smem_addr(drain), 1);
        for (uint32_t i = 0; i < kEpiWarps; ++i) ptx::mbar_init(ptx::smem_addr(res_full + i), 1);
        *abort_flag = 0;
        *issued_word = 0;
        ptx::fence_barrier_init();
    } else if (threadIdx.x == 32) {
        ptx::prefetch_tensormap(&P.mapA);
        ptx::prefetch_tensormap(&P.mapB);
        ptx::prefetch_tensormap(&P.mapAs);
        ptx::prefetch_tensormap(&P.mapBs);
    }
    if (warp == 2) {
        ptx::tmem_alloc_pair(ptx::smem_addr(tmem_holder), 512);
        ptx::tmem_relinquish_alloc_permit_pair();
    }
    ptx::tc_fence_before_sync();
    ptx::cluster_sync_all();
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_holder, 0);
    ptx::griddep_wait();
    uint32_t issued = 0;

    if (warp < 4) {
        if (warp == 0 && lane == 0) {
            // ---------------------------------------------------- TMA producer
            const uint32_t ring_base = ptx::smem_addr(ring);
            uint32_t it = 0;
            bool ok = true;
            for (uint32_t tile = unit; ok && tile < uint32_t(P.num_tiles); tile += units) {
                uint32_t mt, nt;
                raster_tile(tile, P.m_tiles, P.n_tiles, P.group_m, mt, nt);
                const int32_t a0 = int32_t(mt * kTile + rank * 128), b0 = int32_t(nt * kTile + rank * 128);
                for (int32_t ks = 0; ks < P.num_ks; ++ks, ++it) {
                    const uint32_t slot = it % kPairStages, ph = (it / kPairStages) & 1u;
                    if (!mbar_wait<true>(ptx::smem_addr(empty + slot), ph ^ 1u, P.ctl, abort_flag, kSiteProducerEmpty,
                                         it)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb_local = ptx::smem_addr(full + slot);
                    const uint32_t fb = ptx::mapa_shared(fb_local, 0);
                    if (rank == 0) ptx::mbar_arrive_expect_tx(fb_local, 2 * kPairStageBytes);
                    if (inject_skip_unit(P.inject, unit, it)) continue;   // self test
                    const uint32_t stage = ring_base + slot * kPairStageBytes, scales = stage + 2 * kSliceBytes;
                    ptx::tma_load_2d_pair(stage, &P.mapA, fb, ks * 128, a0);
                    ptx::tma_load_2d_pair(stage + kSliceBytes, &P.mapB, fb, ks * 128, b0);
                    ptx::tma_load_2d_pair(scales, &P.mapAs, fb, ks * 256, a0 / 128);
                    ptx::tma_load_2d_pair(scales + kScaleBytes, &P.mapBs, fb, ks * 256, int32_t(nt) * 2);
                }
            }
            ptx::griddep_launch_dependents();
            issued = it;
            *issued_word = it;
        } else if (warp == 1 && rank == 0) {
            // ---------------------------------------------------- MMA issuer
            const uint32_t ring_base = ptx::smem_addr(ring);
            constexpr uint32_t idesc0 = mx_idesc(256, kTile, 0), idesc1 = mx_idesc(256, kTile, 1);
            constexpr uint32_t hi = desc_hi(1024), s_hi = kScaleDescHi;
            const uint32_t a_first = desc_lo(ring_base, 16), b_first = desc_lo(ring_base + kSliceBytes, 16);
            const uint32_t s_first = desc_lo(ring_base + 2 * kSliceBytes, 0);
            const uint32_t sf = tmem_base + kScaleCol;
            const uint32_t tiles = (uint32_t(P.num_tiles) - unit + units - 1) / units, count = tiles * uint32_t(P.num_ks);
            uint32_t it = 0, copied = 0, slot = 0, ph = 0;
            bool ok = true;
            for (uint32_t tl = 0; ok && tl < tiles; ++tl) {
                const uint32_t a = tl & 1u, aph = (tl >> 1) & 1u;
                if (!mbar_wait_warp<true>(ptx::smem_addr(acc_empty + a), aph ^ 1u, P.ctl, abort_flag, kSiteMmaAccEmpty,
                                          tl))
                    break;
                // The columns shared with the tile before (the first tile has none).
                if (!mbar_wait_warp<true>(ptx::smem_addr(shared_empty), (tl & 1u) ^ 1u, P.ctl, abort_flag,
                                          kSiteMmaAccEmpty, tl))
                    break;
                const uint32_t d_tmem = tmem_base + a * kAccStep;
                for (int32_t ks = 0; ks < P.num_ks; ++ks, ++it) {
                    const bool wait = copied == it;
                    if (wait && !mbar_wait_warp<true>(ptx::smem_addr(full + slot), ph, P.ctl, abort_flag, kSiteMmaFull, it)) {
                        ok = false;
                        break;
                    }
                    // The next stage's scales, if it is there, in front of this one's MMAs.
                    const uint32_t next = slot + 1 == kPairStages ? 0 : slot + 1, next_ph = next == 0 ? ph ^ 1u : ph;
                    const bool ahead = it + 1 < count &&
                                       __all_sync(0xffffffffu, mbar_test<true>(ptx::smem_addr(full + next), next_ph));
                    ptx::tc_fence_after_sync();
                    if (ptx::elect_one()) {
                        const uint32_t at = slot * (kPairStageBytes / 16), next_at = next * (kPairStageBytes / 16);
                        const uint32_t sfa = sf + (it & 1u) * kScaleSet, next_sfa = sf + (~it & 1u) * kScaleSet;
                        const int32_t steps = min(4, (P.blocks - ks * 8 + 1) / 2);
                        if (wait) mx_copy_scales<2, 2>(s_first + at, s_hi, sfa, sfa + 8u);
                        if (ahead) mx_copy_scales<2, 2>(s_first + next_at, s_hi, next_sfa, next_sfa + 8u);
                        mx_mmas<2, 2>(steps, d_tmem, a_first + at, b_first + at, hi, sfa, sfa + 8u, idesc0, idesc1,
                                      uint32_t(ks));
                        ptx::mma_commit_pair_multicast(ptx::smem_addr(empty + slot), 0x3);
                        if (ks + 1 == P.num_ks) ptx::mma_commit_pair_multicast(ptx::smem_addr(acc_full + a), 0x3);
                    }
                    __syncwarp();
                    copied = it + (ahead ? 2u : 1u);
                    slot = next;
                    ph = next_ph;
                }
            }
            if (ptx::elect_one()) {
                ptx::mma_commit_pair_multicast(ptx::smem_addr(drain), 0x1);
                mbar_wait_drain(ptx::smem_addr(drain), 0, P.ctl.timeout_ns);
            }
        }
    } else {
        // -------------------------------------------------------- epilogue
        const uint32_t q = warp & 3u, ew = warp - 4u, strip = ew / 4u;
        const int32_t col0 = int32_t(strip) * 32;      // and 128 columns on: two chunks of 32
        const uint32_t slot = ptx::smem_addr(epi) + ew * kSlotBytes;
        const uint32_t res_bar = ptx::smem_addr(res_full + ew);
        const uint32_t row_off = lane * 64u, swz = (lane >> 1) & 3u;   // 64-byte swizzle
        const bool has_r = P.has_r != 0;
        uint32_t res_issued = 0, res_taken = 0, tl = 0;
        bool ok = true;
        for (uint32_t tile = unit; ok && tile < uint32_t(P.num_tiles); tile += units, ++tl) {
            uint32_t mt, nt;
            raster_tile(tile, P.m_tiles, P.n_tiles, P.group_m, mt, nt);
            const int32_t row0 = int32_t(mt * kTile + rank * 128u + q * 32u), n0 = int32_t(nt * kTile) + col0;
            const int32_t rows = P.M - row0;
            const int32_t chunks = rows <= 0 || n0 >= P.N ? 0 : n0 + 128 >= P.N ? 1 : 2;
            const uint32_t a = tl & 1u, aph = (tl >> 1) & 1u;
            // The 64 columns shared with the other accumulator: the last of the first, the first of the second.
            const bool shares = a == 0 ? strip >= 2 : strip < 2;
            const int32_t first = a == 0 && chunks == 2 ? 1 : 0;
            // Columns that this warp has read go back to the even CTA's MMAs.
            auto release = [&](uint64_t* bar) {
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster_tmem(ptx::mapa_shared(ptx::smem_addr(bar), 0));
            };
            // The residual of a chunk, into the staging slot once its last store has read it.
            auto fetch_residual = [&](int32_t c) {
                if (P.tma_r != 0) {
                    if (lane == 0) {
                        ptx::bulk_wait_group_read<0>();
                        ptx::mbar_arrive_expect_tx(res_bar, kSlotBytes);
                        ptx::tma_load_2d(slot, &P.mapR, res_bar, n0 + c * 128, row0);
                    }
                    ++res_issued;
                }
            };
            if (has_r && chunks > 0) fetch_residual(first);
            if (!mbar_wait_warp<true>(ptx::smem_addr(acc_full + a), aph, P.ctl, abort_flag, kSiteEpiAccFull, tl)) break;
            ptx::tc_fence_after_sync();
            const uint32_t acc = tmem_base + ((q * 32u) << 16) + a * kAccStep + uint32_t(col0);
            if (chunks == 0) {
                if (shares) release(shared_empty);
                release(acc_empty + a);
                continue;
            }
            for (int32_t i = 0; i < chunks; ++i) {
                const int32_t c = i ^ first, n = n0 + c * 128;
                float z[32];
                {
                    uint32_t raw[32];
                    ptx::tmem_ld_32x32b_x32(acc + uint32_t(c) * 128u, raw);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(raw[j]);
                }
                if (i == 0 && shares) release(shared_empty);
                if (i + 1 == chunks) release(acc_empty + a);
                if (P.bias != nullptr) {
                    const float* b = P.bias + n;
                    if (P.bias_vec != 0 && n + 32 <= P.N) {
#pragma unroll
                        for (int v = 0; v < 8; ++v) {
                            const float4 x = __ldg(reinterpret_cast<const float4*>(b) + v);
                            z[4 * v] += x.x, z[4 * v + 1] += x.y, z[4 * v + 2] += x.z, z[4 * v + 3] += x.w;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (n + j < P.N) z[j] += __ldg(b + j);
                    }
                }
#pragma unroll
                for (int j = 0; j < 32; j += 2) act_value2<ACT>(z[j], z[j + 1]);
                if (has_r) {
                    if (P.tma_r != 0) {
                        if (!mbar_wait_warp(res_bar, res_taken & 1u, P.ctl, abort_flag, kSiteEpiResidual, tl)) {
                            ok = false;
                            break;
                        }
                        ++res_taken;
                    } else {
                        // Rows that TMA cannot address: a row at a time, a column a lane.
                        if (lane == 0) ptx::bulk_wait_group_read<0>();
                        __syncwarp();
                        for (int32_t r = 0; r < min(rows, 32); ++r) {
                            const uint32_t at = slot + uint32_t(r) * 64u +
                                                (((lane >> 3) ^ ((uint32_t(r) >> 1) & 3u)) << 4) + (lane & 7u) * 2u;
                            if (n + int32_t(lane) < P.N)
                                ptx::st_shared_u16(at, __bfloat16_as_ushort(P.R[int64_t(row0 + r) * P.ldr + n + int32_t(lane)]));
                        }
                        __syncwarp();
                    }
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) {
                        const uint4 v = ptx::ld_shared_v4(slot + row_off + ((j ^ swz) << 4));
                        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (uint32_t u = 0; u < 4; ++u) {
                            z[8 * j + 2 * u] += __uint_as_float(x[u] << 16);
                            z[8 * j + 2 * u + 1] += __uint_as_float(x[u] & 0xFFFF0000u);
                        }
                    }
                    __syncwarp();
                } else {
                    if (lane == 0) ptx::bulk_wait_group_read<0>();
                    __syncwarp();
                }
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) {
                    uint32_t x[4];
#pragma unroll
                    for (uint32_t u = 0; u < 4; ++u) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(z[8 * j + 2 * u], z[8 * j + 2 * u + 1]);
                        x[u] = *reinterpret_cast<const uint32_t*>(&v);
                    }
                    ptx::st_shared_v4(slot + row_off + ((j ^ swz) << 4), x[0], x[1], x[2], x[3]);
                }
                if (P.tma_c != 0) {
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::tma_store_2d(&P.mapC, slot, n, row0);
                        ptx::bulk_commit_group();
                    }
                } else {
                    __syncwarp();
                    for (int32_t r = 0; r < min(rows, 32); ++r) {
                        const uint32_t at = slot + uint32_t(r) * 64u +
                                            (((lane >> 3) ^ ((uint32_t(r) >> 1) & 3u)) << 4) + (lane & 7u) * 2u;
                        if (n + int32_t(lane) < P.N)
                            P.C[int64_t(row0 + r) * P.ldc + n + int32_t(lane)] =
                                __ushort_as_bfloat16(ptx::ld_shared_u16(at));
                    }
                    __syncwarp();
                    if (P.tma_r != 0) ptx::fence_proxy_async_smem();
                    __syncwarp();
                }
                if (has_r && i + 1 < chunks) fetch_residual(c ^ 1);
            }
        }
        if (lane == 0) {
            // After an abort a residual load may still be in flight.
            if (res_issued != res_taken) mbar_wait_drain(res_bar, res_taken & 1u, P.ctl.timeout_ns);
            ptx::bulk_wait_group<0>();
        }
    }

    __syncwarp();
    ptx::tc_fence_before_sync();
    ptx::cluster_sync_all();
    if (warp == 0 && lane == 0 && rank == 0) {
        const uint32_t flag = ptx::smem_addr(const_cast<int*>(abort_flag));
        const bool aborted = *abort_flag != 0 || ptx::ld_shared_cluster_u32(ptx::mapa_shared(flag, 1)) != 0;
        const uint32_t peer = ptx::ld_shared_cluster_u32(ptx::mapa_shared(ptx::smem_addr(issued_word), 1));
        if (aborted)
            umma::drain_ring<2>(full, kPairStages, issued, peer, kPairStageBytes, P.inject, unit, P.ctl.timeout_ns);
    }
    ptx::cluster_sync_all();
    if (warp == 2) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc_pair(tmem_base, 512);
    }
}

}  // namespace mx
}  // namespace gbr
