// linear_pair.cuh -- the fused linear layer and its gradients' products on
// CTA pairs: the persistent warp-specialised tcgen05 pipeline of
// gemm_umma.cuh (256 x 256 tiles, cta_group::2, a 3-slot ring of 128-K stages,
// two accumulators in Tensor Memory) for operands of either orientation and
// with another epilogue.
//
//   product            first operand        second operand
//   C  = A B           A  K-major           B  MN-major
//   dA = dZ B^T        dZ K-major           B  K-major
//   dB = A^T dZ        A  MN-major          dZ MN-major
//
// A K-major operand is loaded as one box of 128 rows x 64 k; an MN-major one,
// whose rows run along k, as two panels of 64 k rows x 64 columns: 16 KiB a
// CTA and 64-k slice either way, and the matrix descriptors and the
// instruction descriptor's transpose bits say which.  No operand is copied.
//
// Epilogue, 16 warps, each 32 rows x 64 columns of a tile, 32 columns at a time:
//   tcgen05.ld -> + bias -> (Z: round, stage, TMA store) -> activation ->
//   dropout -> + residual -> round, stage, TMA store
// through one 2 KiB staging slot a warp; the residual arrives by TMA in the
// very slot that the result then overwrites.  The chain from the accumulator
// to the store is long and its parts wait for one another, so it takes warps,
// four a scheduler, to keep it going.  GELU with Z, 4 / 8 / 16 warps: 4096 x
// 4096 x 14336 324 / 268 / 265 us (253 without an epilogue), 8192 x 64 x 14336,
// where it decides, - / 145 / 125 us.

// Split tail: where the last, partial round has tiles for at most half of the
// pairs, each of those tiles is cut in two along K and given to two pairs.  A
// part goes to scratch; whoever finishes second adds the other's part to its
// own accumulator and runs the epilogue.  Nobody waits, and since a + b = b + a
// the result does not depend on who was second.
#pragma once
#include "gemm_umma.cuh"
#include "operators.h"

namespace gbr {
namespace linear {

using umma::kAccCols;
using umma::kTmemCols;
using umma::sw128_desc;

constexpr uint32_t kTile = 256;                        // rows and columns of a tile
constexpr uint32_t kStages = 3, kSlices = 2;           // 64-k slices per ring stage
constexpr uint32_t kSliceBytes = 128 * 128;            // one operand, one CTA, 64 k
constexpr uint32_t kStageBytes = 2 * kSlices * kSliceBytes;
constexpr uint32_t kPanelBytes = 64 * 128;
constexpr uint32_t kBarBytes = 256;
constexpr size_t kSmemBytes = 1024 + kStages * kStageBytes + kUmmaEpiBytes + kBarBytes;
constexpr int kThreads = 640;                          // 4 warps of roles, 16 of the epilogue
constexpr uint32_t kEpiWarps = 16;
constexpr uint32_t kSlotBytes = 32 * 64;               // 32 rows x 32 columns
static_assert(kEpiWarps * kSlotBytes == kUmmaEpiBytes, "one staging slot a warp");
// fp32 parts of split tiles: per tile, part, CTA of the pair and warp 32 rows x
// 64 columns as [column / 4][row] float4; before them one arrival count per
// tile, CTA and warp, zeroed.
constexpr int64_t kPartVecs = 16 * 32;
inline size_t pair_count_bytes(int64_t split_tiles) { return size_t(split_tiles) * 2 * kEpiWarps * 4; }
inline size_t pair_part_bytes(int64_t split_tiles) { return size_t(split_tiles) * 4 * kEpiWarps * kPartVecs * 16; }

// The work of a product on `units` pairs: tiles 0 .. whole - 1 in rounds, then
// (if split > 0) the last `split` tiles in halves.
struct PairWork {
    int32_t m_tiles, n_tiles, num_tiles, num_kb, group_m;
    int32_t whole, split;
    uint32_t* count;
    float4* parts;
};

struct PairItem {
    uint32_t tile;
    int32_t kb0, kb1;
    int32_t part;                                      // 0 or 1 of a split tile, -1: whole
    int32_t sk;                                        // split tile
};

// Item j of a pair; every role walks the same sequence.
__device__ __forceinline__ bool pair_item(const PairWork& w, uint32_t unit, uint32_t units, uint32_t j, PairItem& x) {
    x.tile = unit + j * units;
    x.kb0 = 0;
    x.kb1 = w.num_kb;
    x.part = -1;
    x.sk = 0;
    if (x.tile < uint32_t(w.whole)) return true;
    if (w.split == 0 || unit >= 2u * uint32_t(w.split) || j != uint32_t(w.whole) / units) return false;
    x.sk = int32_t(unit / 2u);
    x.tile = uint32_t(w.whole + x.sk);
    x.part = int32_t(unit & 1u);
    if (x.part == 0) x.kb1 = w.num_kb / 2;
    else x.kb0 = w.num_kb / 2;
    return true;
}

struct PairParams {
    CUtensorMap mapA, mapB, mapC, mapZ, mapR;
    const float* bias;
    int32_t M, N;                                      // of the output
    PairWork w;
    uint32_t has_z, has_r;
    uint32_t bias_vec;                                 // bias starts on 16 bytes
    Dropout drop;
    KernelCtl ctl;
    FaultInjection inject;                             // self test only
};

template <bool A_MN, bool B_MN>
__host__ __device__ constexpr uint32_t pair_idesc() {
    return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(A_MN) << 15) | (uint32_t(B_MN) << 16) |
           ((kTile >> 3) << 17) | ((kTile >> 4) << 24);
}

template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t slice, uint32_t k) {
    return MN ? sw128_desc(slice + k * 16u * 128u, kPanelBytes, 1024)
              : sw128_desc(slice + k * 32u, 16, 1024);
}

// One 64-k slice of an operand: this CTA's 128 rows (or columns) from `r0`.
template <bool MN>
__device__ __forceinline__ void load_slice(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                           int32_t r0, int32_t k0) {
    if (MN) {
        ptx::tma_load_2d_pair(dst, map, bar, r0, k0);
        ptx::tma_load_2d_pair(dst + kPanelBytes, map, bar, r0 + 64, k0);
    } else {
        ptx::tma_load_2d_pair(dst, map, bar, k0, r0);
    }
}

template <bool A_MN, bool B_MN, int ACT, bool PLAIN>
__global__ void __launch_bounds__(kThreads, 1)
    linear_pair_kernel(const __grid_constant__ PairParams P) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = align_1024(smem_raw);
    uint8_t* epi = ring + kStages * kStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(epi + kUmmaEpiBytes);
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint64_t* res_full = drain + 1;                    // [16 warps]
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(res_full + kEpiWarps);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    uint32_t* issued_word = tmem_holder + 2;

    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
    const uint32_t rank = ptx::cluster_ctarank();
    const uint32_t unit = blockIdx.x / 2, units = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kStages; ++i) {
            ptx::mbar_init(ptx::smem_addr(full + i), 1);
            ptx::mbar_init(ptx::smem_addr(empty + i), 1);
        }
        for (uint32_t a = 0; a < 2; ++a) {
            ptx::mbar_init(ptx::smem_addr(acc_full + a), 1);
            ptx::mbar_init(ptx::smem_addr(acc_empty + a), 2 * kEpiWarps);
        }
        ptx::mbar_init(ptx::smem_addr(drain), 1);
        for (uint32_t i = 0; i < kEpiWarps; ++i) ptx::mbar_init(ptx::smem_addr(res_full + i), 1);
        *abort_flag = 0;
        *issued_word = 0;
        ptx::fence_barrier_init();
    } else if (threadIdx.x == 32) {
        ptx::prefetch_tensormap(&P.mapA);
        ptx::prefetch_tensormap(&P.mapB);
        ptx::prefetch_tensormap(&P.mapC);
    }
    if (warp == 2) {
        ptx::tmem_alloc_pair(ptx::smem_addr(tmem_holder), kTmemCols);
        ptx::tmem_relinquish_alloc_permit_pair();
    }
    ptx::tc_fence_before_sync();
    ptx::cluster_sync_all();
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_holder;
    ptx::griddep_wait();
    uint32_t issued = 0;

    if (warp < 4) {
        if (warp == 0 && lane == 0) {
            // ---------------------------------------------------- TMA producer
            const uint32_t ring_base = ptx::smem_addr(ring);
            uint32_t it = 0;
            bool ok = true;
            PairItem w;
            for (uint32_t j = 0; ok && pair_item(P.w, unit, units, j, w); ++j) {
                uint32_t mt, nt;
                raster_tile(w.tile, P.w.m_tiles, P.w.n_tiles, P.w.group_m, mt, nt);
                const int32_t a0 = int32_t(mt * kTile + rank * 128), b0 = int32_t(nt * kTile + rank * 128);
                for (int32_t kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                    const uint32_t slot = it % kStages, ph = (it / kStages) & 1u;
                    if (!mbar_wait<true>(ptx::smem_addr(empty + slot), ph ^ 1u, P.ctl, abort_flag,
                                         kSiteProducerEmpty, it)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb_local = ptx::smem_addr(full + slot);
                    const uint32_t fb = ptx::mapa_shared(fb_local, 0);
                    if (rank == 0) ptx::mbar_arrive_expect_tx(fb_local, 2 * kStageBytes);
                    if (inject_skip_unit(P.inject, unit, it)) continue;   // self test
                    const uint32_t stage = ring_base + slot * kStageBytes;
#pragma unroll
                    for (uint32_t h = 0; h < kSlices; ++h) {
                        const int32_t k0 = (kb * int32_t(kSlices) + int32_t(h)) * 64;
                        load_slice<A_MN>(stage + h * kSliceBytes, &P.mapA, fb, a0, k0);
                        load_slice<B_MN>(stage + (kSlices + h) * kSliceBytes, &P.mapB, fb, b0, k0);
                    }
                }
            }
            ptx::griddep_launch_dependents();
            issued = it;
            *issued_word = it;
        } else if (warp == 1 && lane == 0 && rank == 0) {
            // ---------------------------------------------------- MMA issuer
            const uint32_t ring_base = ptx::smem_addr(ring);
            constexpr uint32_t idesc = pair_idesc<A_MN, B_MN>();
            uint32_t it = 0, tl = 0;
            bool ok = true;
            PairItem w;
            for (; ok && pair_item(P.w, unit, units, tl, w); ++tl) {
                const uint32_t a = tl & 1u, aph = (tl >> 1) & 1u;
                if (!mbar_wait<true>(ptx::smem_addr(acc_empty + a), aph ^ 1u, P.ctl, abort_flag,
                                     kSiteMmaAccEmpty, tl))
                    break;
                ptx::tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + a * kAccCols;
                for (int32_t kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                    const uint32_t slot = it % kStages, ph = (it / kStages) & 1u;
                    if (!mbar_wait<true>(ptx::smem_addr(full + slot), ph, P.ctl, abort_flag,
                                         kSiteMmaFull, it)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after_sync();
                    const uint32_t stage = ring_base + slot * kStageBytes;
#pragma unroll
                    for (uint32_t h = 0; h < kSlices; ++h)
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k)
                            ptx::mma_f16_pair(d_tmem, operand_desc<A_MN>(stage + h * kSliceBytes, k),
                                              operand_desc<B_MN>(stage + (kSlices + h) * kSliceBytes, k),
                                              idesc, (kb != w.kb0 || h != 0 || k != 0) ? 1u : 0u);
                    ptx::mma_commit_pair_multicast(ptx::smem_addr(empty + slot), 0x3);
                }
                if (!ok) break;
                if (w.kb1 > w.kb0) {
                    ptx::mma_commit_pair_multicast(ptx::smem_addr(acc_full + a), 0x3);
                } else {
                    ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_addr(acc_full + a), 0));
                    ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_addr(acc_full + a), 1));
                }
            }
            ptx::mma_commit_pair_multicast(ptx::smem_addr(drain), 0x1);
            mbar_wait_drain(ptx::smem_addr(drain), 0, P.ctl.timeout_ns);
        }
    } else {
        // -------------------------------------------------------- epilogue
        const uint32_t q = warp & 3u, ew = warp - 4u;  // TMEM lane quarter; epilogue warp
        const int32_t col0 = int32_t(ew / 4u) * 64;    // first of this warp's columns in the tile
        const uint32_t slot = ptx::smem_addr(epi) + ew * kSlotBytes;
        const uint32_t res_bar = ptx::smem_addr(res_full + ew);
        const uint32_t row_off = lane * 64u, swz = (lane >> 1) & 3u;   // 64-byte swizzle
        const bool has_z = !PLAIN && P.has_z != 0, has_r = !PLAIN && P.has_r != 0;
        uint32_t res_issued = 0, res_taken = 0;
        bool ok = true;
        PairItem w;
        for (uint32_t tl = 0; ok && pair_item(P.w, unit, units, tl, w); ++tl) {
            uint32_t mt, nt;
            raster_tile(w.tile, P.w.m_tiles, P.w.n_tiles, P.w.group_m, mt, nt);
            const int32_t row0 = int32_t(mt * kTile + rank * 128u + q * 32u), n0 = int32_t(nt * kTile) + col0;
            // 32-column chunks that hold something.
            const int32_t chunks = row0 < P.M && n0 < P.N ? min(2, (P.N - n0 + 31) / 32) : 0;
            const uint32_t a = tl & 1u, aph = (tl >> 1) & 1u;
            const uint32_t ae = ptx::smem_addr(acc_empty + a);
            // The residual of a chunk, into the staging slot once its last store has read it.
            auto fetch_residual = [&](int32_t c) {
                if (lane == 0) {
                    ptx::bulk_wait_group_read<0>();
                    ptx::mbar_arrive_expect_tx(res_bar, kSlotBytes);
                    ptx::tma_load_2d(slot, &P.mapR, res_bar, n0 + c * 32, row0);
                }
                ++res_issued;
            };
            const bool early = has_r && !has_z && w.part < 0 && chunks > 0;
            if (early) fetch_residual(0);
            if (!mbar_wait_warp<true>(ptx::smem_addr(acc_full + a), aph, P.ctl, abort_flag,
                                      kSiteEpiAccFull, tl))
                break;
            ptx::tc_fence_after_sync();
            const uint32_t acc = tmem_base + ((q * 32u) << 16) + a * kAccCols + uint32_t(col0);
            if (chunks == 0) {
                umma::acc_release<2>(ae, lane);
                continue;
            }
            const float4* other = nullptr;             // the other half of a split tile: this warp's block
            if (w.part >= 0) {
                const int64_t half = 2 * kEpiWarps * kPartVecs;
                float4* blk = P.w.parts + (int64_t(w.sk) * 4 * kEpiWarps + rank * kEpiWarps + ew) * kPartVecs + lane;
                uint32_t* count = P.w.count + (uint32_t(w.sk) * 2u + rank) * kEpiWarps + ew;
                float4* mine = blk + w.part * half;
                for (int32_t c = 0; c < chunks; ++c) {
                    uint32_t x[32];
                    ptx::tmem_ld_32x32b_x32(acc + uint32_t(c * 32), x);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        mine[(c * 8 + v) * 32] =
                            make_float4(__uint_as_float(x[4 * v]), __uint_as_float(x[4 * v + 1]),
                                        __uint_as_float(x[4 * v + 2]), __uint_as_float(x[4 * v + 3]));
                }
                __threadfence();
                __syncwarp();
                uint32_t before = 0;
                if (lane == 0) before = atomicAdd(count, 1u);
                if (__shfl_sync(0xffffffffu, before, 0) == 0u) {
                    umma::acc_release<2>(ae, lane);    // the other pair finishes the tile
                    continue;
                }
                __threadfence();
                other = blk + (1 - w.part) * half;
            }
            if (has_r && !has_z && !early) fetch_residual(0);
            for (int32_t c = 0; c < chunks; ++c) {
                float z[32];
                {
                    uint32_t raw[32];
                    ptx::tmem_ld_32x32b_x32(acc + uint32_t(c) * 32u, raw);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(raw[j]);
                    if (w.kb1 == w.kb0) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) z[j] = 0.f;
                    }
                }
                if (other != nullptr) {
                    float4 x[8];
#pragma unroll
                    for (int v = 0; v < 8; ++v) x[v] = __ldcg(other + (c * 8 + v) * 32);
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        z[4 * v] += x[v].x, z[4 * v + 1] += x[v].y, z[4 * v + 2] += x[v].z, z[4 * v + 3] += x[v].w;
                }
                if (c + 1 == chunks) umma::acc_release<2>(ae, lane);
                if (!PLAIN && P.bias != nullptr) {
                    const int32_t n = n0 + c * 32;
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
                auto stage_and_store = [&](const CUtensorMap* map) {
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
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::tma_store_2d(map, slot, n0 + c * 32, row0);
                        ptx::bulk_commit_group();
                    }
                };
                if (has_z) {
                    if (lane == 0) ptx::bulk_wait_group_read<0>();
                    __syncwarp();
                    stage_and_store(&P.mapZ);
                    if (has_r) fetch_residual(c);      // while the activation is computed
                }
                if (!PLAIN) {
#pragma unroll
                    for (int j = 0; j < 32; j += 2) act_value2<ACT>(z[j], z[j + 1]);
                }
                if (!PLAIN && P.drop.threshold != 0) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const uint4 bits = dropout_bits(P.drop, uint32_t(row0) + lane,
                                                        uint32_t(n0 + c * 32) / 8u + uint32_t(g));
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            z[8 * g + i] = dropout_keep(P.drop, bits, i) ? z[8 * g + i] * P.drop.scale : 0.f;
                    }
                }
                if (has_r) {
                    if (!mbar_wait_warp(res_bar, res_taken & 1u, P.ctl, abort_flag, kSiteEpiResidual, tl)) {
                        ok = false;
                        break;
                    }
                    ++res_taken;
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
                } else {
                    if (lane == 0) ptx::bulk_wait_group_read<0>();
                    __syncwarp();
                }
                stage_and_store(&P.mapC);
                if (has_r && !has_z && c + 1 < chunks) fetch_residual(c + 1);
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
            umma::drain_ring<2>(full, kStages, issued, peer, kStageBytes, P.inject, unit,
                                P.ctl.timeout_ns);
    }
    ptx::cluster_sync_all();
    if (warp == 2) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc_pair(tmem_base, kTmemCols);
    }
}

}  // namespace linear
}  // namespace gbr
