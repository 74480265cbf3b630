// mxfp4.cu -- host side of the 4-bit product: tensor maps, the choice of the
// kernel and the launch.
#include "mxfp4_pair.cuh"
#include "mxfp4_tile.cuh"

#include "gbr.h"

#include <algorithm>
#include <cstring>

namespace gbr {

void* mxfp4_pair_kernel_ptr(int act);
void* mxfp4_tile_kernel_ptr(int act);

namespace {

using bf16 = __nv_bfloat16;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// 128 bytes (256 values) of `box_rows` rows.
int map_data(CUtensorMap* map, const uint8_t* p, int64_t rows, int64_t blocks, uint32_t box_rows, const char* what) {
    const uint64_t dims[2] = {uint64_t(blocks) * 16, uint64_t(rows)};
    const uint64_t strides[1] = {uint64_t(blocks) * 16};
    const uint32_t box[2] = {128, box_rows};
    return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                             what);
}

// Two tiles of scales (8 blocks) of `box_rows` times 128 rows, as 32-bit words.  What lies past the end arrives as
// zeros, which are finite scales.
int map_scales(CUtensorMap* map, const uint8_t* p, int64_t rows, int64_t blocks, uint32_t box_rows, const char* what) {
    const uint64_t dims[2] = {uint64_t(cdiv(blocks, 4)) * 128, uint64_t(cdiv(rows, 128))};
    const uint64_t strides[1] = {uint64_t(cdiv(blocks, 4)) * kMxTileBytes};
    const uint32_t box[2] = {256, box_rows};
    return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_INT32, 2, p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE,
                             what);
}

// The epilogue's 32 x 32 blocks of a bf16 matrix.
int map_blocks(CUtensorMap* map, const Mat& m, int64_t rows, int64_t cols, const char* what) {
    const uint64_t dims[2] = {uint64_t(cols), uint64_t(rows)};
    const uint64_t strides[1] = {uint64_t(m.ld) * 2};
    const uint32_t box[2] = {32, 32};
    return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, m.p, dims, strides, box,
                             CU_TENSOR_MAP_SWIZZLE_64B, what);
}

bool tma_ready(const Mat& m) { return reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && m.ld % 8 == 0; }

int run_tile(const Mxfp4Args& a, const LinearPlan& plan, const LibCtx& c, cudaStream_t stream) {
    mx::TileParams Q;
    memset(&Q, 0, sizeof(Q));
    linear::TileParams& P = Q.t;
    int r;
    if (a.blocks > 0) {
        if ((r = map_data(&P.mapW, a.B, a.N, a.blocks, 128, "B")) != GBR_OK) return r;
        if ((r = map_data(&P.mapX, a.A, a.M, a.blocks, uint32_t(plan.bt), "A")) != GBR_OK) return r;
        if ((r = map_scales(&Q.mapWs, a.Bs, a.N, a.blocks, 1, "scales of B")) != GBR_OK) return r;
        if ((r = map_scales(&Q.mapXs, a.As, a.M, a.blocks, mx::tile_row_tiles(plan.bt), "scales of A")) != GBR_OK) return r;
    }
    P.bias = a.bias;
    P.R = static_cast<const bf16*>(a.R.p), P.ldr = a.R.ld;
    P.C = static_cast<bf16*>(a.C.w()), P.ldc = a.C.ld;
    P.vec = (!a.R || tma_ready(a.R)) && tma_ready(a.C);
    P.I = a.M, P.J = a.N;
    P.bt = plan.bt;
    P.t_tiles = int32_t(cdiv(a.M, plan.bt));
    P.num_ks = int32_t(cdiv(a.blocks, 8));
    P.split = plan.split;
    P.stages = int32_t(std::min<int64_t>(linear::kTileMaxStages, (plan.budget - 2304) / mx::tile_stage_bytes(plan.bt)));
    P.ctl = c.ctl;
    P.inject = c.inject;
    Q.blocks = a.blocks;
    Q.prefetch = int64_t(a.N) * a.blocks * 17 <= (int64_t(48) << 20);   // well within L2
    const size_t smem = mx::tile_smem_bytes(P.bt, P.stages);
    void* kernel = mxfp4_tile_kernel_ptr(a.act);
    if ((r = raise_kernel_smem(kernel, smem, c.device)) != GBR_OK) return r;
    if (P.t_tiles > 1 && plan.bt % 64 != 0)             // scales of tiles that start elsewhere start at odd columns
        return report_errorf(GBR_ERR_INVALID, "gemm_mxfp4: tiles of %d rows", plan.bt);
    const int64_t ctas = int64_t(P.t_tiles) * cdiv(a.N, 128) * plan.split;
    if (ctas >= (int64_t(1) << 31)) return report_errorf(GBR_ERR_INVALID, "gemm_mxfp4: too many output tiles");
    void* args[] = {&Q};
    const cudaError_t e = launch_kernel(kernel, dim3(unsigned(ctas)), linear::kTileThreads, smem, plan.split, args, stream);
    if (e != cudaSuccess) return report_cuda(e, "launching gemm_mxfp4");
    count_launch();
    return GBR_OK;
}

int run_pair(const Mxfp4Args& a, const LibCtx& c, cudaStream_t stream) {
    mx::PairParams P;
    memset(&P, 0, sizeof(P));
    int r;
    if ((r = map_data(&P.mapA, a.A, a.M, a.blocks, 128, "A")) != GBR_OK) return r;
    if ((r = map_data(&P.mapB, a.B, a.N, a.blocks, 128, "B")) != GBR_OK) return r;
    if ((r = map_scales(&P.mapAs, a.As, a.M, a.blocks, 1, "scales of A")) != GBR_OK) return r;
    if ((r = map_scales(&P.mapBs, a.Bs, a.N, a.blocks, 2, "scales of B")) != GBR_OK) return r;
    // A TMA store ends at whole 16 bytes.
    P.tma_c = tma_ready(a.C) && a.N % 8 == 0;
    P.has_r = bool(a.R);
    P.tma_r = P.has_r && tma_ready(a.R);
    P.mapC = P.mapR = P.mapA;                            // where unused
    if (P.tma_c && (r = map_blocks(&P.mapC, a.C, a.M, a.N, "C")) != GBR_OK) return r;
    if (P.tma_r && (r = map_blocks(&P.mapR, a.R, a.M, a.N, "residual")) != GBR_OK) return r;
    P.bias = a.bias;
    P.bias_vec = reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    P.R = static_cast<const bf16*>(a.R.p), P.ldr = a.R.ld;
    P.C = static_cast<bf16*>(a.C.w()), P.ldc = a.C.ld;
    P.M = a.M, P.N = a.N, P.blocks = a.blocks;
    P.m_tiles = int32_t(cdiv(a.M, mx::kTile)), P.n_tiles = int32_t(cdiv(a.N, mx::kTile));
    const int64_t tiles = int64_t(P.m_tiles) * P.n_tiles;
    if (tiles >= (int64_t(1) << 30)) return report_errorf(GBR_ERR_INVALID, "gemm_mxfp4: too many output tiles");
    P.num_tiles = int32_t(tiles);
    P.num_ks = int32_t(cdiv(a.blocks, 8));
    // Tiles that run together share what they read: all of B's columns against the same rows of A where B stays in L2
    // from one row of tiles to the next (us with bands of 1 / 8 rows of tiles: 4096 x 4096 x 14336 79.6 / 83.5, 8192^3
    // 161 / 168, 4096 x 16384 x 14336, B 117 MB, 315 / 273), else all of A's rows against the same of B where A does (the
    // last one: 270), else bands.
    constexpr int64_t kStays = int64_t(48) << 20;
    P.group_m = int64_t(a.N) * a.blocks * 17 <= kStays ? 1 : int64_t(a.M) * a.blocks * 17 <= kStays ? P.m_tiles : 8;
    P.ctl = c.ctl;
    P.inject = c.inject;
    void* kernel = mxfp4_pair_kernel_ptr(a.act);
    if ((r = raise_kernel_smem(kernel, mx::kPairSmemBytes, c.device)) != GBR_OK) return r;
    void* args[] = {&P};
    const int64_t units = std::min<int64_t>(c.sm_count / 2, tiles);
    const cudaError_t e =
        launch_kernel(kernel, dim3(unsigned(2 * units)), mx::kPairThreads, mx::kPairSmemBytes, 2, args, stream);
    if (e != cudaSuccess) return report_cuda(e, "launching gemm_mxfp4");
    count_launch();
    return GBR_OK;
}

}  // namespace

int launch_mxfp4(const Mxfp4Args& a, const LibCtx& c, cudaStream_t stream) {
    // In bytes of operands and in cycles of the tensor core a contraction of 4-bit values is one of a quarter as many
    // bf16 values, so the same estimate serves: over 21 products of 100 to 2048 rows and 640 to 14336 columns it picks what
    // is 3 % slower in the mean than the best of all tiles and splits, and 15 % at worst (346 x 6688 x 6072: 18.1 / 15.7 us).
    const LinearPlan plan = plan_linear(a.M, a.N, a.blocks * 8, c.sm_count);
    return plan.pair && a.blocks > 0 ? run_pair(a, c, stream) : run_tile(a, plan, c, stream);
}

}  // namespace gbr
