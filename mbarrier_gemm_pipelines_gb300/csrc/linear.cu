// linear.cu -- host side of the fused linear layer and its gradients: operands
// that TMA cannot read are re-pitched, tensor maps, the choice of the kernel
// and the launches; and the kernel of dZ and dbias.
#include "linear_pair.cuh"
#include "linear_tile.cuh"

#include "gbr.h"

#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <map>
#include <mutex>
#include <utility>

namespace gbr {

void* linear_pair_forward_kernel(int act);
void* linear_pair_da_kernel();
void* linear_pair_db_kernel();
void* linear_tile_forward_kernel(int act);
void* linear_tile_da_kernel();
void* linear_tile_db_kernel();
void* linear_tile_grads_kernel();

namespace {

using bf16 = __nv_bfloat16;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ------------------------------------------------------------ re-pitching
// dst[r, c] = src[r, c] for bf16 matrices: what TMA cannot address (a pitch or
// a start that is no multiple of 16 bytes) passes through an aligned copy.
// IN: dst has rows on 16 bytes (its padding is written with zeros), src any;
// else the other way round.  A warp takes 256 columns of a row, the any-aligned
// side two bytes a lane (whole lines), the other 16; shared memory turns one
// into the other.  4096 x 14335, 117 MB in and out: one element a thread and turn 270 us.
// The copies before a product, and those after it, are one launch (blockIdx.z
// names the copy; 2047^3 with residual and Z: 42 us with one launch a copy, 36
// together), unless their sizes differ so much that more than 4096 CTAs would
// have nothing to do (37 x 4097 and 4097 x 14335, 14,600 such: 67.7 us one by
// one and 72 together; 554 x 234 and 234 x 2359, 270: 26.6 and 24.9 of both
// gradients).
constexpr int kRepitchRows = 2;

struct Repitch {
    const bf16* src;
    bf16* dst;
    int64_t lds, ldd;
    int32_t rows, cols;
};

struct Repitches {
    Repitch of[3];
};

template <bool IN>
__global__ void __launch_bounds__(256) repitch_kernel(const __grid_constant__ Repitches all) {
    __shared__ __align__(16) uint16_t buf[8][kRepitchRows][256];
    ptx::griddep_wait();
    const Repitch& m = all.of[blockIdx.z];
    const bf16* src = m.src;
    bf16* dst = m.dst;
    const int64_t lds = m.lds, ldd = m.ldd;
    const int32_t rows = m.rows, cols = m.cols;
    const int32_t lane = int32_t(threadIdx.x) % 32, warp = int32_t(threadIdx.x) / 32, c0 = int32_t(blockIdx.x) * 256;
    const int32_t step = int32_t(gridDim.y) * 8 * kRepitchRows;
    for (int64_t r0 = (int64_t(blockIdx.y) * 8 + warp) * kRepitchRows; r0 < rows; r0 += step) {
        const int32_t n = int32_t(rows - r0 < kRepitchRows ? rows - r0 : kRepitchRows);
        const uint16_t* s = reinterpret_cast<const uint16_t*>(src) + r0 * lds + c0;
        uint16_t* d = reinterpret_cast<uint16_t*>(dst) + r0 * ldd + c0;
        if (IN) {
            uint16_t v[kRepitchRows][8];
#pragma unroll
            for (int i = 0; i < kRepitchRows; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i][j] = i < n && c0 + lane + 32 * j < cols ? __ldg(s + i * lds + lane + 32 * j) : uint16_t(0);
#pragma unroll
            for (int i = 0; i < kRepitchRows; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) buf[warp][i][lane + 32 * j] = v[i][j];
            __syncwarp();
            for (int i = 0; i < n; ++i)
                if (c0 + 8 * lane < cols)
                    *reinterpret_cast<uint4*>(d + i * ldd + 8 * lane) =
                        *reinterpret_cast<const uint4*>(&buf[warp][i][8 * lane]);
        } else {
            for (int i = 0; i < n; ++i)
                if (c0 + 8 * lane < cols)
                    *reinterpret_cast<uint4*>(&buf[warp][i][8 * lane]) =
                        *reinterpret_cast<const uint4*>(s + i * lds + 8 * lane);
            __syncwarp();
            for (int i = 0; i < n; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c0 + lane + 32 * j < cols) d[i * ldd + lane + 32 * j] = buf[warp][i][lane + 32 * j];
        }
        __syncwarp();
    }
}

// Copies collected for a launch.
struct RepitchList {
    Repitches all = {};
    dim3 grid[3];                  // each copy's own
    int n = 0;

    void add(Mat src, Mat dst, int32_t rows, int32_t cols) {
        all.of[n] = {static_cast<const bf16*>(src.p), static_cast<bf16*>(dst.w()), src.ld, dst.ld, rows, cols};
        grid[n++] = dim3(unsigned(cdiv(cols, 256)),
                         unsigned(std::min<int64_t>(cdiv(rows, 8 * kRepitchRows), 4096)));
    }
    int launch(bool in, cudaStream_t stream) {
        if (n == 0) return GBR_OK;
        dim3 over(1, 1, unsigned(n));
        double busy = 0;
        for (int i = 0; i < n; ++i) {
            over.x = std::max(over.x, grid[i].x);
            over.y = std::max(over.y, grid[i].y);
            busy += double(grid[i].x) * grid[i].y;
        }
        if (double(over.x) * over.y * n - busy <= 4096.0) return launch(all, over, in, stream);
        for (int i = 0; i < n; ++i) {
            const int r = launch({{all.of[i]}}, grid[i], in, stream);
            if (r != GBR_OK) return r;
        }
        return GBR_OK;
    }

private:
    static int launch(Repitches some, dim3 ctas, bool in, cudaStream_t stream) {
        void* args[] = {&some};
        const cudaError_t e = launch_kernel(in ? reinterpret_cast<void*>(&repitch_kernel<true>)
                                               : reinterpret_cast<void*>(&repitch_kernel<false>),
                                            ctas, 256, 0, 1, args, stream);
        if (e != cudaSuccess) return report_cuda(e, "launching the re-pitching copy");
        count_launch();
        return GBR_OK;
    }
};

bool tma_ready(const Mat& m) {
    return reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && m.ld % 8 == 0;
}

// The pitch of a single row is never stepped over: one that TMA takes.
void one_row(Mat* m, int32_t rows, int32_t cols) {
    if (rows == 1) m->ld = cdiv(cols, 8) * 8;
}

// Makes `m` readable by TMA (copy_in) or writable: itself, or an aligned copy.
// A TMA store ends at whole 16 bytes: measured, a row of 201 bf16 columns takes
// 7 columns of its pitch's padding along, so an output whose rows end inside
// 16 bytes is written to a copy and copied back.
int aligned_mat(Mat* m, int32_t rows, int32_t cols, bool copy_in, Scratch& ws, RepitchList* copies) {
    one_row(m, rows, cols);
    if (tma_ready(*m) && (copy_in || cols % 8 == 0)) return GBR_OK;
    Mat t;
    t.ld = cdiv(cols, 8) * 8;
    void* p = nullptr;
    const int r = ws.take(size_t(rows) * size_t(t.ld) * 2, "cudaMallocFromPoolAsync(aligned operand)", &p);
    if (r != GBR_OK) return r;
    t.p = p;
    if (copy_in) copies->add(*m, t, rows, cols);
    *m = t;
    return GBR_OK;
}

// A 2-D map over rows x cols bf16.
int map_2d(CUtensorMap* map, const Mat& m, int64_t rows, int64_t cols, uint32_t box_cols, uint32_t box_rows,
           const char* what, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
    const uint64_t dims[2] = {uint64_t(cols), uint64_t(rows)};
    const uint64_t strides[1] = {uint64_t(m.ld) * 2};
    const uint32_t box[2] = {box_cols, box_rows};
    return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, m.p, dims, strides, box,
                             swizzle, what);
}

// ------------------------------------------------------------ CTA pairs
struct Product {
    Mat A, B;                      // as stored
    bool a_mn, b_mn;               // A: stored [I, Kc] (k-major) or [Kc, I]; B: [J, Kc] or [Kc, J]
    int32_t I, J, Kc;              // output rows, columns, contraction length
    Mat C, Z, R;
    const float* bias;
    Dropout drop;
    void* pair_kernel;             // linear_pair.cuh
    void* tile_kernel;             // linear_tile.cuh
};

// The tiles of a product on `units` CTA pairs.  The last round is split where
// it has tiles for at most half of the pairs and half a tile's products are
// worth more than the exchange of the parts (about 5 us: 16 k-blocks of 128).
linear::PairWork pair_work(const Product& p, int64_t units) {
    linear::PairWork w;
    memset(&w, 0, sizeof(w));
    w.m_tiles = int32_t(cdiv(p.I, linear::kTile));
    w.n_tiles = int32_t(cdiv(p.J, linear::kTile));
    w.num_tiles = int32_t(std::min<int64_t>(int64_t(w.m_tiles) * w.n_tiles, INT32_MAX));
    w.num_kb = int32_t(cdiv(p.Kc, 64 * linear::kSlices));
    w.group_m = 8;
    const int64_t rest = w.num_tiles % units;
    if (2 * rest <= units && w.num_kb / 2 >= 16) w.split = int32_t(rest);
    w.whole = w.num_tiles - w.split;
    return w;
}

// Zeroes words in the order of the stream, without a memset between kernels
// that overlap their launches.
__global__ void __launch_bounds__(256) zero_kernel(uint32_t* p, int32_t words) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    for (int32_t i = int32_t(blockIdx.x * 256 + threadIdx.x); i < words; i += int32_t(gridDim.x) * 256) p[i] = 0;
}

int run_pair(const Product& p, const LibCtx& c, cudaStream_t stream) {
    linear::PairParams P;
    memset(&P, 0, sizeof(P));
    int r;
    constexpr auto kSw64 = CU_TENSOR_MAP_SWIZZLE_64B;     // the epilogue's 32 x 32 boxes
    if ((r = map_2d(&P.mapC, p.C, p.I, p.J, 32, 32, "C", kSw64)) != GBR_OK) return r;
    P.mapA = P.mapB = P.mapZ = P.mapR = P.mapC;          // where unused
    if (p.Kc > 0) {
        r = p.a_mn ? map_2d(&P.mapA, p.A, p.Kc, p.I, 64, 64, "A") : map_2d(&P.mapA, p.A, p.I, p.Kc, 64, 128, "A");
        if (r != GBR_OK) return r;
        r = p.b_mn ? map_2d(&P.mapB, p.B, p.Kc, p.J, 64, 64, "B") : map_2d(&P.mapB, p.B, p.J, p.Kc, 64, 128, "B");
        if (r != GBR_OK) return r;
    }
    if (p.Z && (r = map_2d(&P.mapZ, p.Z, p.I, p.J, 32, 32, "Z", kSw64)) != GBR_OK) return r;
    if (p.R && (r = map_2d(&P.mapR, p.R, p.I, p.J, 32, 32, "residual", kSw64)) != GBR_OK) return r;
    P.has_z = bool(p.Z);
    P.has_r = bool(p.R);
    P.bias = p.bias;
    P.M = p.I, P.N = p.J;
    P.bias_vec = reinterpret_cast<uintptr_t>(p.bias) % 16 == 0;
    const int64_t tiles = cdiv(p.I, linear::kTile) * cdiv(p.J, linear::kTile);
    if (tiles >= (int64_t(1) << 31)) return report_errorf(GBR_ERR_INVALID, "linear: too many output tiles");
    const int64_t units = c.sm_count / 2;
    P.w = pair_work(p, units);
    Scratch ws(c, stream);
    if (P.w.split > 0) {
        const size_t counts = (linear::pair_count_bytes(P.w.split) + 255) & ~size_t(255);
        void* q;
        if ((r = ws.take(counts + linear::pair_part_bytes(P.w.split), "cudaMallocFromPoolAsync(split tiles)", &q)) !=
            GBR_OK)
            return r;
        P.w.count = static_cast<uint32_t*>(q);
        P.w.parts = reinterpret_cast<float4*>(static_cast<uint8_t*>(q) + counts);
        int32_t words = int32_t(counts / 4);
        void* zargs[] = {&P.w.count, &words};
        const cudaError_t e =
            launch_kernel(reinterpret_cast<void*>(&zero_kernel), dim3(1), 256, 0, 1, zargs, stream);
        if (e != cudaSuccess) return report_cuda(e, "launching the zeroing of the split tiles' counts");
        count_launch();
    }
    P.drop = p.drop;
    P.ctl = c.ctl;
    P.inject = c.inject;
    if ((r = raise_kernel_smem(p.pair_kernel, linear::kSmemBytes, c.device)) != GBR_OK) return r;
    void* args[] = {&P};
    const int64_t busy = std::min<int64_t>(units, P.w.whole > 0 && P.w.split > 0 ? units : P.w.whole + 2 * P.w.split);
    const cudaError_t e = launch_kernel(p.pair_kernel, dim3(unsigned(2 * busy)), linear::kThreads,
                                        linear::kSmemBytes, 2, args, stream);
    if (e != cudaSuccess) return report_cuda(e, "launching a linear kernel");
    count_launch();
    return GBR_OK;
}

// ------------------------------------------------------------ single tiles
struct TilePlan {
    int32_t bt, split, stages;
    double cycles;                 // estimate, see below
};

// Estimated SM cycles of the product on either kernel, for the choice between
// them, of the tile and of the split; fitted to measured sweeps of M 1..4096
// with (K, N) from (512, 512) to (4096, 14336) on a 152-SM GB300.
//   An SM takes in about 64 bytes a cycle from L2, about 40 where the wide
//   operand comes from HBM and no other row tile shares it; all SMs together
//   3500 from HBM.  DSMEM moves about 12 bytes a cycle and SM.
//   CTA pairs: 32 KiB a CTA and 64-k slice, 512 cycles at full rate (which is
//   also the tensor core's), 640 where less than one round of tiles runs; a
//   round is never below the 4800 of a tile's epilogue; 13500 to start, fill
//   the ring and drain the last tile.
// A tile's rows are finished at about 28 cycles each by the CTAs that share it;
// that decides against the pairs, among single tiles it hides under the others'
// loads, and counting it there picks worse ones (256 x 512 x 512: 6.1 -> 8.5 us).
// Measured against each other (us, single tiles / CTA pairs; forward unless
// said): rows 1 of 4096 x 4096 7.0 / 22, 128 12.9 / 20, 512 19.4 / 21.7, 1024
// 28.6 / 25; rows 128 of 4096 x 14336 27 / 30, 256 37 / 31; 301 x 520 x 1000
// 6.4 / 10.7; 1024^3 8.1 / 11.0; 4096 x 1024 x 1024 15.4 / 12.0; 2048 x 256 x
// 2048 11.5 / 8.3; dB of 512 x 1024 x 4096 13.2 / 9.2, of 4096 x 512 x 512
// 10.1 / 20, of 512 x 4096 x 4096 51 / 18.  Over 540 products (M 256..8192,
// K 64..4096, N 256..4096, all three directions) the choice is 1 % slower in
// the mean than the best of what was measured, and 10 % at worst.
double pair_cycles(const Product& p, int sms) {
    const linear::PairWork w = pair_work(p, sms / 2);
    const double whole = double(cdiv(w.whole, sms / 2)), half = w.split > 0 ? 0.5 : 0.0;
    const double rounds = whole + half, slices = double(cdiv(p.Kc, 64));
    return 13500.0 + (w.split > 0 ? 8000.0 : 0.0) +
           rounds * (rounds <= 1.0 ? 640.0 * slices : std::max(512.0 * slices, 4800.0));
}

// Shared memory of one of two CTAs an SM, and of one alone; the stages that fit.
constexpr int64_t kTileHalf = 110 * 1024, kTileWhole = 218 * 1024;
int tile_stages(int bt, int64_t budget) {
    return int(std::min<int64_t>(linear::kTileMaxStages, (budget - 2304) / linear::tile_stage_bytes(bt)));
}
// CTAs that fit at once, one an SM.  Of large clusters fewer do: 144 CTAs in
// fours, 120 in eights.
int64_t tile_fit(int cluster, int sms) { return cluster == 8 ? sms * 15 / 19 : cluster == 4 ? sms * 18 / 19 : sms; }

TilePlan plan_tile(const Product& p, int sms) {
    TilePlan best = {0, 0, 0, 1e30};
    double finish = 0.0;
    const int64_t nks = cdiv(p.Kc, 64);
    const double hbm = double(p.Kc) * double(p.J) * 2.0 / 3500.0;
    for (int bt : {int(std::min<int64_t>(256, cdiv(p.I, 16) * 16)), 64, 128, 256}) {
        if (p.a_mn && bt % 64 != 0) continue;           // MN-major rows come in panels of 64
        if (bt > 64 && bt >= p.I + 64) continue;
        const int64_t stage = linear::tile_stage_bytes(bt);
        const int64_t t_tiles = cdiv(p.I, bt), tiles = t_tiles * cdiv(p.J, 128);
        const double rows = double(std::min<int64_t>(p.I, bt));
        for (int s : {1, 2, 4, 8}) {
            if (s > nks && s > 1) continue;
            // Two an SM, eights fit as fours do alone.
            const int64_t fit = tile_fit(s, sms), fit2 = 2 * (s == 8 ? tile_fit(4, sms) : sms), slices = cdiv(nks, s);
            // A slice's loads; the wide operand from HBM or shared through L2.
            const double load = 16384.0 / (t_tiles == 1 ? 40.0 : 64.0) + bt * 2.0;
            // Two CTAs an SM where a tile's parts and a ring worth having fit
            // twice, unless one each is all there is and gains by the larger
            // ring: more slices than the smaller one holds, and its turn, about
            // 2200 cycles at best, not hidden by its loads (512^3, two slices a
            // CTA: 6.5 us one an SM, whose memory leaves no room for the next
            // launch's set-up, 5.8 two; one row of 4096^2 7.5 and 6.9; dB of
            // 8192 x 512 x 512, 32 slices: 14.2 and 18.1).
            const int64_t small = (kTileHalf - 2304) / stage;
            const bool ample = slices <= small || load >= 2200.0 / double(small);
            const int per_sm = bt <= 128 && (ample || tiles * s > fit) ? 2 : 1;
            const int64_t n = per_sm == 2 ? cdiv(tiles * s, sms) : cdiv(tiles * s, fit);
            const int64_t budget = per_sm == 2 ? kTileHalf : kTileWhole, rounds = cdiv(tiles * s, per_sm == 2 ? fit2 : fit);
            const int stages = tile_stages(bt, budget);
            const double feed =
                std::max(double(n * slices) * load, ample ? 0.0 : double(rounds * slices) * 2200.0 / double(stages));
            // HBM gives its rate to all SMs together; fewer get less of it.
            const double busy = std::sqrt(double(sms) / double(std::min<int64_t>(sms, tiles * s)));
            const double parts = double(n) * rows * 512.0 * (double(s - 1) / s / 12.0 + 1.0 / 64.0);
            const double cycles = 6000.0 + std::max(feed, hbm * busy) + parts + 60.0 * (s - 1) +
                                  3000.0 * double(rounds - 1);      // the cluster's barriers; rounds
            if (cycles < best.cycles) best = {bt, s, stages, cycles}, finish = double(n) * rows * 28.0 / s;
        }
    }
    best.cycles += finish;
    return best;
}

bool vec16(const Mat& m) { return !m || tma_ready(m); }

int tile_params(Product p, const TilePlan& plan, const LibCtx& c, linear::TileParams* out) {
    one_row(&p.A, p.a_mn ? p.Kc : p.I, p.a_mn ? p.I : p.Kc);
    one_row(&p.B, p.b_mn ? p.Kc : p.J, p.b_mn ? p.J : p.Kc);
    linear::TileParams& P = *out;
    memset(&P, 0, sizeof(P));
    int r;
    if (p.Kc > 0) {
        if ((r = p.b_mn ? map_2d(&P.mapW, p.B, p.Kc, p.J, 64, 64, "wide operand")
                        : map_2d(&P.mapW, p.B, p.J, p.Kc, 64, 128, "wide operand")) != GBR_OK)
            return r;
        if ((r = p.a_mn ? map_2d(&P.mapX, p.A, p.Kc, p.I, 64, 64, "narrow operand")
                        : map_2d(&P.mapX, p.A, p.I, p.Kc, 64, uint32_t(plan.bt), "narrow operand")) != GBR_OK)
            return r;
    }
    P.bias = p.bias;
    P.R = static_cast<const bf16*>(p.R.p), P.ldr = p.R.ld;
    P.C = static_cast<bf16*>(p.C.w()), P.ldc = p.C.ld;
    P.Z = static_cast<bf16*>(p.Z.w()), P.ldz = p.Z.ld;
    P.vec = vec16(p.R) && vec16(p.C) && vec16(p.Z);
    P.I = p.I, P.J = p.J;
    P.bt = plan.bt;
    P.t_tiles = int32_t(cdiv(p.I, plan.bt));
    P.num_ks = int32_t(cdiv(p.Kc, 64));
    P.split = plan.split;
    P.stages = plan.stages;
    P.tmem_cols = 32;
    while (int32_t(P.tmem_cols) < plan.bt) P.tmem_cols *= 2;
    P.drop = p.drop;
    P.ctl = c.ctl;
    P.inject = c.inject;
    return GBR_OK;
}

int64_t tile_ctas(const Product& p, const TilePlan& plan) { return cdiv(p.I, plan.bt) * cdiv(p.J, 128) * plan.split; }

int launch_tiles(void* kernel, void* params, int64_t ctas, size_t smem, int cluster, const LibCtx& c,
                 cudaStream_t stream) {
    const int r = raise_kernel_smem(kernel, smem, c.device);
    if (r != GBR_OK) return r;
    void* args[] = {params};
    const cudaError_t e = launch_kernel(kernel, dim3(unsigned(ctas)), linear::kTileThreads, smem, cluster, args, stream);
    if (e != cudaSuccess) return report_cuda(e, "launching a linear kernel");
    count_launch();
    return GBR_OK;
}

int run_tile(const Product& p, const TilePlan& plan, const LibCtx& c, cudaStream_t stream) {
    linear::TileParams P;
    const int r = tile_params(p, plan, c, &P);
    if (r != GBR_OK) return r;
    return launch_tiles(p.tile_kernel, &P, tile_ctas(p, plan), linear::tile_smem_bytes(plan.bt, plan.stages),
                        plan.split, c, stream);
}

// Runs the product with whatever TMA cannot address replaced by aligned copies.
int run_product(Product p, const LibCtx& c, cudaStream_t stream) {
    Scratch ws(c, stream);
    int r;
    const Mat C = p.C, Z = p.Z;
    const TilePlan plan = plan_tile(p, c.sm_count);
    const bool tile = plan.cycles < pair_cycles(p, c.sm_count);
    RepitchList in, out;
    if (p.Kc > 0) {
        if ((r = aligned_mat(&p.A, p.a_mn ? p.Kc : p.I, p.a_mn ? p.I : p.Kc, true, ws, &in)) != GBR_OK) return r;
        if ((r = aligned_mat(&p.B, p.b_mn ? p.Kc : p.J, p.b_mn ? p.J : p.Kc, true, ws, &in)) != GBR_OK) return r;
    }
    // The kernel of single tiles reads and writes everything else with plain accesses.
    if (!tile) {
        if (p.R && (r = aligned_mat(&p.R, p.I, p.J, true, ws, &in)) != GBR_OK) return r;
        if ((r = aligned_mat(&p.C, p.I, p.J, false, ws, nullptr)) != GBR_OK) return r;
        if (p.Z && (r = aligned_mat(&p.Z, p.I, p.J, false, ws, nullptr)) != GBR_OK) return r;
        if (p.C.p != C.p) out.add(p.C, C, p.I, p.J);
        if (p.Z.p != Z.p) out.add(p.Z, Z, p.I, p.J);
    }
    if ((r = in.launch(true, stream)) != GBR_OK) return r;
    if ((r = tile ? run_tile(p, plan, c, stream) : run_pair(p, c, stream)) != GBR_OK) return r;
    return out.launch(false, stream);
}

// The gradients' products, dA and dB: one grid, which waits for dZ as any launch
// does, where both take single tiles and nothing has to be copied first.  The
// larger cluster serves both (the smaller split divides it, all being powers of
// two), and where that is more CTAs than fit one an SM, rings that let two in,
// which each product for itself may not want.  Tiles of more than 128 rows leave
// no room for two: with those, no more CTAs than two rounds.
// Gradients with dZ and dbias (GELU), one after the other / in one grid, us:
// 64 x 512 x 512 13.4 / 9.1, 301 x 520 x 1000 17.6 / 13.6, 1024^3 22.4 / 16.0,
// 4096 x 512 x 512 29.2 / 20.2, 700 x 1032 x 264 17.3 / 13.4.  Over 46 sizes drawn
// at random that share a grid dA and dB take 0.65 of the time in the mean, over 45
// more with two rounds or more 0.90, and 1.12 at worst, with one row, where dB alone
// would go without dA's cluster (1 x 1400 x 3424 14.1 / 15.8).  2 x 12136 x 336,
// three rounds with tiles of 256 rows: 16.2 / 19.3.
int run_grads(const Product& da, const Product& db, const LibCtx& c, cudaStream_t stream) {
    // What TMA reads, or a matrix of one row, whose pitch does not matter.
    auto ready = [](Mat m, int32_t rows) {
        one_row(&m, rows, 8);
        return tma_ready(m);
    };
    TilePlan pa = plan_tile(da, c.sm_count), pb = plan_tile(db, c.sm_count);
    const int cluster = std::max(pa.split, pb.split);
    const int64_t first = cdiv(tile_ctas(da, pa), cluster) * cluster, second = cdiv(tile_ctas(db, pb), cluster) * cluster;
    const int64_t fit = tile_fit(cluster, c.sm_count);
    const bool pairable = pa.bt <= 128 && pb.bt <= 128;
    int r;
    if (pa.cycles >= pair_cycles(da, c.sm_count) || pb.cycles >= pair_cycles(db, c.sm_count) || da.Kc == 0 || db.Kc == 0 ||
        (!pairable && first + second > 2 * fit) || !ready(da.A, da.I) || !ready(da.B, da.J) || !ready(db.A, db.Kc)) {
        if ((r = run_product(da, c, stream)) != GBR_OK) return r;
        return run_product(db, c, stream);
    }
    if (pairable && first + second > fit)
        for (TilePlan* p : {&pa, &pb}) p->stages = std::min(p->stages, tile_stages(p->bt, kTileHalf));
    linear::TileGradParams G;
    if ((r = tile_params(da, pa, c, &G.da)) != GBR_OK || (r = tile_params(db, pb, c, &G.db)) != GBR_OK) return r;
    G.first = uint32_t(first);
    G.cluster = uint32_t(cluster);
    const size_t smem = std::max(linear::tile_smem_bytes(pa.bt, pa.stages), linear::tile_smem_bytes(pb.bt, pb.stages));
    return launch_tiles(linear_tile_grads_kernel(), &G, first + second, smem, cluster, c, stream);
}

// ------------------------------------------------------------ dZ and dbias
// dZ = drop(dC) act'(Z), and dbias = its column sums before the rounding.
// Bound by memory: dC and Z are read and dZ is written once.  A thread stands
// on 8 columns and walks down its rows, two at a time; a CTA is TX threads
// along the columns and 256 / TX along the rows, and a cluster of 8 CTAs shares
// the rows.  Sums: in a thread, then over the CTA's rows of threads, then over
// the cluster's CTAs in rank order, so that they never depend on timing.  Where
// the columns alone do not fill the GPU the rows are cut into `chunks` as well
// (blockIdx.y), whose sums go to scratch and are added in order by a second,
// small kernel (7954 x 88: 48 us with one cluster, whose CTAs read 1000 rows each).
// Two rows a turn and registers for four CTAs an SM: 58 us of 4096 x 14336
// GELU (235 MB read, 4 TB/s; no dZ); four rows 68, six CTAs 72.
constexpr int kDzThreads = 256, kDzCluster = 8, kDzRows = 2, kDzCtas = 4;

// VEC: rows of dC and Z start on 16 bytes.  The loads of kDzRows rows are
// issued, as raw 16 bytes, before the first is used.
template <int ACT, int TX, bool VEC>
__global__ void __launch_bounds__(kDzThreads, kDzCtas) dz_kernel(const LinearGradArgs a, float* sums) {
    __shared__ float part[kDzThreads / TX][TX * 8];
    ptx::griddep_wait();
    const uint32_t rank = ptx::cluster_ctarank();
    const int32_t tx = int32_t(threadIdx.x) % TX, ty = int32_t(threadIdx.x) / TX;
    const int32_t c = (int32_t(blockIdx.x / kDzCluster) * TX + tx) * 8, left = a.N - c;
    constexpr int32_t kPer = kDzThreads / TX;
    const int64_t share = int64_t(blockIdx.y) * kDzCluster + rank, shares = int64_t(gridDim.y) * kDzCluster;
    const int32_t r0 = int32_t(a.M * share / shares), r1 = int32_t(a.M * (share + 1) / shares);
    const bf16 *dC = static_cast<const bf16*>(a.dC.p) + c, *Z = static_cast<const bf16*>(a.Z.p) + c;
    bf16* dZ = static_cast<bf16*>(a.dZ.w());
    float sum[8] = {};
    auto one = [&](const uint4& rd, const uint4& rz, int64_t row) {
        float d[8], z[8];
        unpack8(rd, d);
        if (ACT != kActNone) {
            unpack8(rz, z);
#pragma unroll
            for (int j = 0; j < 8; j += 2) act_slope2<ACT>(d[j], d[j + 1], z[j], z[j + 1]);
        }
        if (a.drop.threshold != 0) {
            const uint4 bits = dropout_bits(a.drop, uint32_t(row), uint32_t(c / 8));
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = dropout_keep(a.drop, bits, j) ? d[j] * a.drop.scale : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += d[j];
        // dZ is this library's scratch: 16-byte aligned rows, padded to 8 columns.
        if (dZ != nullptr) store8(dZ + row * a.dZ.ld + c, d);
    };
    if (left > 0) {
        int64_t row = r0 + ty;
        uint4 rd[kDzRows], rz[kDzRows] = {};
        if (VEC && left >= 8) {
            for (; row + (kDzRows - 1) * kPer < r1; row += kPer * kDzRows) {
#pragma unroll
                for (int i = 0; i < kDzRows; ++i) {
                    rd[i] = *reinterpret_cast<const uint4*>(dC + (row + i * kPer) * a.dC.ld);
                    if (ACT != kActNone) rz[i] = *reinterpret_cast<const uint4*>(Z + (row + i * kPer) * a.Z.ld);
                }
#pragma unroll
                for (int i = 0; i < kDzRows; ++i) one(rd[i], rz[i], row + i * kPer);
            }
        }
        for (; row < r1; row += kPer) {
            rd[0] = load8_raw(dC + row * a.dC.ld, min(left, 8));
            if (ACT != kActNone) rz[0] = load8_raw(Z + row * a.Z.ld, min(left, 8));
            one(rd[0], rz[0], row);
        }
    }
    if (a.dbias == nullptr) return;                     // uniform over the cluster
#pragma unroll
    for (int j = 0; j < 8; ++j) part[ty][tx * 8 + j] = sum[j];
    __syncthreads();
    for (int32_t j = int32_t(threadIdx.x); j < TX * 8; j += kDzThreads) {
        float t = 0.f;
#pragma unroll
        for (int y = 0; y < kPer; ++y) t += part[y][j];
        part[0][j] = t;
    }
    ptx::cluster_sync_all();
    // Each CTA finishes one eighth of the columns.
    constexpr int32_t kShare = TX * 8 / kDzCluster;
    const int32_t j = int32_t(rank) * kShare + int32_t(threadIdx.x);
    const int32_t n = int32_t(blockIdx.x / kDzCluster) * TX * 8 + j;
    if (int32_t(threadIdx.x) < kShare && n < a.N) {
        const uint32_t at = ptx::smem_addr(&part[0][j]);
        float t = 0.f;
#pragma unroll
        for (uint32_t s = 0; s < kDzCluster; ++s)
            t += __uint_as_float(ptx::ld_shared_cluster_u32(ptx::mapa_shared(at, s)));
        if (sums != nullptr) sums[int64_t(blockIdx.y) * a.N + n] = t;
        else a.dbias[n] = t;
    }
    ptx::cluster_sync_all();   // the peers' sums have been read
}

__global__ void __launch_bounds__(256) dbias_kernel(const float* sums, float* dbias, int32_t N, int32_t chunks) {
    ptx::griddep_wait();
    const int32_t n = int32_t(blockIdx.x * 256 + threadIdx.x);
    if (n >= N) return;
    float t = 0.f;
#pragma unroll 8
    for (int32_t c = 0; c < chunks; ++c) t += sums[int64_t(c) * N + n];
    dbias[n] = t;
}

template <int TX, bool VEC>
void* dz_kernel_ptr(int act) {
    switch (act) {
        case kActRelu: return reinterpret_cast<void*>(&dz_kernel<kActRelu, TX, VEC>);
        case kActGelu: return reinterpret_cast<void*>(&dz_kernel<kActGelu, TX, VEC>);
        case kActGeluTanh: return reinterpret_cast<void*>(&dz_kernel<kActGeluTanh, TX, VEC>);
        case kActSilu: return reinterpret_cast<void*>(&dz_kernel<kActSilu, TX, VEC>);
        default: return reinterpret_cast<void*>(&dz_kernel<kActNone, TX, VEC>);
    }
}

}  // namespace

int launch_linear(const LinearArgs& a, const LibCtx& c, cudaStream_t stream) {
    Product p = {};
    p.A = a.A, p.B = a.B;
    p.a_mn = false, p.b_mn = true;
    p.I = a.M, p.J = a.N, p.Kc = a.K;
    p.C = a.C, p.Z = a.Z, p.R = a.R;
    p.bias = a.bias;
    p.drop = a.drop;
    p.pair_kernel = linear_pair_forward_kernel(a.act);
    p.tile_kernel = linear_tile_forward_kernel(a.act);
    return run_product(p, c, stream);
}

int launch_linear_dz(const LinearGradArgs& a, const LibCtx& c, cudaStream_t stream) {
    LinearGradArgs arg = a;
    const bool vec = vec16(a.dC) && vec16(a.Z);
    // 128 columns a CTA; rows cut until there are four CTAs an SM, what fits at
    // once, as long as a CTA keeps 128 rows (8192 x 4096, GELU: 47 us with two an
    // SM, 35 with four, 37 with eight).
    // Where that leaves SMs idle, 32 columns, unless the cut rows make up for it
    // (with GELU and dA, us: 1024^3 17.2 / 12.2, 2048 x 512 x 1024 17.3 / 14.1;
    // 8000 x 100 x 101, which would come down from 56 CTAs to 32, 14.1 / 18.1).
    auto cut = [&](int tx, int64_t* tiles) {
        *tiles = cdiv(a.N, tx * 8);
        return std::max<int64_t>(1, std::min<int64_t>(4 * int64_t(c.sm_count) / (*tiles * kDzCluster),
                                                      a.M / (8 * (kDzThreads / tx) * kDzCluster)));
    };
    int64_t tiles, chunks = cut(16, &tiles), tiles4, chunks4 = cut(4, &tiles4);
    const bool narrow = tiles * chunks * kDzCluster < c.sm_count && tiles4 * chunks4 >= tiles * chunks;
    if (narrow) tiles = tiles4, chunks = chunks4;
    Scratch ws(c, stream);
    void* sums = nullptr;
    if (chunks > 1 && a.dbias != nullptr) {
        const int r = ws.take(size_t(chunks) * size_t(a.N) * sizeof(float), "cudaMallocFromPoolAsync(dbias)", &sums);
        if (r != GBR_OK) return r;
    }
    void* args[] = {&arg, &sums};
    void* kernel = narrow ? (vec ? dz_kernel_ptr<4, true>(a.act) : dz_kernel_ptr<4, false>(a.act))
                          : (vec ? dz_kernel_ptr<16, true>(a.act) : dz_kernel_ptr<16, false>(a.act));
    cudaError_t e = launch_kernel(kernel,
                                  dim3(unsigned(tiles * kDzCluster), unsigned(chunks)), kDzThreads, 0, kDzCluster,
                                  args, stream);
    if (e != cudaSuccess) return report_cuda(e, "launching the gradient's dZ");
    count_launch();
    if (sums != nullptr) {
        int32_t n = int32_t(chunks);
        void* bargs[] = {&sums, &arg.dbias, &arg.N, &n};
        e = launch_kernel(reinterpret_cast<void*>(&dbias_kernel), dim3(unsigned(cdiv(a.N, 256))), 256, 0, 1, bargs,
                          stream);
        if (e != cudaSuccess) return report_cuda(e, "launching the sums of dbias");
        count_launch();
    }
    return GBR_OK;
}

int launch_linear_grads(Mat A, Mat B, Mat dZ, Mat dA, Mat dB, int32_t M, int32_t N, int32_t K, const LibCtx& c,
                        cudaStream_t stream) {
    Product a = {}, b = {};
    a.A = dZ, a.B = B;
    a.a_mn = false, a.b_mn = false;
    a.I = M, a.J = K, a.Kc = N;
    a.C = dA;
    a.pair_kernel = linear_pair_da_kernel();
    a.tile_kernel = linear_tile_da_kernel();
    b.A = A, b.B = dZ;
    b.a_mn = true, b.b_mn = true;
    b.I = K, b.J = N, b.Kc = M;
    b.C = dB;
    b.pair_kernel = linear_pair_db_kernel();
    b.tile_kernel = linear_tile_db_kernel();
    if (dA && dB) return run_grads(a, b, c, stream);
    return dA ? run_product(a, c, stream) : run_product(b, c, stream);
}

}  // namespace gbr
