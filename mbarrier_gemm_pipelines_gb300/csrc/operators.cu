// operators.cu -- entry points of the feed-forward operators (include/gbr.h):
// validation, scratch and the order of the launches.
#include "gbr.h"
#include "operators.h"

#include <algorithm>
#include <cmath>
#include <exception>
#include <initializer_list>
#include <limits>
#include <map>
#include <mutex>
#include <utility>

namespace gbr {
namespace {

constexpr int64_t kLim = int64_t(1) << 31;

// A row-major matrix argument as the caller describes it.
struct View {
    const char* name;
    const void* p;
    int64_t rows, cols, ld;
    int64_t esize;
};

bool empty(const View& v) { return v.p == nullptr || v.rows == 0 || v.cols == 0; }

// Whether some element of a shares memory with some element of b.  Two column
// ranges of one wider matrix interleave without sharing anything.
bool share(const View& a, const View& b) {
    if (empty(a) || empty(b)) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    const uint64_t aw = uint64_t(a.cols * a.esize), bw = uint64_t(b.cols * b.esize);
    const uint64_t ap = uint64_t(a.ld * a.esize), bp = uint64_t(b.ld * b.esize);
    const uintptr_t a1 = a0 + uint64_t(a.rows - 1) * ap + aw, b1 = b0 + uint64_t(b.rows - 1) * bp + bw;
    if (a1 <= b0 || b1 <= a0) return false;
    if (ap == bp && ap > 0) {
        const uint64_t d = b0 >= a0 ? (b0 - a0) % ap : (ap - (a0 - b0) % ap) % ap;
        if (d >= aw && d + bw <= ap) return false;
    }
    return true;
}

// The same elements in the same places: an in-place update.
bool same(const View& a, const View& b) {
    return a.p == b.p && (a.ld == b.ld || a.rows <= 1) && a.esize == b.esize;
}

int check_view(const char* fn, const View& v) {
    if (empty(v)) return GBR_OK;
    if (v.ld < v.cols && v.rows > 1)
        return report_errorf(GBR_ERR_INVALID, "%s: rows of %s overlap (row stride %lld < %lld columns)",
                             fn, v.name, static_cast<long long>(v.ld), static_cast<long long>(v.cols));
    if (v.ld < 0 || v.ld > (int64_t(1) << 40))
        return report_errorf(GBR_ERR_INVALID, "%s: row stride of %s out of range", fn, v.name);
    if (reinterpret_cast<uintptr_t>(v.p) % uint64_t(v.esize) != 0)
        return report_errorf(GBR_ERR_ALIGN, "%s: %s is not aligned to its element size", fn, v.name);
    return GBR_OK;
}

int check_drop(const char* fn, double p, uint64_t seed, uint64_t offset, Dropout* d) {
    if (!(p >= 0.0 && p <= 1.0)) return report_errorf(GBR_ERR_INVALID, "%s: p must be in [0, 1]", fn);
    d->threshold = uint32_t(std::nearbyint(p * 65536.0));
    d->scale = d->threshold >= 65536u ? 0.f : float(65536.0 / double(65536u - d->threshold));
    d->key0 = uint32_t(seed);
    d->key1 = uint32_t(seed >> 32);
    d->off0 = uint32_t(offset);
    d->off1 = uint32_t(offset >> 32);
    return GBR_OK;
}

int check_sizes(const char* fn, int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0 || M >= kLim || N >= kLim || K >= kLim)
        return report_errorf(GBR_ERR_INVALID, "%s: sizes must be in [0, 2^31)", fn);
    return GBR_OK;
}

// Kernels count past a row's end in 32 bits.
int check_columns(const char* fn, int64_t cols) {
    if (cols >= kLim / 2) return report_errorf(GBR_ERR_INVALID, "%s: columns must be below 2^30", fn);
    return GBR_OK;
}

int check_type(const char* fn, int dtype, bool* bf16) {
    if (dtype != GBR_BF16 && dtype != GBR_F32_FFMA && dtype != GBR_F32_TF32)
        return report_errorf(GBR_ERR_UNSUPPORTED, "%s: bf16 or fp32 elements only", fn);
    *bf16 = dtype == GBR_BF16;
    return GBR_OK;
}

// What residual_norm and its gradients have in common.
int check_norm(const char* fn, int64_t rows, int64_t cols, int64_t gates, const void* gate, double scale, double eps,
               int dtype, ResidualNormArgs* a) {
    int r = check_type(fn, dtype, &a->bf16);
    if (r != GBR_OK || (r = check_sizes(fn, rows, cols, 0)) != GBR_OK || (r = check_columns(fn, cols)) != GBR_OK) return r;
    // Both go to the kernels as fp32, where a larger one would be infinite and an eps that vanishes no longer keep rows of
    // zeros from 0 / 0.
    constexpr double kMost = std::numeric_limits<float>::max();
    if (!(eps >= 0.0 && eps <= kMost) || (eps > 0.0 && float(eps) == 0.f) || !(std::fabs(scale) <= kMost))
        return report_errorf(GBR_ERR_INVALID, "%s: eps must not be negative, eps and scale within fp32", fn);
    if (gate == nullptr) gates = 0;
    else if (gates < 0 || (gates == 0 ? rows != 0 : rows % gates != 0))
        return report_errorf(GBR_ERR_INVALID, "%s: the rows must be a multiple of the gate's", fn);
    a->rows = int32_t(rows), a->cols = int32_t(cols), a->gates = int32_t(gates);
    a->per_gate = gates > 0 ? int32_t(rows / gates) : 0;
    a->scale = float(scale), a->eps = float(eps);
    return GBR_OK;
}

int check_rows(const char* fn, int64_t T, int64_t top_k, int64_t D, int num_experts, int dtype, bool* bf16) {
    int r = check_type(fn, dtype, bf16);
    if (r != GBR_OK || (r = check_sizes(fn, T, top_k, D)) != GBR_OK || (r = check_columns(fn, D)) != GBR_OK) return r;
    if (T * top_k >= kLim) return report_errorf(GBR_ERR_INVALID, "%s: T * top_k must be below 2^31", fn);
    if (num_experts < 1 || num_experts > kSortMaxExperts)
        return report_errorf(GBR_ERR_INVALID, "%s: num_experts must be 1..%d", fn, kSortMaxExperts);
    return GBR_OK;
}

int check_outputs(const char* fn, std::initializer_list<const View*> in, std::initializer_list<const View*> out) {
    int r;
    for (auto list : {in, out})
        for (const View* v : list)
            if ((r = check_view(fn, *v)) != GBR_OK) return r;
    for (const View* o : out)
        for (auto list : {in, out})
            for (const View* v : list)
                if (v != o && share(*o, *v))
                    return report_errorf(GBR_ERR_INVALID, "%s: %s overlaps %s", fn, o->name, v->name);
    return GBR_OK;
}

int check_mx(const char* fn, int64_t rows, int64_t cols, int dtype, bool* bf16) {
    int r = check_type(fn, dtype, bf16);
    if (r != GBR_OK || (r = check_sizes(fn, rows, cols, 0)) != GBR_OK) return r;
    return check_columns(fn, std::max(rows, cols));     // either may lie along X's rows
}

int check_mx_pointers(const char* fn, const void* data, const void* scales) {
    if (reinterpret_cast<uintptr_t>(data) % 16 || reinterpret_cast<uintptr_t>(scales) % 16)
        return report_errorf(GBR_ERR_ALIGN, "%s: 4-bit data and their scales must be 16-byte aligned", fn);
    return GBR_OK;
}

// No C++ exception leaves a C entry point.
template <class F>
int guarded(const char* fn, F&& f) noexcept {
    try {
        return f();
    } catch (const std::exception& e) {
        try {
            return report_errorf(GBR_ERR_CUDA, "%s: %s", fn, e.what());
        } catch (...) {
            return GBR_ERR_CUDA;
        }
    } catch (...) {
        return GBR_ERR_CUDA;
    }
}

}  // namespace

cudaError_t launch_kernel(void* kernel, dim3 grid, int threads, size_t smem, int cluster, void** args,
                         cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
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
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

int raise_kernel_smem(void* kernel, size_t smem, int dev) {
    static std::mutex mu;
    static std::map<std::pair<void*, int>, size_t> set;
    std::lock_guard<std::mutex> lk(mu);
    const cudaError_t e = raise_smem_limit(kernel, smem, &set[{kernel, dev}]);
    return e == cudaSuccess ? int(GBR_OK) : report_cuda(e, "cudaFuncSetAttribute(shared memory)");
}

int Scratch::take(size_t bytes, const char* what, void** out) {
    if (n_ >= int(sizeof(p_) / sizeof(p_[0]))) return report_errorf(GBR_ERR_CUDA, "%s: too many blocks", what);
    const cudaError_t e = cudaMallocFromPoolAsync(&p_[n_], bytes, c_.pool, st_);
    if (e != cudaSuccess) return report_cuda(e, what);
    *out = p_[n_++];
    return GBR_OK;
}

}  // namespace gbr

using namespace gbr;

extern "C" {

int dropout_add(const void* X, int64_t ldx, const void* residual, int64_t ldr, void* Y, int64_t ldy,
                int64_t rows, int64_t cols, int dtype, double p, uint64_t seed, uint64_t offset,
                gbr_stream_t stream) {
    const char* fn = "dropout_add";
    return guarded(fn, [&]() -> int {
        if (dtype != GBR_BF16 && dtype != GBR_F32_FFMA && dtype != GBR_F32_TF32)
            return report_errorf(GBR_ERR_UNSUPPORTED, "%s: bf16 or fp32 elements only", fn);
        int r = check_sizes(fn, rows, cols, 0);
        DropoutAddArgs a = {};
        if (r != GBR_OK || (r = check_drop(fn, p, seed, offset, &a.drop)) != GBR_OK) return r;
        if (rows == 0 || cols == 0) return GBR_OK;
        if (!X || !Y) return report_errorf(GBR_ERR_INVALID, "%s: NULL buffer", fn);
        const int64_t es = dtype == GBR_BF16 ? 2 : 4;
        const View vx = {"X", X, rows, cols, ldx, es}, vr = {"residual", residual, rows, cols, ldr, es},
                   vy = {"Y", Y, rows, cols, ldy, es};
        for (const View* v : {&vx, &vr, &vy})
            if ((r = check_view(fn, *v)) != GBR_OK) return r;
        for (const View* v : {&vx, &vr})
            if (share(vy, *v) && !same(vy, *v))
                return report_errorf(GBR_ERR_INVALID, "%s: Y overlaps %s", fn, v->name);
        LibCtx c;
        if ((r = lib_ctx(&c)) != GBR_OK) return r;
        a.X = X, a.R = residual, a.Y = Y;
        a.ldx = ldx, a.ldr = ldr, a.ldy = ldy;
        a.rows = int32_t(rows), a.cols = int32_t(cols);
        a.bf16 = dtype == GBR_BF16;
        const cudaError_t e = launch_dropout_add(a, c.sm_count, reinterpret_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return report_cuda(e, "launching dropout_add");
        count_launch();
        return GBR_OK;
    });
}

int gemm_bias_act(const void* A, int64_t lda, const void* B, int64_t ldb, const float* bias,
                  const void* residual, int64_t ldr, void* C, int64_t ldc, void* Z, int64_t ldz,
                  int64_t M, int64_t N, int64_t K, int dtype, int act, double p, uint64_t seed,
                  uint64_t offset, gbr_stream_t stream) {
    const char* fn = "gemm_bias_act";
    return guarded(fn, [&]() -> int {
        if (dtype != GBR_BF16) return report_errorf(GBR_ERR_UNSUPPORTED, "%s: only GBR_BF16 is built", fn);
        if (act < 0 || act >= kActs) return report_errorf(GBR_ERR_INVALID, "%s: unknown activation %d", fn, act);
        LinearArgs a = {};
        int r = check_sizes(fn, M, N, K);
        if (r != GBR_OK || (r = check_drop(fn, p, seed, offset, &a.drop)) != GBR_OK) return r;
        if (M == 0 || N == 0) return GBR_OK;
        if (!C || (K > 0 && (!A || !B))) return report_errorf(GBR_ERR_INVALID, "%s: NULL buffer", fn);
        const View va = {"A", A, M, K, lda, 2}, vb = {"B", B, K, N, ldb, 2}, vr = {"residual", residual, M, N, ldr, 2},
                   vc = {"C", C, M, N, ldc, 2}, vz = {"Z", Z, M, N, ldz, 2}, vbias = {"bias", bias, 1, N, N, 4};
        for (const View* v : {&va, &vb, &vr, &vc, &vz, &vbias})
            if ((r = check_view(fn, *v)) != GBR_OK) return r;
        for (const View* v : {&va, &vb, &vbias, &vr}) {
            if (share(vc, *v) && !(v == &vr && same(vc, vr)))
                return report_errorf(GBR_ERR_INVALID, "%s: C overlaps %s", fn, v->name);
            if (share(vz, *v)) return report_errorf(GBR_ERR_INVALID, "%s: Z overlaps %s", fn, v->name);
        }
        if (share(vc, vz)) return report_errorf(GBR_ERR_INVALID, "%s: C overlaps Z", fn);
        LibCtx c;
        if ((r = lib_ctx(&c)) != GBR_OK) return r;
        a.A = {A, lda}, a.B = {B, ldb}, a.R = {residual, ldr}, a.C = {C, ldc}, a.Z = {Z, ldz};
        a.bias = bias;
        a.M = int32_t(M), a.N = int32_t(N), a.K = int32_t(K);
        a.act = act;
        return launch_linear(a, c, reinterpret_cast<cudaStream_t>(stream));
    });
}

int gemm_bias_act_backward(const void* dC, int64_t lddc, const void* A, int64_t lda, const void* B,
                           int64_t ldb, const void* Z, int64_t ldz, void* dA, int64_t ldda, void* dB,
                           int64_t lddb, float* dbias, int64_t M, int64_t N, int64_t K, int dtype, int act,
                           double p, uint64_t seed, uint64_t offset, gbr_stream_t stream) {
    const char* fn = "gemm_bias_act_backward";
    return guarded(fn, [&]() -> int {
        if (dtype != GBR_BF16) return report_errorf(GBR_ERR_UNSUPPORTED, "%s: only GBR_BF16 is built", fn);
        if (act < 0 || act >= kActs) return report_errorf(GBR_ERR_INVALID, "%s: unknown activation %d", fn, act);
        LinearGradArgs g = {};
        int r = check_sizes(fn, M, N, K);
        if (r != GBR_OK || (r = check_drop(fn, p, seed, offset, &g.drop)) != GBR_OK) return r;
        const bool want_da = dA != nullptr && M > 0 && K > 0, want_db = dB != nullptr && N > 0 && K > 0;
        const bool want_bias = dbias != nullptr && N > 0;
        if (!want_da && !want_db && !want_bias) return GBR_OK;
        const bool some = M > 0 && N > 0;             // dC holds something
        if (some && (!dC || (act != kActNone && !Z) || (want_da && !B) || (want_db && !A)))
            return report_errorf(GBR_ERR_INVALID, "%s: NULL buffer", fn);
        const View vdc = {"dC", dC, M, N, lddc, 2}, va = {"A", want_db ? A : nullptr, M, K, lda, 2},
                   vb = {"B", want_da ? B : nullptr, K, N, ldb, 2},
                   vz = {"Z", act != kActNone ? Z : nullptr, M, N, ldz, 2}, vda = {"dA", dA, M, K, ldda, 2},
                   vdb = {"dB", dB, K, N, lddb, 2}, vdbias = {"dbias", dbias, 1, N, N, 4};
        for (const View* v : {&vdc, &va, &vb, &vz, &vda, &vdb, &vdbias})
            if ((r = check_view(fn, *v)) != GBR_OK) return r;
        for (const View* o : {&vda, &vdb, &vdbias})
            for (const View* v : {&vdc, &va, &vb, &vz, &vda, &vdb, &vdbias})
                if (v != o && share(*o, *v))
                    return report_errorf(GBR_ERR_INVALID, "%s: %s overlaps %s", fn, o->name, v->name);
        LibCtx c;
        if ((r = lib_ctx(&c)) != GBR_OK) return r;
        cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
        // dZ is dC itself unless dropout or an activation lies between them.
        const bool plain = act == kActNone && g.drop.threshold == 0;
        const bool products = want_da || want_db;
        g.dC = {dC, lddc};
        g.Z = {vz.p, ldz};
        g.M = int32_t(M), g.N = int32_t(N);
        g.act = act;
        g.dbias = want_bias ? dbias : nullptr;
        Scratch ws(c, st);
        Mat dz = {dC, lddc};
        if (!plain && products && some) {
            const int64_t ld = (N + 7) / 8 * 8;
            void* q;
            if ((r = ws.take(size_t(M) * size_t(ld) * 2, "cudaMallocFromPoolAsync(dZ)", &q)) != GBR_OK) return r;
            dz = {q, ld};
            g.dZ = dz;
        }
        if ((want_bias || g.dZ) && (r = launch_linear_dz(g, c, st)) != GBR_OK) return r;
        if (!products) return GBR_OK;
        return launch_linear_grads({A, lda}, {B, ldb}, dz, {want_da ? dA : nullptr, ldda}, {want_db ? dB : nullptr, lddb},
                                   g.M, g.N, int32_t(K), c, st);
    });
}

int moe_layer(const void* X, const float* Wr, const void* W1, const float* b1, const void* W2,
              const float* b2, void* Y, int64_t* expert_ids, float* expert_weights, int64_t T, int64_t D,
              int64_t F, int num_experts, int top_k, int act, int gated, int dtype, gbr_stream_t stream) {
    const char* fn = "moe_layer";
    return guarded(fn, [&]() -> int {
        if (dtype != GBR_BF16) return report_errorf(GBR_ERR_UNSUPPORTED, "%s: only GBR_BF16 is built", fn);
        if (act < 0 || act >= kActs) return report_errorf(GBR_ERR_INVALID, "%s: unknown activation %d", fn, act);
        if (gated != 0 && gated != 1) return report_errorf(GBR_ERR_INVALID, "%s: gated must be 0 or 1", fn);
        int r = check_sizes(fn, T, D, F);
        if (r != GBR_OK) return r;
        if (F >= kLim / 2) return report_errorf(GBR_ERR_INVALID, "%s: F must be below 2^30", fn);
        if (T > kMoeMaxTokens)
            return report_errorf(GBR_ERR_INVALID, "%s: at most %d tokens a call (gemm_bias_relu_grouped serves more)",
                                 fn, kMoeMaxTokens);
        if (num_experts < 1 || num_experts > kMoeMaxExperts)
            return report_errorf(GBR_ERR_INVALID, "%s: num_experts must be 1..%d", fn, kMoeMaxExperts);
        if (top_k < 1 || top_k > kMoeMaxTopK || top_k > num_experts)
            return report_errorf(GBR_ERR_INVALID, "%s: top_k must be 1..min(%d, num_experts)", fn, kMoeMaxTopK);
        if (T == 0) return GBR_OK;
        if (D == 0 || F == 0) return report_errorf(GBR_ERR_INVALID, "%s: D and F must be positive", fn);
        if (!X || !Wr || !W1 || !W2 || !Y) return report_errorf(GBR_ERR_INVALID, "%s: NULL buffer", fn);
        if (D % 8 || F % 8) return report_errorf(GBR_ERR_ALIGN, "%s: D and F must be multiples of 8", fn);
        for (const void* q : {X, static_cast<const void*>(Wr), W1, static_cast<const void*>(b1), W2,
                              static_cast<const void*>(b2), static_cast<const void*>(Y),
                              static_cast<const void*>(expert_ids), static_cast<const void*>(expert_weights)})
            if (reinterpret_cast<uintptr_t>(q) % 16)
                return report_errorf(GBR_ERR_ALIGN, "%s: buffers must be 16-byte aligned", fn);
        const int64_t E = num_experts, F1 = gated ? 2 * F : F;
        const View in[] = {{"X", X, 1, T * D, T * D, 2},           {"Wr", Wr, 1, D * E, D * E, 4},
                           {"W1", W1, 1, E * D * F1, E * D * F1, 2}, {"b1", b1, 1, E * F1, E * F1, 4},
                           {"W2", W2, 1, E * F * D, E * F * D, 2},   {"b2", b2, 1, E * D, E * D, 4}};
        const View out[] = {{"Y", Y, 1, T * D, T * D, 2},
                            {"expert_ids", expert_ids, 1, T * top_k, T * top_k, 8},
                            {"expert_weights", expert_weights, 1, T * top_k, T * top_k, 4}};
        for (const View& o : out) {
            for (const View& v : in)
                if (share(o, v)) return report_errorf(GBR_ERR_INVALID, "%s: %s overlaps %s", fn, o.name, v.name);
            for (const View& v : out)
                if (&v != &o && share(o, v))
                    return report_errorf(GBR_ERR_INVALID, "%s: %s overlaps %s", fn, o.name, v.name);
        }
        LibCtx c;
        if ((r = lib_ctx(&c)) != GBR_OK) return r;
        cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
        MoeArgs a = {};
        a.X = X, a.Wr = Wr, a.W1 = W1, a.b1 = b1, a.W2 = W2, a.b2 = b2, a.Y = Y;
        a.T = int32_t(T), a.D = int32_t(D), a.F = int32_t(F), a.E = num_experts, a.top_k = top_k;
        a.act = act, a.gated = gated != 0;
        // The routing goes to scratch where the caller does not ask for it.
        auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
        const size_t route = up(size_t(T * top_k) * 8), own = moe_scratch_bytes(a, c);
        Scratch ws(c, st);
        void* q;
        if ((r = ws.take(2 * route + own, "cudaMallocFromPoolAsync(expert layer)", &q)) != GBR_OK) return r;
        uint8_t* base = static_cast<uint8_t*>(q);
        a.ids = expert_ids ? expert_ids : reinterpret_cast<int64_t*>(base);
        a.weights = expert_weights ? expert_weights : reinterpret_cast<float*>(base + route);
        return launch_moe(a, base + 2 * route, c, st);
    });
}

int residual_norm(const void* X, int64_t ldx, const void* R, int64_t ldr, const float* post, const void* gate,
                  int64_t ldg, int64_t gates, double scale, const float* pre, double eps, void* S, int64_t lds, void* H,
                  int64_t ldh, int64_t rows, int64_t cols, int dtype, gbr_stream_t stream) {
    const char* fn = "residual_norm";
    return guarded(fn, [&]() -> int {
        ResidualNormArgs a = {};
        int r = check_norm(fn, rows, cols, gates, gate, scale, eps, dtype, &a);
        if (r != GBR_OK) return r;
        if (rows == 0 || cols == 0 || (!S && !H)) return GBR_OK;
        if ((H != nullptr) != (pre != nullptr))
            return report_errorf(GBR_ERR_INVALID, "%s: H and pre go together", fn);
        if (!X) return report_errorf(GBR_ERR_INVALID, "%s: NULL buffer", fn);
        const int64_t es = a.bf16 ? 2 : 4;
        const View vx = {"X", X, rows, cols, ldx, es}, vr = {"R", R, rows, cols, ldr, es},
                   vg = {"gate", gate, gates, cols, ldg, es}, vs = {"S", S, rows, cols, lds, es},
                   vh = {"H", H, rows, cols, ldh, es}, vpost = {"post", post, 1, cols, cols, 4},
                   vpre = {"pre", pre, 1, cols, cols, 4};
        for (const View* v : {&vx, &vr, &vg, &vs, &vh, &vpost, &vpre})
            if ((r = check_view(fn, *v)) != GBR_OK) return r;
        for (const View* o : {&vs, &vh})
            for (const View* v : {&vx, &vr, &vg, &vpost, &vpre})
                if (share(*o, *v) && !((v == &vx || v == &vr) && same(*o, *v)))
                    return report_errorf(GBR_ERR_INVALID, "%s: %s overlaps %s", fn, o->name, v->name);
        if (share(vs, vh)) return report_errorf(GBR_ERR_INVALID, "%s: S overlaps H", fn);
        LibCtx c;
        if ((r = lib_ctx(&c)) != GBR_OK) return r;
        a.X = {X, ldx}, a.R = {R, ldr}, a.G = {gate, ldg}, a.S = {S, lds}, a.H = {H, ldh};
        a.post = post, a.pre = pre;
        return launch_residual_norm(a, c, reinterpret_cast<cudaStream_t>(stream));
    });
}

int residual_norm_backward(const void* dS, int64_t ldds, const void* dH, int64_t lddh, const void* X, int64_t ldx,
                           const void* S, int64_t lds, const float* post, const void* gate, int64_t ldg, int64_t gates,
                           double scale, const float* pre, double eps, void* dX, int64_t lddx, void* dR, int64_t lddr,
                           float* dpost, void* dgate, int64_t lddg, float* dpre, int64_t rows, int64_t cols, int dtype,
                           gbr_stream_t stream) {
    const char* fn = "residual_norm_backward";
    return guarded(fn, [&]() -> int {
        ResidualNormArgs f = {};
        int r = check_norm(fn, rows, cols, gates, gate, scale, eps, dtype, &f);
        if (r != GBR_OK) return r;
        if ((dpost && !post) || (dpre && !pre) || (dgate && !gate))
            return report_errorf(GBR_ERR_INVALID, "%s: a gradient of a weight or gate that is not there", fn);
        if (cols == 0 || (!dX && !dR && !dpost && !dgate && !dpre)) return GBR_OK;
        const bool some = rows > 0;
        if (f.gates == 0) gate = nullptr;               // none of its rows is there
        const bool need_x = post || gate;
        if (some && ((need_x && !X) || (pre && (!dH || !S)) || (!dS && !pre)))
            return report_errorf(GBR_ERR_INVALID, "%s: NULL buffer", fn);
        const int64_t es = f.bf16 ? 2 : 4;
        const View vds = {"dS", dS, rows, cols, ldds, es}, vdh = {"dH", pre ? dH : nullptr, rows, cols, lddh, es},
                   vx = {"X", need_x ? X : nullptr, rows, cols, ldx, es}, vs = {"S", pre ? S : nullptr, rows, cols, lds, es},
                   vg = {"gate", gate, gates, cols, ldg, es}, vpost = {"post", post, 1, cols, cols, 4},
                   vpre = {"pre", pre, 1, cols, cols, 4}, vdx = {"dX", dX, rows, cols, lddx, es},
                   vdr = {"dR", dR, rows, cols, lddr, es}, vdg = {"dgate", dgate, gates, cols, lddg, es},
                   vdpost = {"dpost", dpost, 1, cols, cols, 4}, vdpre = {"dpre", dpre, 1, cols, cols, 4};
        const View* const all[] = {&vds, &vdh, &vx, &vs, &vg, &vpost, &vpre, &vdx, &vdr, &vdg, &vdpost, &vdpre};
        for (const View* v : all)
            if ((r = check_view(fn, *v)) != GBR_OK) return r;
        for (const View* o : {&vdx, &vdr, &vdg, &vdpost, &vdpre})
            for (const View* v : all)
                if (v != o && share(*o, *v))
                    return report_errorf(GBR_ERR_INVALID, "%s: %s overlaps %s", fn, o->name, v->name);
        LibCtx c;
        if ((r = lib_ctx(&c)) != GBR_OK) return r;
        ResidualNormGradArgs a = {};
        a.dS = {dS, ldds}, a.dH = {vdh.p, lddh}, a.X = {vx.p, ldx}, a.S = {vs.p, lds}, a.G = {gate, ldg};
        a.post = post, a.pre = pre;
        a.dX = {dX, lddx}, a.dR = {dR, lddr}, a.dG = {dgate, lddg};
        a.dpost = dpost, a.dpre = dpre;
        a.rows = f.rows, a.cols = f.cols, a.gates = f.gates, a.per_gate = f.per_gate;
        a.scale = f.scale, a.eps = f.eps, a.bf16 = f.bf16;
        return launch_residual_norm_grad(a, c, reinterpret_cast<cudaStream_t>(stream));
    });
}

int moe_sort(const int64_t* expert_ids, int64_t choices, int num_experts, int32_t* positions, int32_t* offsets,
             gbr_stream_t stream) {
    const char* fn = "moe_sort";
    return guarded(fn, [&]() -> int {
        if (choices < 0 || choices >= kLim) return report_errorf(GBR_ERR_INVALID, "%s: choices must be in [0, 2^31)", fn);
        if (num_experts < 1 || num_experts > kSortMaxExperts)
            return report_errorf(GBR_ERR_INVALID, "%s: num_experts must be 1..%d", fn, kSortMaxExperts);
        if (!offsets || (choices > 0 && (!expert_ids || !positions)))
            return report_errorf(GBR_ERR_INVALID, "%s: NULL buffer", fn);
        const View in = {"expert_ids", expert_ids, 1, choices, choices, 8},
                   pos = {"positions", positions, 1, choices, choices, 4},
                   off = {"offsets", offsets, 1, num_experts + 1, num_experts + 1, 4};
        int r;
        for (const View* v : {&in, &pos, &off})
            if ((r = check_view(fn, *v)) != GBR_OK) return r;
        if (share(pos, in) || share(off, in) || share(pos, off))
            return report_errorf(GBR_ERR_INVALID, "%s: overlapping buffers", fn);
        LibCtx c;
        if ((r = lib_ctx(&c)) != GBR_OK) return r;
        return launch_moe_sort({expert_ids, positions, offsets, int32_t(choices), num_experts}, c,
                               reinterpret_cast<cudaStream_t>(stream));
    });
}

int moe_dispatch(const void* X, int64_t ldx, const int32_t* positions, const int32_t* offsets, int num_experts, void* Xs,
                 int64_t ldxs, int64_t T, int64_t top_k, int64_t D, int dtype, gbr_stream_t stream) {
    const char* fn = "moe_dispatch";
    return guarded(fn, [&]() -> int {
        MoeRowsArgs a = {};
        int r = check_rows(fn, T, top_k, D, num_experts, dtype, &a.bf16);
        if (r != GBR_OK || T == 0 || top_k == 0 || D == 0) return r;
        if (!X || !positions || !offsets || !Xs) return report_errorf(GBR_ERR_INVALID, "%s: NULL buffer", fn);
        const int64_t es = a.bf16 ? 2 : 4;
        const View vx = {"X", X, T, D, ldx, es}, vo = {"Xs", Xs, T * top_k, D, ldxs, es},
                   vp = {"positions", positions, 1, T * top_k, T * top_k, 4},
                   vf = {"offsets", offsets, 1, num_experts + 1, num_experts + 1, 4};
        if ((r = check_outputs(fn, {&vx, &vp, &vf}, {&vo})) != GBR_OK) return r;
        LibCtx c;
        if ((r = lib_ctx(&c)) != GBR_OK) return r;
        a.X = {X, ldx}, a.Ys = {Xs, ldxs};
        a.positions = positions, a.offsets = offsets;
        a.T = int32_t(T), a.k = int32_t(top_k), a.D = int32_t(D), a.experts = num_experts;
        return launch_moe_dispatch(a, c, reinterpret_cast<cudaStream_t>(stream));
    });
}

int moe_combine(const void* Ys, int64_t ldys, int64_t rows, const int32_t* positions, const float* weights,
                const void* residual, int64_t ldr, void* Y, int64_t ldy, int64_t T, int64_t top_k, int64_t D, int dtype,
                gbr_stream_t stream) {
    const char* fn = "moe_combine";
    return guarded(fn, [&]() -> int {
        MoeRowsArgs a = {};
        int r = check_rows(fn, T, top_k, D, 1, dtype, &a.bf16);
        if (r != GBR_OK) return r;
        if (rows < 0 || rows >= kLim) return report_errorf(GBR_ERR_INVALID, "%s: rows must be in [0, 2^31)", fn);
        if (T == 0 || D == 0) return GBR_OK;
        if (!Y || (top_k > 0 && (!positions || (rows > 0 && !Ys))))
            return report_errorf(GBR_ERR_INVALID, "%s: NULL buffer", fn);
        const int64_t es = a.bf16 ? 2 : 4;
        const View vi = {"Ys", Ys, rows, D, ldys, es}, vr = {"residual", residual, T, D, ldr, es}, vy = {"Y", Y, T, D, ldy, es},
                   vp = {"positions", positions, 1, T * top_k, T * top_k, 4},
                   vw = {"weights", weights, 1, T * top_k, T * top_k, 4};
        for (const View* v : {&vi, &vr, &vy, &vp, &vw})
            if ((r = check_view(fn, *v)) != GBR_OK) return r;
        for (const View* v : {&vi, &vr, &vp, &vw})
            if (share(vy, *v) && !(v == &vr && same(vy, vr)))
                return report_errorf(GBR_ERR_INVALID, "%s: Y overlaps %s", fn, v->name);
        LibCtx c;
        if ((r = lib_ctx(&c)) != GBR_OK) return r;
        a.Ys = {Ys, ldys}, a.R = {residual, ldr}, a.Y = {Y, ldy};
        a.positions = positions, a.weights = weights;
        a.T = int32_t(T), a.k = int32_t(top_k), a.D = int32_t(D);
        return launch_moe_combine(a, rows, c, reinterpret_cast<cudaStream_t>(stream));
    });
}

int moe_combine_backward(const void* dY, int64_t lddy, const void* Ys, int64_t ldys, const int32_t* positions,
                         const int32_t* offsets, int num_experts, const float* weights, void* dYs, int64_t lddys,
                         float* dweights, int64_t T, int64_t top_k, int64_t D, int dtype, gbr_stream_t stream) {
    const char* fn = "moe_combine_backward";
    return guarded(fn, [&]() -> int {
        MoeCombineGradArgs a = {};
        int r = check_rows(fn, T, top_k, D, num_experts, dtype, &a.bf16);
        if (r != GBR_OK) return r;
        if (D == 0) dYs = nullptr;                      // no element to write
        if (T == 0 || top_k == 0 || (!dYs && !dweights)) return r;
        if (!positions || !weights || (dYs && !offsets) || (D > 0 && (!dY || (dweights && !Ys))))
            return report_errorf(GBR_ERR_INVALID, "%s: NULL buffer", fn);
        const int64_t es = a.bf16 ? 2 : 4, n = T * top_k;
        const View vd = {"dY", dY, T, D, lddy, es}, vi = {"Ys", dweights ? Ys : nullptr, n, D, ldys, es},
                   vp = {"positions", positions, 1, n, n, 4}, vw = {"weights", weights, 1, n, n, 4},
                   vf = {"offsets", dYs ? offsets : nullptr, 1, num_experts + 1, num_experts + 1, 4},
                   vo = {"dYs", dYs, n, D, lddys, es}, vdw = {"dweights", dweights, 1, n, n, 4};
        if ((r = check_outputs(fn, {&vd, &vi, &vp, &vw, &vf}, {&vo, &vdw})) != GBR_OK) return r;
        LibCtx c;
        if ((r = lib_ctx(&c)) != GBR_OK) return r;
        a.dY = {dY, lddy}, a.Ys = {vi.p, ldys}, a.dYs = {dYs, lddys};
        a.positions = positions, a.offsets = offsets, a.weights = weights, a.dweights = dweights;
        a.T = int32_t(T), a.k = int32_t(top_k), a.D = int32_t(D), a.experts = num_experts;
        return launch_moe_combine_grad(a, c, reinterpret_cast<cudaStream_t>(stream));
    });
}

int64_t mxfp4_data_bytes(int64_t rows, int64_t cols) {
    return rows < 0 || cols < 0 || rows >= kLim || cols >= kLim ? -1 : rows * ((cols + 31) / 32) * 16;
}
int64_t mxfp4_scale_bytes(int64_t rows, int64_t cols) {
    return rows < 0 || cols < 0 || rows >= kLim || cols >= kLim ? -1 : ((rows + 127) / 128) * ((cols + 127) / 128) * 512;
}

int quantize_mxfp4(const void* X, int64_t ldx, void* data, void* scales, int64_t rows, int64_t cols, int transposed,
                   int dtype, gbr_stream_t stream) {
    const char* fn = "quantize_mxfp4";
    return guarded(fn, [&]() -> int {
        Mxfp4Quantize a = {};
        int r = check_mx(fn, rows, cols, dtype, &a.bf16);
        if (r != GBR_OK) return r;
        if (transposed != 0 && transposed != 1) return report_errorf(GBR_ERR_INVALID, "%s: transposed must be 0 or 1", fn);
        if (rows == 0 || cols == 0) return GBR_OK;
        if (!X || !data || !scales) return report_errorf(GBR_ERR_INVALID, "%s: NULL buffer", fn);
        const int64_t es = a.bf16 ? 2 : 4, nd = mxfp4_data_bytes(rows, cols), ns = mxfp4_scale_bytes(rows, cols);
        const View vx = {"X", X, transposed ? cols : rows, transposed ? rows : cols, ldx, es},
                   vd = {"data", data, 1, nd, nd, 1}, vs = {"scales", scales, 1, ns, ns, 1};
        if ((r = check_outputs(fn, {&vx}, {&vd, &vs})) != GBR_OK || (r = check_mx_pointers(fn, data, scales)) != GBR_OK)
            return r;
        LibCtx c;
        if ((r = lib_ctx(&c)) != GBR_OK) return r;
        a.X = {X, ldx};
        a.data = static_cast<uint8_t*>(data), a.scales = static_cast<uint8_t*>(scales);
        a.rows = int32_t(rows), a.cols = int32_t(cols), a.transposed = transposed != 0;
        return launch_mxfp4_quantize(a, c, reinterpret_cast<cudaStream_t>(stream));
    });
}

int dequantize_mxfp4(const void* data, const void* scales, void* X, int64_t ldx, int64_t rows, int64_t cols, int dtype,
                     gbr_stream_t stream) {
    const char* fn = "dequantize_mxfp4";
    return guarded(fn, [&]() -> int {
        Mxfp4Dequantize a = {};
        int r = check_mx(fn, rows, cols, dtype, &a.bf16);
        if (r != GBR_OK || rows == 0 || cols == 0) return r;
        if (!X || !data || !scales) return report_errorf(GBR_ERR_INVALID, "%s: NULL buffer", fn);
        const int64_t es = a.bf16 ? 2 : 4, nd = mxfp4_data_bytes(rows, cols), ns = mxfp4_scale_bytes(rows, cols);
        const View vx = {"X", X, rows, cols, ldx, es}, vd = {"data", data, 1, nd, nd, 1}, vs = {"scales", scales, 1, ns, ns, 1};
        if ((r = check_outputs(fn, {&vd, &vs}, {&vx})) != GBR_OK || (r = check_mx_pointers(fn, data, scales)) != GBR_OK)
            return r;
        LibCtx c;
        if ((r = lib_ctx(&c)) != GBR_OK) return r;
        a.X = {X, ldx};
        a.data = static_cast<const uint8_t*>(data), a.scales = static_cast<const uint8_t*>(scales);
        a.rows = int32_t(rows), a.cols = int32_t(cols);
        return launch_mxfp4_dequantize(a, c, reinterpret_cast<cudaStream_t>(stream));
    });
}

int gemm_mxfp4(const void* A, const void* A_scales, const void* B, const void* B_scales, const float* bias,
               const void* residual, int64_t ldr, void* C, int64_t ldc, int64_t M, int64_t N, int64_t K, int act,
               gbr_stream_t stream) {
    const char* fn = "gemm_mxfp4";
    return guarded(fn, [&]() -> int {
        if (act < 0 || act >= kActs) return report_errorf(GBR_ERR_INVALID, "%s: unknown activation %d", fn, act);
        int r = check_sizes(fn, M, N, K);
        if (r == GBR_OK) r = check_columns(fn, std::max({M, N, K}));
        if (r != GBR_OK || M == 0 || N == 0) return r;
        if (!C || (K > 0 && (!A || !A_scales || !B || !B_scales)))
            return report_errorf(GBR_ERR_INVALID, "%s: NULL buffer", fn);
        if (K > 0 && ((r = check_mx_pointers(fn, A, A_scales)) != GBR_OK || (r = check_mx_pointers(fn, B, B_scales)) != GBR_OK))
            return r;
        const int64_t na = mxfp4_data_bytes(M, K), nb = mxfp4_data_bytes(N, K), sa = mxfp4_scale_bytes(M, K),
                      sb = mxfp4_scale_bytes(N, K);
        const View va = {"A", A, 1, na, na, 1}, vas = {"A's scales", A_scales, 1, sa, sa, 1}, vb = {"B", B, 1, nb, nb, 1},
                   vbs = {"B's scales", B_scales, 1, sb, sb, 1}, vr = {"residual", residual, M, N, ldr, 2},
                   vc = {"C", C, M, N, ldc, 2}, vbias = {"bias", bias, 1, N, N, 4};
        for (const View* v : {&vr, &vc, &vbias})
            if ((r = check_view(fn, *v)) != GBR_OK) return r;
        for (const View* v : {&va, &vas, &vb, &vbs, &vbias, &vr})
            if (share(vc, *v) && !(v == &vr && same(vc, vr)))
                return report_errorf(GBR_ERR_INVALID, "%s: C overlaps %s", fn, v->name);
        LibCtx c;
        if ((r = lib_ctx(&c)) != GBR_OK) return r;
        Mxfp4Args a = {};
        a.A = static_cast<const uint8_t*>(A), a.As = static_cast<const uint8_t*>(A_scales);
        a.B = static_cast<const uint8_t*>(B), a.Bs = static_cast<const uint8_t*>(B_scales);
        a.bias = bias;
        a.R = {residual, ldr}, a.C = {C, ldc};
        a.M = int32_t(M), a.N = int32_t(N), a.blocks = int32_t((K + 31) / 32);
        a.act = act;
        return launch_mxfp4(a, c, reinterpret_cast<cudaStream_t>(stream));
    });
}

// The self tests of the operators' pipelines: the normal call with one stage
// left unfilled (see gbr_selftest_gemm_skip_load).
int gbr_selftest_linear_skip_load(const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K, int cta,
                                  int item, uint64_t limit_ns, gbr_stream_t stream) {
    int r = begin_injection(cta, item, limit_ns);
    if (r != GBR_OK) return r;
    r = gemm_bias_act(A, K, B, N, nullptr, nullptr, 0, C, N, nullptr, 0, M, N, K, GBR_BF16, GBR_ACT_NONE, 0.0, 0, 0,
                      stream);
    end_injection();
    return r;
}

int gbr_selftest_moe_skip_load(const void* X, const float* Wr, const void* W1, const void* W2, void* Y, int64_t T,
                               int64_t D, int64_t F, int num_experts, int top_k, int cta, int item,
                               uint64_t limit_ns, gbr_stream_t stream) {
    int r = begin_injection(cta, item, limit_ns);
    if (r != GBR_OK) return r;
    r = moe_layer(X, Wr, W1, nullptr, W2, nullptr, Y, nullptr, nullptr, T, D, F, num_experts, top_k, GBR_ACT_RELU, 0,
                  GBR_BF16, stream);
    end_injection();
    return r;
}

int gbr_selftest_mxfp4_skip_load(const void* A, const void* A_scales, const void* B, const void* B_scales, void* C,
                                 int64_t M, int64_t N, int64_t K, int cta, int item, uint64_t limit_ns,
                                 gbr_stream_t stream) {
    int r = begin_injection(cta, item, limit_ns);
    if (r != GBR_OK) return r;
    r = gemm_mxfp4(A, A_scales, B, B_scales, nullptr, nullptr, 0, C, N, M, N, K, GBR_ACT_NONE, stream);
    end_injection();
    return r;
}

}  // extern "C"
