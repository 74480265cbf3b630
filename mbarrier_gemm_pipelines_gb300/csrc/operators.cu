// operators.cu -- entry points of the feed-forward operators (include/gbr.h):
// validation, scratch and the order of the launches.
#include "gbr.h"
#include "operators.h"

#include <cmath>
#include <exception>
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

}  // extern "C"
