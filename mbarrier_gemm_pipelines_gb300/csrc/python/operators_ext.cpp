// operators_ext.cpp -- Python binding of the feed-forward operators (the end of
// include/gbr.h): checks of the tensors, allocation of the outputs, the call.
// No arithmetic, no CPU path.  A compiled module because these operators'
// smallest calls take the GPU a few microseconds: with the same checks in
// Python and the call through ctypes one token's gemm_bias_act took the host
// 12 us, a small dropout_add 10 and the gradients of a 301 x 520 x 1000 product
// 30; through this file 4.0, 3.5 and 11.
//
// _operators.py holds the functions that users call, with their defaults and
// documentation, and passes every argument on by position.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/record_function.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdarg>
#include <cstdint>
#include <exception>

#include "gbr.h"

namespace {

PyObject* g_error = nullptr;       // mbarrier_gemm_pipelines_gb300.GbrError
PyObject* g_no_memory = nullptr;   // torch.OutOfMemoryError

// Raised by the checks once a Python exception is set.
struct Refused {};

[[noreturn]] void refuse(PyObject* kind, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    PyErr_FormatV(kind, fmt, ap);
    va_end(ap);
    throw Refused();
}

void check(int code) {
    if (code == GBR_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", code, gbr_last_error());
    if (e != nullptr) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Refused();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}

// The device of the call: the first tensor's, which has to be the current one.
int first_device(const at::Tensor& t, const char* name) {
    if (!t.is_cuda())
        refuse(PyExc_ValueError, "%s must be a CUDA tensor (this library has no CPU path)", name);
    const int dev = t.get_device(), now = c10::cuda::current_device();
    if (dev != now)
        refuse(PyExc_ValueError, "%s is on cuda:%d, the current device is cuda:%d", name, dev, now);
    return dev;
}

void check_type(const at::Tensor& t, const char* name, at::ScalarType type, int dev) {
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, "%s has dtype %s, expected %s", name, c10::toString(t.scalar_type()),
               c10::toString(type));
    if (!t.is_cuda())
        refuse(PyExc_ValueError, "%s must be a CUDA tensor (this library has no CPU path)", name);
    if (t.get_device() != dev)
        refuse(PyExc_ValueError, "%s is on cuda:%d, not on cuda:%d", name, int(t.get_device()), dev);
}

// A 2-D tensor whose rows are contiguous.
struct Mat {
    void* p = nullptr;
    int64_t rows = 0, cols = 0, ld = 0;
};

Mat mat(const at::Tensor& t, const char* name, at::ScalarType type, int dev) {
    check_type(t, name, type, dev);
    if (t.dim() != 2) refuse(PyExc_ValueError, "%s must be 2-D", name);
    Mat m;
    m.p = t.data_ptr();
    m.rows = t.size(0);
    m.cols = t.size(1);
    if (m.cols > 1 && t.stride(1) != 1) refuse(PyExc_ValueError, "the rows of %s must be contiguous", name);
    m.ld = m.rows > 1 ? t.stride(0) : (m.cols > 0 ? m.cols : 1);
    return m;
}

Mat mat_of(PyObject* o, const char* name, at::ScalarType type, int dev, int64_t rows, int64_t cols) {
    const Mat m = mat(tensor(o, name), name, type, dev);
    if (m.rows != rows || m.cols != cols)
        refuse(PyExc_ValueError, "%s must be [%lld, %lld], got [%lld, %lld]", name, static_cast<long long>(rows),
               static_cast<long long>(cols), static_cast<long long>(m.rows), static_cast<long long>(m.cols));
    return m;
}

// A contiguous tensor of that shape.
void* packed(const at::Tensor& t, const char* name, at::ScalarType type, int dev, at::IntArrayRef shape) {
    check_type(t, name, type, dev);
    if (t.sizes() != shape) {
        PyObject* want = PyList_New(0);
        for (int64_t n : shape) {
            PyObject* v = PyLong_FromLongLong(n);
            PyList_Append(want, v);
            Py_XDECREF(v);
        }
        PyErr_Format(PyExc_ValueError, "%s must have shape %R", name, want);
        Py_XDECREF(want);
        throw Refused();
    }
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    return t.data_ptr();
}

int act_code(PyObject* o) {
    static const char* const names[] = {"none", "relu", "gelu", "gelu_tanh", "silu"};
    for (int i = 0; PyUnicode_Check(o) && i < 5; ++i)
        if (PyUnicode_CompareWithASCIIString(o, names[i]) == 0) return i;
    refuse(PyExc_ValueError, "act must be one of none, relu, gelu, gelu_tanh, silu, got %R", o);
}

uint64_t bits64(PyObject* o, const char* name) {
    PyObject* i = PyNumber_Index(o);
    const unsigned long long v = i != nullptr ? PyLong_AsUnsignedLongLong(i) : 0;
    Py_XDECREF(i);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse(PyExc_ValueError, "%s must be an integer in [0, 2^64)", name);
    }
    return v;
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return v;
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}

// For the int arguments of the library, which refuses what this cuts off.
int as_int(int64_t v) { return int(std::max<int64_t>(-1, std::min<int64_t>(v, INT32_MAX))); }

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused();
    return v != 0;
}

// Whether somebody would see at::empty: a dispatch mode or another key that was added to this thread, or a profiler.  (The
// fill of new memory under deterministic algorithms is left out: the library writes every output whole.)
bool outputs_watched() {
    const c10::DispatchKeySet added = c10::impl::tls_local_dispatch_key_set().included_ - c10::default_included_set;
    return !added.empty() || at::getStepCallbacksUnlessEmpty(at::RecordScope::FUNCTION).has_value();
}

// The call's stream: the current one, or the `stream` argument, which is then the current one until the call
// ends, so that the outputs made here are that stream's to PyTorch's allocator.  From the current stream's share it could
// hand out memory that a kernel there still reads, and give an output away while the other stream writes it.
class CallStream {
public:
    CallStream(PyObject* o, int dev)
        : handle_(c10::cuda::getCurrentCUDAStream(dev).stream()), device_(dev), watched_(outputs_watched()) {
        if (o == Py_None) return;
        PyObject* v = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
        if (v == nullptr) throw Refused();
        const cudaStream_t given = static_cast<cudaStream_t>(PyLong_AsVoidPtr(v));
        Py_DECREF(v);
        if (given == nullptr && PyErr_Occurred()) throw Refused();
        if (given == handle_) return;
        handle_ = given;
        // cudaStreamLegacy is the null stream by another name.
        guard_.reset_stream(given == nullptr || given == cudaStreamLegacy
                                ? c10::cuda::getDefaultCUDAStream(dev)
                                : c10::cuda::getStreamFromExternal(given, c10::DeviceIndex(dev)));
    }
    operator gbr_stream_t() const { return reinterpret_cast<gbr_stream_t>(handle_); }
    int device() const { return device_; }
    bool watched() const { return watched_; }

private:
    cudaStream_t handle_;
    int device_;
    bool watched_;
    c10::cuda::OptionalCUDAStreamGuard guard_;
};

// A tensor of the caller's that the call has written: its version moves, so that autograd refuses a graph that saved
// it before.  (A tensor made in inference mode has none.)
PyObject* written(PyObject* o) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    return Py_NewRef(o);
}

// A new tensor on the call's stream, past the dispatcher where nobody watches it: at::empty took 1.3 us of the host's time,
// more than half of a call with two outputs and one launch.
[[gnu::cold, gnu::noinline]] at::Tensor fresh_seen(at::IntArrayRef shape, at::ScalarType type, c10::Device on) {
    at::Tensor t = at::empty(shape, at::TensorOptions(type).device(on));
    packed(t, "a new output", type, on.index(), shape);      // a mode may give anything
    return t;
}
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const CallStream& st) {
    const c10::Device on(c10::kCUDA, c10::DeviceIndex(st.device()));
    if (C10_UNLIKELY(st.watched())) return fresh_seen(shape, type, on);
    return at::Tensor(at::detail::empty_cuda(shape, type, on, std::nullopt));
}

// An output: the caller's, or a new one.
struct Out {
    PyObject* given = nullptr;
    at::Tensor made;
    Mat m;
    PyObject* wrap() const { return given != nullptr ? written(given) : THPVariable_Wrap(made); }
};

Out out_mat(PyObject* o, const char* name, const at::Tensor& like, const CallStream& st, int64_t rows, int64_t cols) {
    Out r;
    if (o != Py_None) {
        r.given = o;
        r.m = mat_of(o, name, like.scalar_type(), st.device(), rows, cols);
    } else {
        r.made = fresh({rows, cols}, like.scalar_type(), st);
        r.m.p = r.made.data_ptr();
        r.m.rows = rows, r.m.cols = cols, r.m.ld = cols > 0 ? cols : 1;
    }
    return r;
}

// Runs `body` with C++ exceptions turned into Python's; an output that finds no memory raises what torch.empty would.
template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& body) {
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused&) {
        return nullptr;
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(g_no_memory, e.what_without_backtrace());
        return nullptr;
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// The library call itself runs without the interpreter's lock.
template <class F>
void call(F&& f) {
    int code;
    Py_BEGIN_ALLOW_THREADS
    code = f();
    Py_END_ALLOW_THREADS
    check(code);
}

// dropout_add(X, residual, p, seed, offset, Y, stream)
PyObject* dropout_add_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        const at::Tensor& X = tensor(a[0], "X");
        const at::ScalarType type = X.scalar_type();
        if (type != at::kBFloat16 && type != at::kFloat)
            refuse(PyExc_TypeError, "X must be bf16 or fp32, got %s", c10::toString(type));
        const int dev = first_device(X, "X");
        if (X.dim() == 0) refuse(PyExc_ValueError, "X must have at least one dimension");
        const CallStream st(a[6], dev);
        const bool has_r = a[1] != Py_None, has_y = a[5] != Py_None;
        at::Tensor made;
        if (!has_y) made = fresh(X.sizes(), type, st);
        const at::Tensor& Y = has_y ? tensor(a[5], "Y") : made;
        Mat x, r, y;
        if (X.dim() == 2) {
            x = mat(X, "X", type, dev);
            if (has_r) r = mat_of(a[1], "residual", type, dev, x.rows, x.cols);
            y = has_y ? mat_of(a[5], "Y", type, dev, x.rows, x.cols) : mat(Y, "Y", type, dev);
        } else {
            // Rows of the last dimension.
            x.p = packed(X, "X", type, dev, X.sizes());
            x.cols = X.size(-1);
            x.rows = x.cols > 0 ? X.numel() / x.cols : 0;
            x.ld = x.cols > 0 ? x.cols : 1;
            r = y = x;
            r.p = has_r ? packed(tensor(a[1], "residual"), "residual", type, dev, X.sizes()) : nullptr;
            y.p = packed(Y, "Y", type, dev, X.sizes());
        }
        const double p = number(a[2]);
        const uint64_t seed = bits64(a[3], "seed"), offset = bits64(a[4], "offset");
        call([&] {
            return dropout_add(x.p, x.ld, has_r ? r.p : nullptr, r.ld, y.p, y.ld, x.rows, x.cols,
                               type == at::kBFloat16 ? GBR_BF16 : GBR_F32_FFMA, p, seed, offset, st);
        });
        return has_y ? written(a[5]) : THPVariable_Wrap(made);
    });
}

// gemm_bias_act(A, B, bias, residual, act, p, seed, offset, C, Z, return_z, stream)
PyObject* gemm_bias_act_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const at::Tensor &tA = tensor(a[0], "A"), &tB = tensor(a[1], "B");
        const int dev = first_device(tA, "A");
        const Mat A = mat(tA, "A", at::kBFloat16, dev), B = mat(tB, "B", at::kBFloat16, dev);
        if (A.cols != B.rows)
            refuse(PyExc_ValueError, "shape mismatch: A [%lld, %lld], B [%lld, %lld]", static_cast<long long>(A.rows),
                   static_cast<long long>(A.cols), static_cast<long long>(B.rows), static_cast<long long>(B.cols));
        const int64_t M = A.rows, N = B.cols;
        const float* bias = nullptr;
        if (a[2] != Py_None)
            bias = static_cast<const float*>(packed(tensor(a[2], "bias"), "bias", at::kFloat, dev, {N}));
        Mat R;
        if (a[3] != Py_None) R = mat_of(a[3], "residual", at::kBFloat16, dev, M, N);
        const int act = act_code(a[4]);
        const double p = number(a[5]);
        const uint64_t seed = bits64(a[6], "seed"), offset = bits64(a[7], "offset");
        const bool want_z = a[9] != Py_None || truth(a[10]);
        const CallStream st(a[11], dev);
        const Out C = out_mat(a[8], "C", tA, st, M, N);
        Out Z;
        if (want_z) Z = out_mat(a[9], "Z", tA, st, M, N);
        call([&] {
            return gemm_bias_act(A.p, A.ld, B.p, B.ld, bias, R.p, R.ld, C.m.p, C.m.ld, Z.m.p, Z.m.ld, M, N, A.cols,
                                 GBR_BF16, act, p, seed, offset, st);
        });
        if (!want_z) return C.wrap();
        return Py_BuildValue("NN", C.wrap(), Z.wrap());
    });
}

// gemm_bias_act_backward(dC, A, B, Z, act, p, seed, offset, dA, dB, dbias, needs, stream)
PyObject* gemm_bias_act_backward_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        const at::Tensor &tdC = tensor(a[0], "dC"), &tA = tensor(a[1], "A"), &tB = tensor(a[2], "B");
        const int dev = first_device(tdC, "dC");
        const Mat A = mat(tA, "A", at::kBFloat16, dev), B = mat(tB, "B", at::kBFloat16, dev);
        if (A.cols != B.rows)
            refuse(PyExc_ValueError, "shape mismatch: A [%lld, %lld], B [%lld, %lld]", static_cast<long long>(A.rows),
                   static_cast<long long>(A.cols), static_cast<long long>(B.rows), static_cast<long long>(B.cols));
        const int64_t M = A.rows, K = A.cols, N = B.cols;
        const Mat dC = mat_of(a[0], "dC", at::kBFloat16, dev, M, N);
        const int act = act_code(a[4]);
        Mat Z;
        if (a[3] != Py_None) Z = mat_of(a[3], "Z", at::kBFloat16, dev, M, N);
        else if (act != GBR_ACT_NONE)
            refuse(PyExc_ValueError, "Z (the pre-activation of the forward call) is needed for act=%R", a[4]);
        const double p = number(a[5]);
        const uint64_t seed = bits64(a[6], "seed"), offset = bits64(a[7], "offset");
        PyObject* needs = PySequence_Fast(a[11], "needs must be three truth values");
        if (needs == nullptr) throw Refused();
        bool want[3] = {};
        const bool three = PySequence_Fast_GET_SIZE(needs) == 3;
        int bad = 0;
        for (int i = 0; three && i < 3; ++i) {
            const int v = PyObject_IsTrue(PySequence_Fast_GET_ITEM(needs, i));
            bad |= v < 0;
            want[i] = v > 0;
        }
        Py_DECREF(needs);
        if (bad) throw Refused();
        if (!three) refuse(PyExc_ValueError, "needs must be three truth values");
        const CallStream st(a[12], dev);
        Out dA, dB, db;
        if (want[0]) dA = out_mat(a[8], "dA", tA, st, M, K);
        if (want[1]) dB = out_mat(a[9], "dB", tA, st, K, N);
        if (want[2]) {
            if (a[10] != Py_None) {
                db.given = a[10];
                db.m.p = packed(tensor(a[10], "dbias"), "dbias", at::kFloat, dev, {N});
            } else {
                db.made = fresh({N}, at::kFloat, st);
                db.m.p = db.made.data_ptr();
            }
        }
        call([&] {
            return gemm_bias_act_backward(dC.p, dC.ld, A.p, A.ld, B.p, B.ld, Z.p, Z.ld, dA.m.p, dA.m.ld, dB.m.p,
                                          dB.m.ld, static_cast<float*>(db.m.p), M, N, K, GBR_BF16, act, p, seed,
                                          offset, st);
        });
        return Py_BuildValue("NNN", want[0] ? dA.wrap() : Py_NewRef(Py_None),
                             want[1] ? dB.wrap() : Py_NewRef(Py_None), want[2] ? db.wrap() : Py_NewRef(Py_None));
    });
}

// moe_layer(X, Wr, W1, b1, W2, b2, top_k, act, gated, Y, return_routing, stream)
PyObject* moe_layer_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const at::Tensor &X = tensor(a[0], "X"), &W2 = tensor(a[4], "W2");
        const int dev = first_device(X, "X");
        if (X.dim() != 2 || W2.dim() != 3) refuse(PyExc_ValueError, "X must be 2-D, W1 and W2 3-D");
        const int64_t T = X.size(0), D = X.size(1), E = W2.size(0), F = W2.size(1);
        const bool gated = truth(a[8]);
        const int64_t F1 = gated ? 2 * F : F, top_k = integer(a[6]);
        const int act = act_code(a[7]);
        const void* x = packed(X, "X", at::kBFloat16, dev, {T, D});
        const void* wr = packed(tensor(a[1], "Wr"), "Wr", at::kFloat, dev, {D, E});
        const void* w1 = packed(tensor(a[2], "W1"), "W1", at::kBFloat16, dev, {E, D, F1});
        const void* w2 = packed(W2, "W2", at::kBFloat16, dev, {E, F, D});
        const void* b1 = a[3] == Py_None ? nullptr : packed(tensor(a[3], "b1"), "b1", at::kFloat, dev, {E, F1});
        const void* b2 = a[5] == Py_None ? nullptr : packed(tensor(a[5], "b2"), "b2", at::kFloat, dev, {E, D});
        const CallStream st(a[11], dev);
        Out Y;
        if (a[9] != Py_None) {
            Y.given = a[9];
            Y.m.p = packed(tensor(a[9], "Y"), "Y", at::kBFloat16, dev, {T, D});
        } else {
            Y.made = fresh({T, D}, at::kBFloat16, st);
            Y.m.p = Y.made.data_ptr();
        }
        const bool routing = truth(a[10]);
        at::Tensor ids, weights;
        if (routing) {
            const int64_t k = top_k < 0 || top_k > E ? 0 : top_k;       // a wrong top_k is refused by the call
            ids = fresh({T, k}, at::kLong, st);
            weights = fresh({T, k}, at::kFloat, st);
        }
        call([&] {
            return moe_layer(x, static_cast<const float*>(wr), w1, static_cast<const float*>(b1), w2,
                             static_cast<const float*>(b2), Y.m.p,
                             routing ? static_cast<int64_t*>(ids.data_ptr()) : nullptr,
                             routing ? static_cast<float*>(weights.data_ptr()) : nullptr, T, D, F, as_int(E),
                             as_int(top_k), act, gated ? 1 : 0, GBR_BF16, st);
        });
        if (!routing) return Y.wrap();
        return Py_BuildValue("NNN", Y.wrap(), THPVariable_Wrap(ids), THPVariable_Wrap(weights));
    });
}

// bf16 or fp32.
at::ScalarType element_type(const at::Tensor& t, const char* name) {
    const at::ScalarType type = t.scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat)
        refuse(PyExc_TypeError, "%s must be bf16 or fp32, got %s", name, c10::toString(type));
    return type;
}
int type_code(at::ScalarType type) { return type == at::kBFloat16 ? GBR_BF16 : GBR_F32_FFMA; }

const float* optional_vector(PyObject* o, const char* name, int dev, int64_t n) {
    return o == Py_None ? nullptr : static_cast<const float*>(packed(tensor(o, name), name, at::kFloat, dev, {n}));
}

// The `count` truth values of `needs`.
void truths(PyObject* o, bool* want, int count) {
    PyObject* needs = PySequence_Fast(o, "needs must be a sequence of truth values");
    if (needs == nullptr) throw Refused();
    const bool fits = PySequence_Fast_GET_SIZE(needs) == count;
    int bad = 0;
    for (int i = 0; fits && i < count; ++i) {
        const int v = PyObject_IsTrue(PySequence_Fast_GET_ITEM(needs, i));
        bad |= v < 0;
        want[i] = v > 0;
    }
    Py_DECREF(needs);
    if (bad) throw Refused();
    if (!fits) refuse(PyExc_ValueError, "needs must be %d truth values", count);
}

// A contiguous output: the caller's, or a new one.
Out out_packed(PyObject* o, const char* name, at::ScalarType type, const CallStream& st, at::IntArrayRef shape) {
    Out r;
    if (o != Py_None) {
        r.given = o;
        r.m.p = packed(tensor(o, name), name, type, st.device(), shape);
    } else {
        r.made = fresh(shape, type, st);
        r.m.p = r.made.data_ptr();
    }
    return r;
}

PyObject* wrap_or_none(bool want, const Out& o) { return want ? o.wrap() : Py_NewRef(Py_None); }

// residual_norm(X, R, post, gate, scale, pre, eps, S, H, stream)
PyObject* residual_norm_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject* {
        const at::Tensor& tX = tensor(a[0], "X");
        const at::ScalarType type = element_type(tX, "X");
        const int dev = first_device(tX, "X");
        const Mat X = mat(tX, "X", type, dev);
        Mat R, G;
        if (a[1] != Py_None) R = mat_of(a[1], "R", type, dev, X.rows, X.cols);
        const float* post = optional_vector(a[2], "post", dev, X.cols);
        if (a[3] != Py_None) {
            G = mat(tensor(a[3], "gate"), "gate", type, dev);
            if (G.cols != X.cols)
                refuse(PyExc_ValueError, "gate must have %lld columns, got %lld", static_cast<long long>(X.cols),
                       static_cast<long long>(G.cols));
            if (G.rows == 0 ? X.rows != 0 : X.rows % G.rows != 0)
                refuse(PyExc_ValueError, "the %lld rows of X are no multiple of gate's %lld",
                       static_cast<long long>(X.rows), static_cast<long long>(G.rows));
        }
        const double scale = number(a[4]), eps = number(a[6]);
        const float* pre = optional_vector(a[5], "pre", dev, X.cols);
        const bool want_h = a[5] != Py_None;
        if (!want_h && a[8] != Py_None) refuse(PyExc_ValueError, "H needs pre");
        const CallStream st(a[9], dev);
        // Where nothing is added, scaled or normalised the sum is X itself, unless H is written over it.
        const bool same = a[7] == Py_None && a[1] == Py_None && a[2] == Py_None && a[3] == Py_None && scale == 1.0 &&
                          (a[8] == Py_None || tensor(a[8], "H").data_ptr() != X.p);
        Out S;
        if (!same) S = out_mat(a[7], "S", tX, st, X.rows, X.cols);
        Out H;
        if (want_h) H = out_mat(a[8], "H", tX, st, X.rows, X.cols);
        // Vectors of no columns have no address.
        if (X.cols > 0)
            call([&] {
                return residual_norm(X.p, X.ld, R.p, R.ld, post, G.p, G.ld, G.rows, scale, pre, eps, S.m.p, S.m.ld, H.m.p,
                                     H.m.ld, X.rows, X.cols, type_code(type), st);
            });
        return Py_BuildValue("NN", same ? Py_NewRef(a[0]) : S.wrap(), wrap_or_none(want_h, H));
    });
}

// residual_norm_backward(dS, dH, X, S, post, gate, scale, pre, eps, dX, dR, dpost, dgate, dpre, needs, stream)
PyObject* residual_norm_backward_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 16, [&]() -> PyObject* {
        const bool has_post = a[4] != Py_None, has_gate = a[5] != Py_None, has_pre = a[7] != Py_None;
        if (a[0] == Py_None && !has_pre) refuse(PyExc_ValueError, "dS is needed without pre");
        const int first = a[0] != Py_None ? 0 : 1;
        const char* first_name = first == 0 ? "dS" : "dH";
        const at::Tensor& like = tensor(a[first], first_name);
        const at::ScalarType type = element_type(like, first_name);
        const int dev = first_device(like, first_name);
        const Mat m = mat(like, first_name, type, dev);
        const int64_t rows = m.rows, cols = m.cols;
        Mat dS, dH, X, S, G;
        if (a[0] != Py_None) dS = m;
        if (has_pre) {
            if (a[1] == Py_None || a[3] == Py_None) refuse(PyExc_ValueError, "dH and S are needed with pre");
            dH = mat_of(a[1], "dH", type, dev, rows, cols);
            S = mat_of(a[3], "S", type, dev, rows, cols);
        }
        if (has_post || has_gate) {
            if (a[2] == Py_None) refuse(PyExc_ValueError, "X is needed with post or gate");
            X = mat_of(a[2], "X", type, dev, rows, cols);
        }
        const float* post = optional_vector(a[4], "post", dev, cols);
        if (has_gate) {
            G = mat(tensor(a[5], "gate"), "gate", type, dev);
            if (G.cols != cols || (G.rows == 0 ? rows != 0 : rows % G.rows != 0))
                refuse(PyExc_ValueError, "gate must have %lld columns and rows that divide %lld",
                       static_cast<long long>(cols), static_cast<long long>(rows));
        }
        const double scale = number(a[6]), eps = number(a[8]);
        const float* pre = optional_vector(a[7], "pre", dev, cols);
        bool want[5] = {};
        truths(a[14], want, 5);
        want[2] = want[2] && has_post, want[3] = want[3] && has_gate, want[4] = want[4] && has_pre;
        const CallStream st(a[15], dev);
        Out dX, dR, dpost, dG, dpre;
        if (want[0]) dX = out_mat(a[9], "dX", like, st, rows, cols);
        if (want[1]) dR = out_mat(a[10], "dR", like, st, rows, cols);
        if (want[2]) dpost = out_packed(a[11], "dpost", at::kFloat, st, {cols});
        if (want[3]) dG = out_mat(a[12], "dgate", like, st, G.rows, cols);
        if (want[4]) dpre = out_packed(a[13], "dpre", at::kFloat, st, {cols});
        if (cols > 0)
            call([&] {
                return residual_norm_backward(dS.p, dS.ld, dH.p, dH.ld, X.p, X.ld, S.p, S.ld, post, G.p, G.ld, G.rows, scale,
                                              pre, eps, dX.m.p, dX.m.ld, dR.m.p, dR.m.ld, static_cast<float*>(dpost.m.p),
                                              dG.m.p, dG.m.ld, static_cast<float*>(dpre.m.p), rows, cols, type_code(type),
                                              st);
            });
        return Py_BuildValue("NNNNN", wrap_or_none(want[0], dX), wrap_or_none(want[1], dR), wrap_or_none(want[2], dpost),
                             wrap_or_none(want[3], dG), wrap_or_none(want[4], dpre));
    });
}

// moe_sort(expert_ids, num_experts, positions, offsets, stream)
PyObject* moe_sort_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject* {
        const at::Tensor& ids = tensor(a[0], "expert_ids");
        const int dev = first_device(ids, "expert_ids");
        if (ids.dim() != 2) refuse(PyExc_ValueError, "expert_ids must be 2-D");
        const void* p = packed(ids, "expert_ids", at::kLong, dev, ids.sizes());
        const int64_t E = integer(a[1]);
        if (E < 1 || E > INT32_MAX - 1) refuse(PyExc_ValueError, "num_experts must be positive");
        const CallStream st(a[4], dev);
        const Out pos = out_packed(a[2], "positions", at::kInt, st, ids.sizes());
        const Out off = out_packed(a[3], "offsets", at::kInt, st, {std::min<int64_t>(E, 1 << 20) + 1});
        call([&] {
            return moe_sort(static_cast<const int64_t*>(p), ids.numel(), as_int(E), static_cast<int32_t*>(pos.m.p),
                            static_cast<int32_t*>(off.m.p), st);
        });
        return Py_BuildValue("NN", pos.wrap(), off.wrap());
    });
}

// Positions [T, top_k] and, unless null, the offsets of the experts.
struct Places {
    int64_t T = 0, k = 0, experts = 1;
    const int32_t *positions = nullptr, *offsets = nullptr;
};
Places places(PyObject* positions, PyObject* offsets, int dev) {
    const at::Tensor& p = tensor(positions, "positions");
    if (p.dim() != 2) refuse(PyExc_ValueError, "positions must be 2-D");
    Places r;
    r.positions = static_cast<const int32_t*>(packed(p, "positions", at::kInt, dev, p.sizes()));
    r.T = p.size(0), r.k = p.size(1);
    if (offsets != nullptr) {
        const at::Tensor& o = tensor(offsets, "offsets");
        if (o.dim() != 1 || o.size(0) < 2) refuse(PyExc_ValueError, "offsets must be [num_experts + 1]");
        r.offsets = static_cast<const int32_t*>(packed(o, "offsets", at::kInt, dev, o.sizes()));
        r.experts = o.size(0) - 1;
    }
    return r;
}

// moe_dispatch(X, positions, offsets, Xs, stream)
PyObject* moe_dispatch_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject* {
        const at::Tensor& tX = tensor(a[0], "X");
        const at::ScalarType type = element_type(tX, "X");
        const int dev = first_device(tX, "X");
        const Mat X = mat(tX, "X", type, dev);
        const Places p = places(a[1], a[2], dev);
        if (p.T != X.rows)
            refuse(PyExc_ValueError, "positions are of %lld tokens, X has %lld rows", static_cast<long long>(p.T),
                   static_cast<long long>(X.rows));
        const CallStream st(a[4], dev);
        const Out Xs = out_mat(a[3], "Xs", tX, st, p.T * p.k, X.cols);
        call([&] {
            return moe_dispatch(X.p, X.ld, p.positions, p.offsets, as_int(p.experts), Xs.m.p, Xs.m.ld, p.T, p.k, X.cols,
                                type_code(type), st);
        });
        return Xs.wrap();
    });
}

// moe_combine(Ys, positions, weights, residual, Y, stream)
PyObject* moe_combine_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject* {
        const at::Tensor& tYs = tensor(a[0], "Ys");
        const at::ScalarType type = element_type(tYs, "Ys");
        const int dev = first_device(tYs, "Ys");
        const Mat Ys = mat(tYs, "Ys", type, dev);
        const Places p = places(a[1], nullptr, dev);
        const void* w = a[2] == Py_None ? nullptr : packed(tensor(a[2], "weights"), "weights", at::kFloat, dev, {p.T, p.k});
        Mat R;
        if (a[3] != Py_None) R = mat_of(a[3], "residual", type, dev, p.T, Ys.cols);
        const CallStream st(a[5], dev);
        const Out Y = out_mat(a[4], "Y", tYs, st, p.T, Ys.cols);
        call([&] {
            return moe_combine(Ys.p, Ys.ld, Ys.rows, p.positions, static_cast<const float*>(w), R.p, R.ld, Y.m.p, Y.m.ld,
                               p.T, p.k, Ys.cols, type_code(type), st);
        });
        return Y.wrap();
    });
}

// moe_combine_backward(dY, Ys, positions, offsets, weights, dYs, dweights, needs, stream)
PyObject* moe_combine_backward_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        const at::Tensor& tdY = tensor(a[0], "dY");
        const at::ScalarType type = element_type(tdY, "dY");
        const int dev = first_device(tdY, "dY");
        const Mat dY = mat(tdY, "dY", type, dev);
        const Places p = places(a[2], a[3], dev);
        if (p.T != dY.rows)
            refuse(PyExc_ValueError, "positions are of %lld tokens, dY has %lld rows", static_cast<long long>(p.T),
                   static_cast<long long>(dY.rows));
        const void* w = packed(tensor(a[4], "weights"), "weights", at::kFloat, dev, {p.T, p.k});
        bool want[2] = {};
        truths(a[7], want, 2);
        Mat Ys;
        if (want[1]) Ys = mat_of(a[1], "Ys", type, dev, p.T * p.k, dY.cols);
        const CallStream st(a[8], dev);
        Out dYs, dw;
        if (want[0]) dYs = out_mat(a[5], "dYs", tdY, st, p.T * p.k, dY.cols);
        if (want[1]) dw = out_packed(a[6], "dweights", at::kFloat, st, {p.T, p.k});
        call([&] {
            return moe_combine_backward(dY.p, dY.ld, Ys.p, Ys.ld, p.positions, p.offsets, as_int(p.experts),
                                        static_cast<const float*>(w), dYs.m.p, dYs.m.ld, static_cast<float*>(dw.m.p), p.T,
                                        p.k, dY.cols, type_code(type), st);
        });
        return Py_BuildValue("NN", wrap_or_none(want[0], dYs), wrap_or_none(want[1], dw));
    });
}

// A 4-bit matrix's data and scales, given as two tensors and its columns.
struct Blocks {
    void *data = nullptr, *scales = nullptr;
    int64_t rows = 0, cols = 0;
};
Blocks blocks(PyObject* data, PyObject* scales, PyObject* columns, const char* data_name, const char* scales_name, int dev) {
    const at::Tensor& d = tensor(data, data_name);
    if (d.dim() != 2) refuse(PyExc_ValueError, "%s must be 2-D", data_name);
    Blocks b;
    b.rows = d.size(0), b.cols = integer(columns);
    if (b.cols < 0 || b.cols > INT32_MAX) refuse(PyExc_ValueError, "columns must be in [0, 2^31)");
    b.data = packed(d, data_name, at::kByte, dev, {b.rows, (b.cols + 31) / 32 * 16});
    b.scales = packed(tensor(scales, scales_name), scales_name, at::kByte, dev,
                      {(b.rows + 127) / 128, (b.cols + 127) / 128, 512});
    return b;
}

// quantize_mxfp4(X, transposed, data, scales, stream) -> (columns, data, scales)
PyObject* quantize_mxfp4_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject* {
        const at::Tensor& tX = tensor(a[0], "X");
        const at::ScalarType type = element_type(tX, "X");
        const int dev = first_device(tX, "X");
        const Mat X = mat(tX, "X", type, dev);
        const bool transposed = truth(a[1]);
        const int64_t rows = transposed ? X.cols : X.rows, cols = transposed ? X.rows : X.cols;
        const CallStream st(a[4], dev);
        const Out data = out_packed(a[2], "data", at::kByte, st, {rows, (cols + 31) / 32 * 16});
        const Out scales = out_packed(a[3], "scales", at::kByte, st, {(rows + 127) / 128, (cols + 127) / 128, 512});
        call([&] {
            return quantize_mxfp4(X.p, X.ld, data.m.p, scales.m.p, rows, cols, transposed ? 1 : 0, type_code(type), st);
        });
        return Py_BuildValue("LNN", static_cast<long long>(cols), data.wrap(), scales.wrap());
    });
}

// dequantize_mxfp4(data, scales, columns, dtype, X, stream)
PyObject* dequantize_mxfp4_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject* {
        const at::Tensor& d = tensor(a[0], "data");
        const int dev = first_device(d, "data");
        const Blocks q = blocks(a[0], a[1], a[2], "data", "scales", dev);
        at::ScalarType type = at::kBFloat16;
        if (a[3] != Py_None) {
            if (!THPDtype_Check(a[3])) refuse(PyExc_TypeError, "dtype must be torch.bfloat16 or torch.float32");
            type = reinterpret_cast<THPDtype*>(a[3])->scalar_type;
            if (type != at::kBFloat16 && type != at::kFloat)
                refuse(PyExc_TypeError, "dtype must be torch.bfloat16 or torch.float32");
        } else if (a[4] != Py_None) {
            type = element_type(tensor(a[4], "X"), "X");
        }
        const CallStream st(a[5], dev);
        Out X;
        if (a[4] != Py_None) {
            X.given = a[4];
            X.m = mat_of(a[4], "X", type, dev, q.rows, q.cols);
        } else {
            X.made = fresh({q.rows, q.cols}, type, st);
            X.m.p = X.made.data_ptr();
            X.m.ld = q.cols > 0 ? q.cols : 1;
        }
        call([&] { return dequantize_mxfp4(q.data, q.scales, X.m.p, X.m.ld, q.rows, q.cols, type_code(type), st); });
        return X.wrap();
    });
}

// gemm_mxfp4(A, A_scales, A_columns, B, B_scales, B_columns, bias, residual, act, C, stream)
PyObject* gemm_mxfp4_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject* {
        const at::Tensor& tA = tensor(a[0], "A");
        const int dev = first_device(tA, "A");
        const Blocks A = blocks(a[0], a[1], a[2], "A", "A's scales", dev), B = blocks(a[3], a[4], a[5], "B", "B's scales", dev);
        if (A.cols != B.cols)
            refuse(PyExc_ValueError, "shape mismatch: A [%lld, %lld], B [%lld, %lld]", static_cast<long long>(A.rows),
                   static_cast<long long>(A.cols), static_cast<long long>(B.rows), static_cast<long long>(B.cols));
        const float* bias = optional_vector(a[6], "bias", dev, B.rows);
        Mat R;
        if (a[7] != Py_None) R = mat_of(a[7], "residual", at::kBFloat16, dev, A.rows, B.rows);
        const int act = act_code(a[8]);
        const CallStream st(a[10], dev);
        Out C;
        if (a[9] != Py_None) {
            C.given = a[9];
            C.m = mat_of(a[9], "C", at::kBFloat16, dev, A.rows, B.rows);
        } else {
            C.made = fresh({A.rows, B.rows}, at::kBFloat16, st);
            C.m.p = C.made.data_ptr();
            C.m.ld = B.rows > 0 ? B.rows : 1;
        }
        call([&] {
            return gemm_mxfp4(A.data, A.scales, B.data, B.scales, bias, R.p, R.ld, C.m.p, C.m.ld, A.rows, B.rows, A.cols,
                              act, st);
        });
        return C.wrap();
    });
}

// set_errors(GbrError, torch.OutOfMemoryError)
PyObject* set_errors_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 2, [&]() -> PyObject* {
        Py_XSETREF(g_error, Py_NewRef(a[0]));
        Py_XSETREF(g_no_memory, Py_NewRef(a[1]));
        Py_RETURN_NONE;
    });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef g_methods[] = {
    {"dropout_add", fast<dropout_add_py>(), METH_FASTCALL, nullptr},
    {"gemm_bias_act", fast<gemm_bias_act_py>(), METH_FASTCALL, nullptr},
    {"gemm_bias_act_backward", fast<gemm_bias_act_backward_py>(), METH_FASTCALL, nullptr},
    {"moe_layer", fast<moe_layer_py>(), METH_FASTCALL, nullptr},
    {"residual_norm", fast<residual_norm_py>(), METH_FASTCALL, nullptr},
    {"residual_norm_backward", fast<residual_norm_backward_py>(), METH_FASTCALL, nullptr},
    {"moe_sort", fast<moe_sort_py>(), METH_FASTCALL, nullptr},
    {"moe_dispatch", fast<moe_dispatch_py>(), METH_FASTCALL, nullptr},
    {"moe_combine", fast<moe_combine_py>(), METH_FASTCALL, nullptr},
    {"moe_combine_backward", fast<moe_combine_backward_py>(), METH_FASTCALL, nullptr},
    {"quantize_mxfp4", fast<quantize_mxfp4_py>(), METH_FASTCALL, nullptr},
    {"dequantize_mxfp4", fast<dequantize_mxfp4_py>(), METH_FASTCALL, nullptr},
    {"gemm_mxfp4", fast<gemm_mxfp4_py>(), METH_FASTCALL, nullptr},
    {"set_errors", fast<set_errors_py>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_operators_ext", nullptr, -1, g_methods, nullptr, nullptr, nullptr,
                        nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__operators_ext() { return PyModule_Create(&g_module); }
