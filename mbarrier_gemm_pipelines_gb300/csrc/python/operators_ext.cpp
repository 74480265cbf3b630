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
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
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

// The call's stream: the current one, or the `stream` argument, which is then the current one until the call
// ends, so that the outputs made here are that stream's to PyTorch's allocator.  From the current stream's share it could
// hand out memory that a kernel there still reads, and give an output away while the other stream writes it.
class CallStream {
public:
    CallStream(PyObject* o, int dev) : handle_(c10::cuda::getCurrentCUDAStream(dev).stream()) {
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

private:
    cudaStream_t handle_;
    c10::cuda::OptionalCUDAStreamGuard guard_;
};

// A tensor of the caller's that the call has written: its version moves, so that autograd refuses a graph that saved
// it before.  (A tensor made in inference mode has none.)
PyObject* written(PyObject* o) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    return Py_NewRef(o);
}

// An output: the caller's, or a new one.
struct Out {
    PyObject* given = nullptr;
    at::Tensor made;
    Mat m;
    PyObject* wrap() const { return given != nullptr ? written(given) : THPVariable_Wrap(made); }
};

Out out_mat(PyObject* o, const char* name, const at::Tensor& like, int dev, int64_t rows, int64_t cols) {
    Out r;
    if (o != Py_None) {
        r.given = o;
        r.m = mat_of(o, name, like.scalar_type(), dev, rows, cols);
    } else {
        r.made = at::empty({rows, cols}, like.options());
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
        if (!has_y) made = at::empty(X.sizes(), X.options());
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
        const Out C = out_mat(a[8], "C", tA, dev, M, N);
        Out Z;
        if (want_z) Z = out_mat(a[9], "Z", tA, dev, M, N);
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
        if (want[0]) dA = out_mat(a[8], "dA", tA, dev, M, K);
        if (want[1]) dB = out_mat(a[9], "dB", tA, dev, K, N);
        if (want[2]) {
            if (a[10] != Py_None) {
                db.given = a[10];
                db.m.p = packed(tensor(a[10], "dbias"), "dbias", at::kFloat, dev, {N});
            } else {
                db.made = at::empty({N}, tdC.options().dtype(at::kFloat));
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
            Y.made = at::empty({T, D}, X.options());
            Y.m.p = Y.made.data_ptr();
        }
        const bool routing = truth(a[10]);
        at::Tensor ids, weights;
        if (routing) {
            const int64_t k = top_k < 0 || top_k > E ? 0 : top_k;       // a wrong top_k is refused by the call
            ids = at::empty({T, k}, X.options().dtype(at::kLong));
            weights = at::empty({T, k}, X.options().dtype(at::kFloat));
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
    {"set_errors", fast<set_errors_py>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_operators_ext", nullptr, -1, g_methods, nullptr, nullptr, nullptr,
                        nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__operators_ext() { return PyModule_Create(&g_module); }
