"""Python binding of the feed-forward operators (end of ``include/gbr.h``).

Argument marshalling only, kept short: a call for one token takes the GPU a few
microseconds, so the checks here read each tensor's type, shape, strides and
device once.  There is no CPU fallback.
"""
from __future__ import annotations

import torch

from ._binding import BF16, F32_FFMA, GbrError, last_error, lib

# gbr_act
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

_bf16, _f32 = torch.bfloat16, torch.float32
_empty = torch.empty
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


_LIMIT = 1 << 64


def _check(code):
    if code:
        raise GbrError(code, last_error())


def _act_code(act):
    code = ACTS.get(act)
    if code is None:
        raise ValueError("act must be one of %s, got %r" % (", ".join(ACTS), act))
    return code


def _check_bits(seed, offset):
    for v, name in ((seed, "seed"), (offset, "offset")):
        if not isinstance(v, int) or not 0 <= v < _LIMIT:
            raise ValueError("%s must be an integer in [0, 2^64)" % name)


def _refuse(t, name, dtype, dev, rows=None, cols=None):
    """Says what is wrong with a tensor that the short checks below turned down."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.get_device() < 0:
        raise ValueError("%s must be a CUDA tensor (this library has no CPU path)" % name)
    if t.get_device() != dev:
        raise ValueError("%s is on cuda:%d, not on cuda:%d" % (name, t.get_device(), dev))
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    if rows is not None and tuple(t.shape) != (rows, cols):
        raise ValueError("%s must be [%d, %d], got %s" % (name, rows, cols, list(t.shape)))
    raise ValueError("the rows of %s must be contiguous" % name)


def _device_of(t, name):
    """The current device, on which the first tensor has to be."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s must be a CUDA tensor (this library has no CPU path)" % name)
    if dev != _current_device():
        raise ValueError("%s is on cuda:%d, the current device is cuda:%d" % (name, dev, _current_device()))
    return dev


def _step(t, rows, cols):
    """Row stride of a 2-D tensor that is not contiguous; -1 where its rows are not either."""
    step, inner = t.stride()
    if inner != 1 and cols > 1:
        return -1
    return step if rows > 1 else cols or 1


def _mat(t, name, dtype, dev):
    """(rows, columns, row stride) of a 2-D tensor on `dev` whose rows are contiguous."""
    if getattr(t, "dtype", None) is not dtype or t.get_device() != dev or t.dim() != 2:
        _refuse(t, name, dtype, dev)
    rows, cols = t.shape
    step = (cols or 1) if t.is_contiguous() else _step(t, rows, cols)
    if step < 0:
        _refuse(t, name, dtype, dev)
    return rows, cols, step


def _mat_of(t, name, dtype, dev, rows, cols):
    """Row stride of a [rows, cols] matrix."""
    if getattr(t, "dtype", None) is not dtype or t.get_device() != dev or t.shape != (rows, cols):
        _refuse(t, name, dtype, dev, rows, cols)
    step = (cols or 1) if t.is_contiguous() else _step(t, rows, cols)
    if step < 0:
        _refuse(t, name, dtype, dev, rows, cols)
    return step


def _packed(t, name, dtype, dev, shape):
    """Data pointer of a contiguous tensor of that shape."""
    if getattr(t, "dtype", None) is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.get_device() != dev:
        raise ValueError("%s is on %s, not on cuda:%d" % (name, t.device, dev))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    raise ValueError("%s must be contiguous" % name)


def _stream_of(stream, dev):
    if stream is None:
        return _raw_stream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def dropout_add(X, residual=None, p=0.5, seed=0, offset=0, Y=None, stream=None):
    """Y = residual + dropout(X) for bf16 or fp32 tensors; returns Y (which may
    be X or residual itself).  The mask depends on (seed, offset) and the
    position in X seen as [rows, last dimension] alone, so the gradient of X is
    ``dropout_add(dY, p=p, seed=seed, offset=offset)``.  Tensors with more than
    two dimensions must be contiguous."""
    dtype = getattr(X, "dtype", None)
    if dtype is not _bf16 and dtype is not _f32:
        raise TypeError("X must be a bf16 or fp32 torch.Tensor, got %s" % (dtype or type(X)))
    dev = _device_of(X, "X")
    if Y is None:
        Y = _empty(X.shape, dtype=dtype, device=X.device)
    x, r, y = X, residual, Y
    if X.dim() != 2:
        shape = X.shape
        if not shape:
            raise ValueError("X must have at least one dimension")
        flat = (shape[:-1].numel(), shape[-1])
        for t, name in ((x, "X"), (r, "residual"), (y, "Y")):
            if t is not None:
                _packed(t, name, dtype, dev, shape)
        x, y, r = x.view(flat), y.view(flat), None if r is None else r.view(flat)
    rows, cols, ldx = _mat(x, "X", dtype, dev)
    ldy = _mat_of(y, "Y", dtype, dev, rows, cols)
    pr, ldr = (None, 0) if r is None else (r.data_ptr(), _mat_of(r, "residual", dtype, dev, rows, cols))
    if seed or offset:
        _check_bits(seed, offset)
    _check(lib().dropout_add(x.data_ptr(), ldx, pr, ldr, y.data_ptr(), ldy, rows, cols,
                             BF16 if dtype is _bf16 else F32_FFMA, p, seed, offset,
                             _raw_stream(dev) if stream is None else _stream_of(stream, dev)))
    return Y


def gemm_bias_act(A, B, bias=None, residual=None, act="none", p=0.0, seed=0, offset=0, C=None, Z=None,
                  return_z=False, stream=None):
    """C = residual + dropout(act(A @ B + bias)) for bf16 matrices (bias fp32);
    returns C, or (C, Z) with the pre-activation Z = A @ B + bias (bf16, what
    gemm_bias_act_backward needs) when return_z is true or Z is given."""
    dev = _device_of(A, "A")
    M, K, lda = _mat(A, "A", _bf16, dev)
    K2, N, ldb = _mat(B, "B", _bf16, dev)
    if K2 != K:
        raise ValueError("shape mismatch: A %s, B %s" % (list(A.shape), list(B.shape)))
    pb = pr = pz = None
    ldr = ldz = 0
    if bias is not None:
        pb = _packed(bias, "bias", _f32, dev, (N,))
    if residual is not None:
        pr, ldr = residual.data_ptr(), _mat_of(residual, "residual", _bf16, dev, M, N)
    if C is None:
        C = _empty((M, N), dtype=_bf16, device=A.device)
        ldc = N or 1
    else:
        ldc = _mat_of(C, "C", _bf16, dev, M, N)
    if Z is not None:
        pz, ldz = Z.data_ptr(), _mat_of(Z, "Z", _bf16, dev, M, N)
    elif return_z:
        Z = _empty((M, N), dtype=_bf16, device=A.device)
        pz, ldz = Z.data_ptr(), N or 1
    if seed or offset:
        _check_bits(seed, offset)
    _check(lib().gemm_bias_act(A.data_ptr(), lda, B.data_ptr(), ldb, pb, pr, ldr, C.data_ptr(), ldc, pz, ldz,
                               M, N, K, BF16, _act_code(act), p, seed, offset,
                               _raw_stream(dev) if stream is None else _stream_of(stream, dev)))
    return C if Z is None else (C, Z)


def gemm_bias_act_backward(dC, A, B, Z=None, act="none", p=0.0, seed=0, offset=0, dA=None, dB=None,
                           dbias=None, needs=(True, True, True), stream=None):
    """Gradients (dA, dB, dbias) of gemm_bias_act for dC, with the Z, p, seed and
    offset of the forward call; the residual's gradient is dC itself.  `needs`
    says which of the three are wanted (None is returned for the others)."""
    code = _act_code(act)
    dev = _device_of(dC, "dC")
    M, K, lda = _mat(A, "A", _bf16, dev)
    K2, N, ldb = _mat(B, "B", _bf16, dev)
    if K2 != K:
        raise ValueError("shape mismatch: A %s, B %s" % (list(A.shape), list(B.shape)))
    lddc = _mat_of(dC, "dC", _bf16, dev, M, N)
    if code != 0 and Z is None:
        raise ValueError("Z (the pre-activation of the forward call) is needed for act=%r" % act)
    pz, ldz = (None, 0) if Z is None else (Z.data_ptr(), _mat_of(Z, "Z", _bf16, dev, M, N))
    want_a, want_b, want_bias = needs
    pa = pb = pbias = None
    ldda = lddb = 0
    if not want_a:
        dA = None
    elif dA is None:
        dA = _empty((M, K), dtype=_bf16, device=dC.device)
        pa, ldda = dA.data_ptr(), K or 1
    else:
        pa, ldda = dA.data_ptr(), _mat_of(dA, "dA", _bf16, dev, M, K)
    if not want_b:
        dB = None
    elif dB is None:
        dB = _empty((K, N), dtype=_bf16, device=dC.device)
        pb, lddb = dB.data_ptr(), N or 1
    else:
        pb, lddb = dB.data_ptr(), _mat_of(dB, "dB", _bf16, dev, K, N)
    if not want_bias:
        dbias = None
    else:
        if dbias is None:
            dbias = _empty((N,), dtype=_f32, device=dC.device)
        pbias = _packed(dbias, "dbias", _f32, dev, (N,))
    if seed or offset:
        _check_bits(seed, offset)
    _check(lib().gemm_bias_act_backward(dC.data_ptr(), lddc, A.data_ptr(), lda, B.data_ptr(), ldb, pz, ldz, pa,
                                        ldda, pb, lddb, pbias, M, N, K, BF16, code, p, seed, offset,
                                        _raw_stream(dev) if stream is None else _stream_of(stream, dev)))
    return dA, dB, dbias


def moe_layer(X, Wr, W1, b1, W2, b2, top_k=2, act="relu", gated=False, Y=None, return_routing=False,
              stream=None):
    """A whole mixture-of-experts layer for up to 64 tokens: router (X @ Wr, the
    top_k largest, softmax over them), the chosen experts' two products and
    their weighted sum.  X [T, D], W1 [E, D, F] (gated: [E, D, 2F], gate columns
    first), W2 [E, F, D] bf16; Wr [D, E], b1 [E, F or 2F], b2 [E, D] fp32 (b1
    and b2 may be None).  Returns Y [T, D] bf16, or (Y, expert_ids int64
    [T, top_k], expert_weights fp32 [T, top_k])."""
    dev = _device_of(X, "X")
    if len(X.shape) != 2 or len(W2.shape) != 3:
        raise ValueError("X must be 2-D, W1 and W2 3-D")
    T, D = X.shape
    E, F = W2.shape[:2]
    F1 = 2 * F if gated else F
    px = _packed(X, "X", _bf16, dev, (T, D))
    pr = _packed(Wr, "Wr", _f32, dev, (D, E))
    p1 = _packed(W1, "W1", _bf16, dev, (E, D, F1))
    p2 = _packed(W2, "W2", _bf16, dev, (E, F, D))
    pb1 = None if b1 is None else _packed(b1, "b1", _f32, dev, (E, F1))
    pb2 = None if b2 is None else _packed(b2, "b2", _f32, dev, (E, D))
    if Y is None:
        Y = _empty((T, D), dtype=_bf16, device=X.device)
    py = _packed(Y, "Y", _bf16, dev, (T, D))
    ids = weights = pi = pw = None
    if return_routing:
        ids = _empty((T, top_k), dtype=torch.int64, device=X.device)
        weights = _empty((T, top_k), dtype=_f32, device=X.device)
        pi, pw = ids.data_ptr(), weights.data_ptr()
    _check(lib().moe_layer(px, pr, p1, pb1, p2, pb2, py, pi, pw, T, D, F, E, top_k, _act_code(act),
                           1 if gated else 0, BF16, _stream_of(stream, dev)))
    return (Y, ids, weights) if return_routing else Y


def selftest_linear_skip_load(A, B, cta, item, limit_ns, stream=None):
    """Runs gemm_bias_act (A @ B alone) with one stage of CTA (or CTA pair) `cta`,
    ring item `item`, left unfilled (see gbr.h); returns the undefined output."""
    dev = _device_of(A, "A")
    M, K, N = A.shape[0], A.shape[1], B.shape[1]
    C = _empty((M, N), dtype=_bf16, device=A.device)
    _check(lib().gbr_selftest_linear_skip_load(_packed(A, "A", _bf16, dev, (M, K)), _packed(B, "B", _bf16, dev, (K, N)),
                                               C.data_ptr(), M, N, K, cta, item, limit_ns, _stream_of(stream, dev)))
    return C


def selftest_moe_skip_load(X, Wr, W1, W2, top_k, cta, item, limit_ns, stream=None):
    """Runs moe_layer (ReLU, no biases) with one stage of CTA `cta`, ring item
    `item`, left unfilled (see gbr.h); returns the undefined output."""
    dev = _device_of(X, "X")
    T, D = X.shape
    E, F = W2.shape[:2]
    Y = _empty((T, D), dtype=_bf16, device=X.device)
    _check(lib().gbr_selftest_moe_skip_load(_packed(X, "X", _bf16, dev, (T, D)), _packed(Wr, "Wr", _f32, dev, (D, E)),
                                            _packed(W1, "W1", _bf16, dev, (E, D, F)),
                                            _packed(W2, "W2", _bf16, dev, (E, F, D)), Y.data_ptr(), T, D, F, E,
                                            top_k, cta, item, limit_ns, _stream_of(stream, dev)))
    return Y
