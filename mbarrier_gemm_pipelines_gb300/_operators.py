"""The feed-forward operators (end of ``include/gbr.h``) for PyTorch tensors.

The functions here give the arguments their names, defaults and documentation;
``csrc/python/operators_ext.cpp`` checks the tensors, makes the outputs and
calls the library.  There is no CPU fallback: a missing build or a CPU tensor
raises.

Outputs have no autograd history: a caller connects the gradients' functions to
its graph.  A tensor that a call writes in place (Y=, C=, Z=, dA=, ...) moves its
version, so that autograd refuses a graph that saved it before.

`stream` is a torch stream or a raw handle; without it a call runs on the
current stream.  With it the outputs that the call makes belong to that stream,
as if made under ``torch.cuda.stream(stream)``: use them there, or after an
event, and ``record_stream`` what another stream goes on using.  Inputs have to
be ready on that stream.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os

from . import _build
from ._binding import GbrError, _cuda_tensor, _outputs_on, _stream_ptr, check, lib

# gbr_act
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

_ext = None


def _load():
    """The compiled binding (it must have been built: ``__graft_entry__.build()``)."""
    global _ext
    if _ext is None:
        import torch                    # its libraries are what the binding is linked to
        lib()
        path = _build.EXT_PATH
        if not os.path.exists(path):
            raise RuntimeError("the Python binding is not built (%s); run __graft_entry__.build()" % path)
        loader = importlib.machinery.ExtensionFileLoader("_operators_ext", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_operators_ext", loader))
        loader.exec_module(module)
        module.set_errors(GbrError, torch.OutOfMemoryError)
        _ext = module
    return _ext


def dropout_add(X, residual=None, p=0.5, seed=0, offset=0, Y=None, stream=None):
    """Y = residual + dropout(X) for bf16 or fp32 tensors; returns Y (which may
    be X or residual itself).  The mask depends on (seed, offset) and the
    position in X seen as [rows, last dimension] alone, so the gradient of X is
    ``dropout_add(dY, p=p, seed=seed, offset=offset)``.  Tensors with more than
    two dimensions must be contiguous."""
    return (_ext or _load()).dropout_add(X, residual, p, seed, offset, Y, stream)


def gemm_bias_act(A, B, bias=None, residual=None, act="none", p=0.0, seed=0, offset=0, C=None, Z=None,
                  return_z=False, stream=None):
    """C = residual + dropout(act(A @ B + bias)) for bf16 matrices (bias fp32);
    returns C, or (C, Z) with the pre-activation Z = A @ B + bias (bf16, what
    gemm_bias_act_backward needs) when return_z is true or Z is given."""
    return (_ext or _load()).gemm_bias_act(A, B, bias, residual, act, p, seed, offset, C, Z, return_z, stream)


def gemm_bias_act_backward(dC, A, B, Z=None, act="none", p=0.0, seed=0, offset=0, dA=None, dB=None,
                           dbias=None, needs=(True, True, True), stream=None):
    """Gradients (dA, dB, dbias) of gemm_bias_act for dC, with the Z, p, seed and
    offset of the forward call; the residual's gradient is dC itself.  `needs`
    says which of the three are wanted (None is returned for the others)."""
    return (_ext or _load()).gemm_bias_act_backward(dC, A, B, Z, act, p, seed, offset, dA, dB, dbias, needs, stream)


def moe_layer(X, Wr, W1, b1, W2, b2, top_k=2, act="relu", gated=False, Y=None, return_routing=False,
              stream=None):
    """A whole mixture-of-experts layer for up to 64 tokens: router (X @ Wr, the
    top_k largest, softmax over them), the chosen experts' two products and
    their weighted sum.  X [T, D], W1 [E, D, F] (gated: [E, D, 2F], gate columns
    first), W2 [E, F, D] bf16; Wr [D, E], b1 [E, F or 2F], b2 [E, D] fp32 (b1
    and b2 may be None).  Returns Y [T, D] bf16, or (Y, expert_ids int64
    [T, top_k], expert_weights fp32 [T, top_k])."""
    return (_ext or _load()).moe_layer(X, Wr, W1, b1, W2, b2, top_k, act, gated, Y, return_routing, stream)


def selftest_linear_skip_load(A, B, cta, item, limit_ns, stream=None):
    """Runs gemm_bias_act (A @ B alone) with one stage of CTA (or CTA pair) `cta`,
    ring item `item`, left unfilled (see gbr.h); returns the undefined output."""
    with _outputs_on(stream):
        C = A.new_empty(A.shape[0], B.shape[1])
    check(lib().gbr_selftest_linear_skip_load(
        *(_cuda_tensor(t, n, (C.dtype,)).data_ptr() for t, n in ((A, "A"), (B, "B"), (C, "C"))), A.shape[0],
        B.shape[1], A.shape[1], cta, item, limit_ns, _stream_ptr(stream)))
    return C


def selftest_moe_skip_load(X, Wr, W1, W2, top_k, cta, item, limit_ns, stream=None):
    """Runs moe_layer (ReLU, no biases) with one stage of CTA `cta`, ring item
    `item`, left unfilled (see gbr.h); returns the undefined output."""
    with _outputs_on(stream):
        Y = X.new_empty(X.shape)
    E, F = W2.shape[:2]
    for t, n in ((X, "X"), (Wr, "Wr"), (W1, "W1"), (W2, "W2")):
        _cuda_tensor(t, n, (Wr.dtype if n == "Wr" else X.dtype,))
    check(lib().gbr_selftest_moe_skip_load(X.data_ptr(), Wr.data_ptr(), W1.data_ptr(), W2.data_ptr(), Y.data_ptr(),
                                           X.shape[0], X.shape[1], F, E, top_k, cta, item, limit_ns,
                                           _stream_ptr(stream)))
    return Y
