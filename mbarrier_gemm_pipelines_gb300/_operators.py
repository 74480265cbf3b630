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
from typing import NamedTuple

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


def residual_norm(X, R=None, post=None, gate=None, scale=1.0, pre=None, eps=1e-6, S=None, H=None, stream=None):
    """What stands between two blocks: S = R + scale * gate * norm(X) * post and
    H = norm(S) * pre, norm dividing each row by sqrt(mean square + eps).
    X (the block's output), R (the residual stream; None: zero) [rows, cols] bf16
    or fp32; post, pre [cols] fp32 and gate [gates, cols] of X's type may be None.
    gate row i * gates // rows goes with row i: one row is a gate per channel,
    as many as X has one per element.  Returns (S, H), H None without pre; S is X
    itself where nothing is added, scaled or normalised (a model's first norm)."""
    return (_ext or _load()).residual_norm(X, R, post, gate, scale, pre, eps, S, H, stream)


def residual_norm_backward(dS, dH, X, S, post=None, gate=None, scale=1.0, pre=None, eps=1e-6, dX=None, dR=None,
                           dpost=None, dgate=None, dpre=None, needs=(True, True, True, True, True), stream=None):
    """Gradients (dX, dR, dpost, dgate, dpre) of residual_norm for dS and dH, with the
    X, post, gate, scale, pre and eps of the forward call and the S it returned.  dS may be
    None with pre (zero), dH and S without it, X without post and gate.  `needs`
    says which are wanted; None is returned for the others and for what the forward call did without."""
    return (_ext or _load()).residual_norm_backward(dS, dH, X, S, post, gate, scale, pre, eps, dX, dR, dpost, dgate,
                                                    dpre, needs, stream)


def moe_sort(expert_ids, num_experts, positions=None, offsets=None, stream=None):
    """Where each choice's row goes when rows are sorted by expert: expert_ids int64
    [T, top_k] -> (positions int32 [T, top_k], offsets int32 [num_experts + 1]).
    Choices of an expert keep their order; an id outside [0, num_experts) is
    struck out (position -1).  Expert e has rows offsets[e] .. offsets[e + 1] - 1."""
    return (_ext or _load()).moe_sort(expert_ids, num_experts, positions, offsets, stream)


def moe_dispatch(X, positions, offsets, Xs=None, stream=None):
    """Rows in the experts' order: Xs[positions[t, j]] = X[t]; rows of Xs [T * top_k, D] from
    offsets[-1] on are zero.  X [T, D] bf16 or fp32.  The gradient of X is
    ``moe_combine(dXs, positions)``."""
    return (_ext or _load()).moe_dispatch(X, positions, offsets, Xs, stream)


def moe_combine(Ys, positions, weights=None, residual=None, Y=None, stream=None):
    """Back to the tokens: Y[t] = residual[t] + sum over j of weights[t, j] *
    Ys[positions[t, j]]; struck-out choices count nothing.  Ys [rows, D] bf16 or
    fp32, weights fp32 [T, top_k] (None: one), residual [T, D] (None: zero)."""
    return (_ext or _load()).moe_combine(Ys, positions, weights, residual, Y, stream)


def moe_combine_backward(dY, Ys, positions, offsets, weights, dYs=None, dweights=None, needs=(True, True), stream=None):
    """Gradients (dYs, dweights) of moe_combine for dY: dYs[positions[t, j]] =
    weights[t, j] * dY[t] (zero from offsets[-1] on), dweights[t, j] = <dY[t],
    Ys[positions[t, j]]> in fp32, 0 for struck-out choices.  The residual's gradient is
    dY itself.  `needs` says which are wanted (Ys may be None without dweights)."""
    return (_ext or _load()).moe_combine_backward(dY, Ys, positions, offsets, weights, dYs, dweights, needs, stream)


class Mxfp4(NamedTuple):
    """A matrix in microscaled 4-bit floating point: blocks of 32 values along
    the columns (layout: gbr.h)."""
    data: "torch.Tensor"            # uint8 [rows, 16 * ceil(columns / 32)]
    scales: "torch.Tensor"          # uint8 [ceil(rows / 128), ceil(columns / 128), 512]
    columns: int


def quantize_mxfp4(X, transposed=False, out=None, stream=None):
    """X [rows, columns] (bf16 or fp32) in 4 bits: each block's scale is
    2^(floor(log2 of its largest size) - 2), its values are rounded to the nearest of
    0, 0.5, 1, 1.5, 2, 3, 4, 6 times that.  With `transposed` X is [columns, rows]:
    weights stored [K, N] give what gemm_mxfp4 takes as B.  `out`: an Mxfp4 to write."""
    data, scales = (None, None) if out is None else (out.data, out.scales)
    columns, data, scales = (_ext or _load()).quantize_mxfp4(X, transposed, data, scales, stream)
    return Mxfp4(data, scales, columns) if out is None or out.columns != columns else out


def dequantize_mxfp4(Q, dtype=None, X=None, stream=None):
    """The values of an Mxfp4, as `dtype` (torch.bfloat16 unless given; or torch.float32)."""
    return (_ext or _load()).dequantize_mxfp4(Q.data, Q.scales, Q.columns, dtype, X, stream)


def gemm_mxfp4(A, B, bias=None, residual=None, act="none", C=None, stream=None):
    """C = residual + act(A @ B.T + bias) of two Mxfp4, A [M, K] and B [N, K]; C and
    residual [M, N] bf16, bias [N] fp32."""
    return (_ext or _load()).gemm_mxfp4(A.data, A.scales, A.columns, B.data, B.scales, B.columns, bias, residual, act, C,
                                        stream)


def _shaped(t, name, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, list(shape), list(t.shape)))


def selftest_mxfp4_skip_load(A, B, cta, item, limit_ns, stream=None):
    """Runs gemm_mxfp4 (A @ B.T alone) with one stage left unfilled, as
    selftest_linear_skip_load; returns the undefined output."""
    import torch
    for Q, n in ((A, "A"), (B, "B")):
        rows = Q.data.shape[0]
        _shaped(Q.data, n, (rows, (A.columns + 31) // 32 * 16))
        _shaped(Q.scales, n + "'s scales", ((rows + 127) // 128, (A.columns + 127) // 128, 512))
    with _outputs_on(stream):
        C = torch.empty((A.data.shape[0], B.data.shape[0]), dtype=torch.bfloat16, device=A.data.device)
    tensors = [_cuda_tensor(t, "operand", (torch.uint8,)) for t in (A.data, A.scales, B.data, B.scales)]
    check(lib().gbr_selftest_mxfp4_skip_load(*(t.data_ptr() for t in tensors), C.data_ptr(), C.shape[0], C.shape[1],
                                             A.columns, cta, item, limit_ns, _stream_ptr(stream)))
    return C


def selftest_linear_skip_load(A, B, cta, item, limit_ns, stream=None):
    """Runs gemm_bias_act (A @ B alone) with one stage of CTA (or CTA pair) `cta`,
    ring item `item`, left unfilled (see gbr.h); returns the undefined output."""
    _shaped(B, "B", (A.shape[1], B.shape[1]))
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
    (T, D), (E, F) = X.shape, W2.shape[:2]
    for t, n, shape in ((Wr, "Wr", (D, E)), (W1, "W1", (E, D, F)), (W2, "W2", (E, F, D))):
        _shaped(t, n, shape)
    for t, n in ((X, "X"), (Wr, "Wr"), (W1, "W1"), (W2, "W2")):
        _cuda_tensor(t, n, (Wr.dtype if n == "Wr" else X.dtype,))
    check(lib().gbr_selftest_moe_skip_load(X.data_ptr(), Wr.data_ptr(), W1.data_ptr(), W2.data_ptr(), Y.data_ptr(),
                                           T, D, F, E, top_k, cta, item, limit_ns,
                                           _stream_ptr(stream)))
    return Y
