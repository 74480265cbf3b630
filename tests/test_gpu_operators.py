"""The feed-forward operators on the GPU against their definitions in 64 bits.

Bars (bf16 keeps 8 significant bits, so a correctly rounded value is off by at
most 2^-8 of itself, and by about 2^-8 / sqrt(3) times 0.7 = 1.6e-3 of it in the
mean square over values of all sizes; U = 2^-9 = 1.95e-3 is that with a margin)
  one rounding (C, Z)                    1.0625 U in relative Frobenius norm;
      fp32 accumulation and the fp32 activations are far below the margin
  dropout, bf16                          2^-8 |y| elementwise, and what fp32 adds
  an operand rounded as well (dA, dB from dZ, Y of the experts from h): the
      operand's roundings are independent and add another U     -> 2.25 U
  dbias (fp32)   (2^-19 + M 2^-24) sum |drop(dC)|, elementwise
  dropout, fp32  three roundings: 2^-22 (|x| scale + |r|), elementwise
"""
import math
import sys

import pytest
import torch

import ffn_reference as ref
from gpu_helpers import load_library, require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -9
ONE, TWO = 1.0625 * U, 2.25 * U
BF = torch.bfloat16


@pytest.fixture(scope="module")
def gbr():
    require_gpu()
    return load_library()


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, std=1.0, dtype=BF):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def rel(got, want):
    got, n = got.double(), want.norm().item()
    e = (got - want).norm().item()
    return e / n if n > 0 else e


def close(got, want, bar):
    assert got.shape == want.shape
    assert rel(got, want) <= bar
    if want.numel():
        assert (got.double() - want).abs().max().item() <= 16 * bar * max(want.abs().max().item(), 1e-30)


def padded(t, left=3, right=5):
    """The same values as a view with odd strides and an odd start."""
    big = torch.full((t.shape[0], t.shape[1] + left + right), float("nan"), device=t.device, dtype=t.dtype)
    big[:, left:left + t.shape[1]] = t
    return big[:, left:left + t.shape[1]]


def spaced(t, pad=24):
    """The same values with a wider row pitch that is a multiple of 16 bytes."""
    big = torch.full((t.shape[0], (t.shape[1] + 7) // 8 * 8 + pad), float("nan"), device=t.device, dtype=t.dtype)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


LINEAR = [
    # M, K, N, act, p, bias, residual, z
    (1, 1, 1, "none", 0.0, True, True, True),
    (1, 4096, 4096, "none", 0.0, True, True, False),
    (1, 64, 50000, "relu", 0.0, True, False, False),
    (2, 7, 9, "gelu", 0.5, True, True, True),
    (3, 0, 40, "silu", 0.1, True, True, True),
    (5, 520, 24, "relu", 0.0, False, False, False),
    (16, 2048, 264, "silu", 0.1, True, True, True),
    (17, 1000, 1000, "gelu_tanh", 0.0, True, False, True),
    (33, 130, 4095, "gelu", 0.1, True, True, False),
    (63, 4096, 136, "none", 0.25, False, True, False),
    (64, 512, 512, "relu", 0.0, True, False, False),
    (65, 512, 512, "relu", 0.0, True, False, False),
    (100, 72, 136, "silu", 0.5, True, True, True),
    (128, 1024, 1024, "gelu", 0.0, True, False, True),
    (129, 4096, 520, "gelu", 0.1, True, True, False),
    (256, 2048, 2048, "none", 0.1, True, True, False),
    (257, 65, 255, "silu", 0.0, True, True, True),
    (301, 520, 1000, "gelu", 0.1, True, True, True),
    (512, 100, 96, "none", 0.0, False, False, False),
    (777, 1023, 1025, "gelu_tanh", 0.5, True, True, True),
    (1024, 256, 3000, "relu", 0.0, True, True, True),
    (2500, 1032, 776, "silu", 0.1, True, True, True),
    (4096, 64, 4096, "gelu", 0.1, True, True, True),
    (70001, 24, 40, "none", 0.1, True, True, False),
    (2048, 4096, 2048, "gelu", 0.0, True, False, True),
]


@pytest.mark.parametrize("M,K,N,act,p,bias,residual,z", LINEAR)
def test_linear(gbr, M, K, N, act, p, bias, residual, z):
    g = rng(M * 7 + K * 3 + N)
    A, B = normal(g, (M, K)), normal(g, (K, N), 1 / math.sqrt(max(K, 1)))
    b = normal(g, (N,), 0.3, torch.float32) if bias else None
    R = normal(g, (M, N)) if residual else None
    seed, off = 0xABCDEF0123456789 + M, (3 << 32) + N
    out = gbr.gemm_bias_act(A, B, b, residual=R, act=act, p=p, seed=seed, offset=off, return_z=z)
    gbr.check_device()
    C, Z = ref.linear(A, B, b, R, act, p, seed, off)
    if z:
        close(out[1], Z, ONE)
        out = out[0]
    close(out, C, ONE)


@pytest.mark.parametrize("M,K,N,act,p", sorted({(c[0], c[1], c[2], c[3], c[4]) for c in LINEAR}))
def test_linear_grad(gbr, M, K, N, act, p):
    g = rng(M + K * 5 + N * 11)
    A, B = normal(g, (M, K)), normal(g, (K, N), 1 / math.sqrt(max(K, 1)))
    Z = normal(g, (M, N)) if act != "none" else None
    dC = normal(g, (M, N))
    seed, off = 0x123456789ABCDEF0 + N, (1 << 40) + M
    dA, dB, db = gbr.gemm_bias_act_backward(dC, A, B, Z, act=act, p=p, seed=seed, offset=off)
    gbr.check_device()
    rA, rB, rb, _ = ref.linear_grad(dC, A, B, Z, act, p, seed, off)
    close(dA, rA, TWO)
    close(dB, rB, TWO)
    bound = (2.0 ** -19 + M * 2.0 ** -24) * ref.drop(dC.double(), p, seed, off).abs().sum(0)
    assert ((db.double() - rb).abs() <= bound + 1e-30).all()


@pytest.mark.parametrize("lay", [padded, spaced])
@pytest.mark.parametrize("M,K,N", [(5, 48, 72), (65, 129, 201), (300, 264, 520)])
def test_strides(gbr, lay, M, K, N):
    """Every operand and output as a view of a wider matrix; nothing outside the views is written."""
    g = rng(M)
    A, B, R = normal(g, (M, K)), normal(g, (K, N), 1 / math.sqrt(K)), normal(g, (M, N))
    b = normal(g, (N,), 0.3, torch.float32)
    C, Z = lay(torch.zeros(M, N, device="cuda", dtype=BF)), lay(torch.zeros(M, N, device="cuda", dtype=BF))
    kw = dict(act="gelu", p=0.25, seed=5, offset=6)
    gbr.gemm_bias_act(lay(A), lay(B), b, residual=lay(R), C=C, Z=Z, **kw)
    rc, rz = ref.linear(A, B, b, R, "gelu", 0.25, 5, 6)
    close(C, rc, ONE)
    close(Z, rz, ONE)
    assert C._base.isnan().sum() == C._base.numel() - C.numel()
    assert Z._base.isnan().sum() == Z._base.numel() - Z.numel()
    dC, Zs = normal(g, (M, N)), normal(g, (M, N))
    dA, dB = lay(torch.zeros(M, K, device="cuda", dtype=BF)), lay(torch.zeros(K, N, device="cuda", dtype=BF))
    gbr.gemm_bias_act_backward(lay(dC), lay(A), lay(B), lay(Zs), dA=dA, dB=dB, **kw)
    gbr.check_device()
    rA, rB, _, _ = ref.linear_grad(dC, A, B, Zs, "gelu", 0.25, 5, 6)
    close(dA, rA, TWO)
    close(dB, rB, TWO)
    assert dA._base.isnan().sum() == dA._base.numel() - dA.numel()
    assert dB._base.isnan().sum() == dB._base.numel() - dB.numel()
    X, Y = normal(g, (M, N)), lay(torch.zeros(M, N, device="cuda", dtype=BF))
    gbr.dropout_add(lay(X), lay(R), p=0.25, seed=1, offset=2, Y=Y)
    close(Y, ref.drop(X.double(), 0.25, 1, 2) + R.double(), ONE)
    assert Y._base.isnan().sum() == Y._base.numel() - Y.numel()


@pytest.mark.parametrize("M,K,N", [(3, 64, 128), (90, 200, 304), (300, 520, 1000)])
def test_in_place_residual(gbr, M, K, N):
    g = rng(N)
    A, B, R = normal(g, (M, K)), normal(g, (K, N), 1 / math.sqrt(K)), normal(g, (M, N))
    want = gbr.gemm_bias_act(A, B, residual=R, p=0.1, seed=3)
    got = R.clone()
    assert gbr.gemm_bias_act(A, B, residual=got, p=0.1, seed=3, C=got) is got
    assert torch.equal(got, want)
    X = R.clone()
    gbr.dropout_add(X, X, p=0.5, seed=9, Y=X)
    assert torch.equal(X, gbr.dropout_add(R, R, p=0.5, seed=9))


@pytest.mark.parametrize("M,K,N", [(4, 256, 256), (100, 256, 300), (600, 256, 520)])
def test_masked_and_infinite_values(gbr, M, K, N):
    """A row of NaN stays in its row; a dropped NaN or Inf is an exact zero; p = 1 drops all."""
    g = rng(M + 1)
    A, B = normal(g, (M, K)), normal(g, (K, N), 1 / math.sqrt(K))
    A[M // 2] = float("nan")
    for act in ("none", "relu", "gelu", "gelu_tanh", "silu"):
        C = gbr.gemm_bias_act(A, B, act=act, p=0.5, seed=1)
        keep = ref.keep_mask(M, N, 0.5, 1, 0, "cuda")[0]
        bad = C.isnan()
        assert torch.equal(bad[M // 2], keep[M // 2])
        bad[M // 2] = False
        assert not bad.any()
        assert (C[~keep] == 0).all()
    R = normal(g, (M, N))
    assert torch.equal(gbr.gemm_bias_act(A, B, residual=R, p=1.0), R)
    # Infinite pre-activations take the activations' limits.
    bias = torch.zeros(N, device="cuda")
    bias[0], bias[1] = float("inf"), float("-inf")
    A[M // 2] = 0
    for act, low in (("relu", 0.0), ("gelu", 0.0), ("gelu_tanh", 0.0), ("silu", 0.0), ("none", float("-inf"))):
        C, Z = gbr.gemm_bias_act(A, B, bias, act=act, return_z=True)
        assert (C[:, 0] == float("inf")).all() and (C[:, 1] == low).all()
        assert torch.isfinite(C[:, 2:]).all()
        dC = torch.ones(M, N, device="cuda", dtype=BF)
        db = gbr.gemm_bias_act_backward(dC, A, B, Z, act=act, needs=(False, False, True))[2]
        assert db[0] == M and db[1] == (M if act == "none" else 0)
    # Gradients: a dropped NaN contributes nothing.
    dC = normal(g, (M, N))
    keep = ref.keep_mask(M, N, 0.5, 2, 0, "cuda")[0]
    clean = gbr.gemm_bias_act_backward(dC, A, B, p=0.5, seed=2)
    dC[~keep] = float("nan")
    for x, y in zip(gbr.gemm_bias_act_backward(dC, A, B, p=0.5, seed=2), clean):
        assert torch.equal(x, y)
    gbr.check_device()


def test_partial_gradients(gbr):
    g = rng(4)
    M, K, N = 150, 96, 200
    A, B, Z, dC = normal(g, (M, K)), normal(g, (K, N)), normal(g, (M, N)), normal(g, (M, N))
    full = gbr.gemm_bias_act_backward(dC, A, B, Z, act="silu", p=0.1)
    for i in range(3):
        needs = tuple(j == i for j in range(3))
        part = gbr.gemm_bias_act_backward(dC, A, B, Z, act="silu", p=0.1, needs=needs)
        assert torch.equal(part[i], full[i])
        assert all(part[j] is None for j in range(3) if j != i)


@pytest.mark.parametrize("M,K,N", [(0, 16, 24), (16, 0, 24), (16, 24, 0)])
def test_empty_sizes(gbr, M, K, N):
    A, B = (torch.ones(s, device="cuda", dtype=BF) for s in ((M, K), (K, N)))
    dC = torch.ones(M, N, device="cuda", dtype=BF)
    outs = [torch.full(s, 7.0, device="cuda", dtype=d) for s, d in (((M, K), BF), ((K, N), BF), ((N,), torch.float32))]
    gbr.gemm_bias_act_backward(dC, A, B, dA=outs[0], dB=outs[1], dbias=outs[2])
    gbr.check_device()
    for got, want in zip(outs, ref.linear_grad(dC, A, B, None, "none")):
        assert torch.equal(got.double(), want)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "none"])
def test_gradient_against_differences(gbr, act):
    """The change of <C, dC> along each gradient, by central differences of the definition in 64 bits."""
    g = rng(8)
    M, K, N = 70, 88, 120
    A, B, b = normal(g, (M, K)), normal(g, (K, N), 1 / math.sqrt(K)), normal(g, (N,), 0.3, torch.float32)
    dC = normal(g, (M, N))
    kw = dict(act=act, p=0.2, seed=77, offset=1)
    _, Z = gbr.gemm_bias_act(A, B, b, return_z=True, **kw)
    grads = gbr.gemm_bias_act_backward(dC, A, B, Z, **kw)

    def loss(A, B, b):
        return (ref.linear(A, B, b, None, act, 0.2, 77, 1)[0] * dC.double()).sum().item()

    for i, x in enumerate((A, B, b)):
        v = grads[i].double() / grads[i].double().norm()
        h, args = 1e-4, [A.double(), B.double(), b.double()]
        ends = []
        for sign in (1, -1):
            moved = list(args)
            moved[i] = args[i] + sign * h * v
            ends.append(loss(*moved))
        slope = (ends[0] - ends[1]) / (2 * h)
        # Z is held in bf16: its rounding moves act' by at most about u |z act''|.
        assert abs(slope - grads[i].double().norm().item()) <= 2 * TWO * abs(slope)


DROP = [(1, 1), (1, 7), (3, 8), (33, 4095), (257, 1000), (1000, 64), (2, 100003), (70001, 9), (4096, 1024)]


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("rows,cols", DROP)
def test_dropout(gbr, rows, cols, dtype):
    g = rng(rows + cols)
    X, R = normal(g, (rows, cols), 1.0, dtype), normal(g, (rows, cols), 1.0, dtype)
    for p, seed, off, res in ((0.1, 0, 0, R), (0.5, 2 ** 64 - 1, 2 ** 64 - 1, None), (0.0, 1, 1, R), (1.0, 1, 1, R)):
        Y = gbr.dropout_add(X, res, p=p, seed=seed, offset=off)
        gbr.check_device()
        x = ref.drop(X.double(), p, seed, off)
        want = x if res is None else x + res.double()
        slack = 2.0 ** -22 * (x.abs() + (0 if res is None else res.double().abs()))
        if dtype is BF:
            slack = slack + 2 * U * want.abs()
        assert ((Y.double() - want).abs() <= slack).all()


def test_dropout_mask(gbr):
    """The share of kept values, and a mask that depends on nothing but its arguments."""
    X = torch.ones(512, 4096, device="cuda")
    Y = gbr.dropout_add(X, p=0.3, seed=1, offset=5)
    n, t = X.numel(), round(0.3 * 65536) / 65536
    kept = (Y != 0).double().mean().item()
    assert abs(kept - (1 - t)) <= 5 * math.sqrt(t * (1 - t) / n)
    assert torch.equal(Y, gbr.dropout_add(X.clone(), p=0.3, seed=1, offset=5))
    assert torch.equal(Y[:, :40], gbr.dropout_add(X[:, :40].contiguous(), p=0.3, seed=1, offset=5))
    assert torch.equal(Y[:7], gbr.dropout_add(X[:7], p=0.3, seed=1, offset=5))
    for kw in (dict(seed=2, offset=5), dict(seed=1, offset=6), dict(seed=1 + 2 ** 32, offset=5),
               dict(seed=1, offset=5 + 2 ** 32)):
        other = gbr.dropout_add(X, p=0.3, **kw)
        same = ((other != 0) == (Y != 0)).double().mean().item()
        assert abs(same - (t * t + (1 - t) ** 2)) <= 0.01
    x3 = torch.ones(4, 5, 24, device="cuda", dtype=BF)
    assert torch.equal(gbr.dropout_add(x3, p=0.5).view(20, 24), gbr.dropout_add(x3.view(20, 24), p=0.5))
    C = gbr.gemm_bias_act(torch.zeros(300, 8, device="cuda", dtype=BF), torch.zeros(8, 520, device="cuda", dtype=BF),
                          torch.ones(520, device="cuda"), p=0.3, seed=1, offset=5)
    assert torch.equal(C != 0, Y[:300, :520] != 0)


def test_dropout_past_32_bits(gbr):
    """Offsets of more than 2^32 bytes: the last rows of a 5.2 GB tensor."""
    rows, cols = 40000, 65536
    X = torch.ones(rows, cols, device="cuda", dtype=BF)
    gbr.dropout_add(X, p=0.5, seed=4, Y=X)
    gbr.check_device()
    keep = ref.keep_mask(1, cols, 0.5, 4, 0)[0]
    assert torch.equal(X[0].cpu() != 0, keep[0])
    tail = gbr.dropout_add(torch.ones(rows, 16, device="cuda", dtype=BF), p=0.5, seed=4)
    assert torch.equal(X[:, :16], tail)


MOE = [
    # T, D, F, E, top_k, act, gated, biases
    (1, 8, 8, 1, 1, "relu", False, True),
    (1, 1024, 2048, 8, 2, "relu", False, True),
    (2, 520, 264, 4, 4, "gelu", False, False),
    (3, 64, 72, 5, 2, "silu", True, True),
    (7, 256, 1000, 256, 8, "gelu_tanh", True, True),
    (16, 512, 512, 8, 2, "relu", False, True),
    (17, 1032, 136, 16, 3, "silu", True, False),
    (33, 2048, 1000, 64, 6, "silu", True, True),
    (64, 1024, 4096, 8, 2, "relu", False, True),
    (64, 264, 328, 2, 1, "none", False, True),
    (64, 128, 24, 64, 8, "gelu", True, True),
    (1, 4096, 14336, 2, 1, "relu", False, True),
    (5, 16, 6000, 3, 3, "gelu", False, True),
]


def moe_inputs(T, D, F, E, gated, biases, seed):
    g = rng(seed)
    F1 = 2 * F if gated else F
    return [normal(g, (T, D)), normal(g, (D, E), 1 / math.sqrt(D), torch.float32),
            normal(g, (E, D, F1), 1 / math.sqrt(D)), normal(g, (E, F1), 0.3, torch.float32) if biases else None,
            normal(g, (E, F, D), 1 / math.sqrt(F)), normal(g, (E, D), 0.3, torch.float32) if biases else None]


@pytest.mark.parametrize("T,D,F,E,top_k,act,gated,biases", MOE)
def test_moe(gbr, T, D, F, E, top_k, act, gated, biases):
    x = moe_inputs(T, D, F, E, gated, biases, T + D + F)
    Y, ids, w = gbr.moe_layer(*x, top_k=top_k, act=act, gated=gated, return_routing=True)
    gbr.check_device()
    ry, rids, rw = ref.moe(*x, top_k, act, gated)
    assert torch.equal(ids, rids)
    # Logits of about 1 from D fp32 products: 2^-24 sqrt(D) |x||w| or so, well below 1e-5.
    assert (w.double() - rw).abs().max().item() <= 1e-5
    close(Y, ry, TWO)
    assert torch.equal(Y, gbr.moe_layer(*x, top_k=top_k, act=act, gated=gated))


def test_moe_routing_edges(gbr):
    T, D, F, E = 9, 64, 64, 6
    x = moe_inputs(T, D, F, E, False, True, 3)
    # Equal logits: the lowest experts, equally weighted.
    x[1].zero_()
    Y, ids, w = gbr.moe_layer(*x, top_k=3, return_routing=True)
    assert torch.equal(ids.cpu(), torch.arange(3, dtype=torch.int64).expand(T, 3)) and (w - 1 / 3).abs().max() < 1e-6
    close(Y, ref.moe(*x, 3, "relu", False)[0], TWO)
    # One expert far ahead of all the others: it gets every token, the second weight vanishes.
    x[0][:, 0] = 1.0
    x[1].zero_()
    x[1][0, 4], x[1][0, 2] = 200.0, 50.0
    Y, ids, w = gbr.moe_layer(*x, top_k=2, return_routing=True)
    assert torch.equal(ids.cpu(), torch.tensor([4, 2], dtype=torch.int64).expand(T, 2))
    assert torch.equal(w.cpu(), torch.tensor([1.0, 0.0]).expand(T, 2))
    close(Y, ref.moe(*x, 2, "relu", False)[0], TWO)
    # A NaN logit ranks last; an expert that nobody takes may hold anything.
    x[1][1, 5] = float("nan")
    x[2][5], x[4][3] = float("nan"), float("inf")
    Y, ids, w = gbr.moe_layer(*x, top_k=2, return_routing=True)
    assert torch.equal(ids.cpu(), torch.tensor([4, 2], dtype=torch.int64).expand(T, 2))
    assert torch.isfinite(Y).all()
    # A token of NaN has its own row alone to spoil.
    x[0][4] = float("nan")
    Y2 = gbr.moe_layer(*x, top_k=2)
    rows = [t for t in range(T) if t != 4]
    # (It also picks experts of its own, which may change the order of the others' sums.)
    close(Y2[rows], Y[rows].double(), TWO)
    assert Y2[4].isnan().all()
    gbr.check_device()


def test_moe_every_token_alone(gbr):
    """A token's output does not depend on which tokens are served with it."""
    x = moe_inputs(20, 512, 264, 8, True, True, 12)
    Y = gbr.moe_layer(*x, top_k=2, act="silu", gated=True)
    for t in (0, 7, 19):
        one = gbr.moe_layer(x[0][t:t + 1].contiguous(), *x[1:], top_k=2, act="silu", gated=True)
        assert rel(one, Y[t:t + 1].double()) <= TWO


def test_streams_and_graphs(gbr):
    """On another stream than the tensors', and captured into a graph: the same bits as the plain call."""
    g = rng(2)
    M, K, N = 300, 520, 264
    A, B, R = normal(g, (M, K)), normal(g, (K, N), 1 / math.sqrt(K)), normal(g, (M, N))
    b = normal(g, (N,), 0.1, torch.float32)
    x = moe_inputs(5, 256, 512, 8, False, True, 9)

    def all_of():
        C, Z = gbr.gemm_bias_act(A, B, b, residual=R, act="gelu", p=0.1, seed=1, return_z=True)
        few = gbr.gemm_bias_act(A[:3], B, b, act="silu")
        return [C, Z, few, *gbr.gemm_bias_act_backward(R, A, B, Z, act="gelu", p=0.1, seed=1),
                gbr.dropout_add(R, C, p=0.3, seed=2), gbr.moe_layer(*x)]

    want = all_of()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = all_of()
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_of()
    for t in got:
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    gbr.check_device()


def test_feed_forward_block(gbr):
    """The operators as they are used together: forward and backward of a whole block, and one step of training."""
    from mbarrier_gemm_pipelines_gb300 import feed_forward
    g = rng(31)
    T, D, F = 192, 136, 520
    block = feed_forward.FeedForward(D, F, act="gelu", p=0.1, seed=99)
    x, dy = normal(g, (T, D)), normal(g, (T, D))
    y = block.forward(x, step=3)
    h, z = ref.linear(x, block.W1, block.b1, None, "gelu")
    want = ref.linear(h.to(BF), block.W2, block.b2, x, "none", 0.1, 99, 3)[0]
    close(y, want, TWO)
    grads = block.backward(dy)
    d2, dW2, db2, _ = ref.linear_grad(dy, h, block.W2, None, "none", 0.1, 99, 3)
    dx, dW1, db1, _ = ref.linear_grad(d2, x, block.W1, z, "gelu")
    for name, w in (("x", dx + dy.double()), ("W1", dW1), ("b1", db1), ("W2", dW2), ("b2", db2)):
        # Two products in a row: the operand roundings of both.
        assert rel(grads[name], w) <= 2 * TWO, name
    gbr.check_device()


@pytest.mark.parametrize("K", [16, 24])
def test_linear_past_32_bits(gbr, K):
    """More than 2^31 outputs, and than 2^32 bytes: the first and last rows of C, Z and dA."""
    M, N = 270336, 8008
    g = rng(K)
    A, B = normal(g, (M, K)), normal(g, (K, N), 1 / math.sqrt(K))
    R = torch.zeros(M, N, device="cuda", dtype=BF)
    R[-3:] = 1.0
    C, Z = gbr.gemm_bias_act(A, B, residual=R, act="silu", p=0.25, seed=8, C=R, return_z=True)
    gbr.check_device()
    for rows in (slice(0, 4), slice(M // 2, M // 2 + 4), slice(M - 4, M)):
        z = A[rows].double() @ B.double()
        close(Z[rows], z, ONE)
        scale = ref.keep_mask(1, 8, 0.25, 8, 0)[1]
        kept = C[rows].double() - (torch.arange(M)[rows] >= M - 3).double().cuda()[:, None]
        on = (kept != 0).double()
        close(kept, on * ref.act(z, "silu") * scale, 2 * TWO)     # (the residual 1 is rounded along)
        assert abs(on.mean().item() - 0.75) <= 0.02
    assert torch.equal(C[:4] != 0, ref.keep_mask(4, N, 0.25, 8, 0, "cuda")[0])
    dA, dB, db = gbr.gemm_bias_act_backward(Z, A, B, needs=(True, True, True))
    gbr.check_device()
    for rows in (slice(0, 4), slice(M - 4, M)):
        close(dA[rows], Z[rows].double() @ B.double().t(), TWO)
    close(db, Z.sum(0, dtype=torch.float64), 2.0 ** -12)


def test_moe_past_32_bits(gbr):
    """Experts whose weights start beyond 2^31 elements."""
    T, D, F, E = 3, 2048, 8192, 160
    g = rng(6)
    X, Wr = normal(g, (T, D)), torch.zeros(D, E, device="cuda")
    Wr[0, E - 1], Wr[0, E // 2], Wr[0, 0] = 3.0, 2.0, 1.0
    X[:, 0] = 1.0
    W1, W2 = (torch.zeros(E, *s, device="cuda", dtype=BF) for s in ((D, F), (F, D)))
    for e in (0, E // 2, E - 1):
        W1[e], W2[e] = normal(g, (D, F), D ** -0.5), normal(g, (F, D), F ** -0.5)
    Y, ids, w = gbr.moe_layer(X, Wr, W1, None, W2, None, top_k=3, return_routing=True)
    gbr.check_device()
    assert torch.equal(ids.cpu(), torch.tensor([E - 1, E // 2, 0]).expand(T, 3))
    close(Y, ref.moe(X, Wr, W1, None, W2, None, 3, "relu", False)[0], TWO)


def test_more_rows_than_tiles_of_a_launch(gbr):
    """Few columns and very many rows: every row tile is visited."""
    M, K, N = 600011, 8, 8
    g = rng(1)
    A, B = normal(g, (M, K)), normal(g, (K, N))
    close(gbr.gemm_bias_act(A, B), A.double() @ B.double(), ONE)
    dA, dB, db = gbr.gemm_bias_act_backward(A, A, B)
    gbr.check_device()
    close(dA, A.double() @ B.double().t(), TWO)
    close(dB, A.double().t() @ A.double(), TWO)
    bound = (2.0 ** -19 + M * 2.0 ** -24) * A.double().abs().sum(0)
    assert ((db.double() - A.double().sum(0)).abs() <= bound).all()


LIMIT_NS = 50_000_000


def expect_timeout(gbr):
    with pytest.raises(gbr.GbrError) as e:
        gbr.check_device()
    assert e.value.code == 6                                    # GBR_ERR_TIMEOUT
    gbr.check_device()                                          # reported once


@pytest.mark.parametrize("M,K,N,cta,item", [
    (37, 512, 4096, 0, 0),          # single tiles shared by a cluster: the first CTA's first stage
    (37, 4096, 4096, 5, 3),         # another CTA, a later stage
    (2048, 512, 4096, 0, 0),        # CTA pairs: the first item
    (2048, 2048, 4096, 3, 9),       # another pair, past the ring
    (2304, 4352, 4096, 1, 40),      # the cut last round
])
def test_linear_stage_never_filled(gbr, M, K, N, cta, item):
    """A stage that is never filled: the wait gives up, the call reports it, the next one is right."""
    g = rng(M)
    A, B = normal(g, (M, K)), normal(g, (K, N), 1 / math.sqrt(K))
    want = gbr.gemm_bias_act(A, B)
    gbr.check_device()
    for _ in range(2):
        gbr.selftest_linear_skip_load(A, B, cta, item, LIMIT_NS)
        expect_timeout(gbr)
    assert torch.equal(gbr.gemm_bias_act(A, B), want)
    gbr.selftest_linear_skip_load(A, B, 100000, 0, LIMIT_NS)    # no such CTA: nothing planted
    gbr.check_device()


@pytest.mark.parametrize("T,cta,item", [(1, 0, 0), (1, 7, 9), (40, 3, 12)])
def test_moe_stage_never_filled(gbr, T, cta, item):
    X, Wr, W1, _, W2, _ = moe_inputs(T, 1024, 10240, 4, False, False, T)      # work for every CTA
    want = gbr.moe_layer(X, Wr, W1, None, W2, None)
    gbr.check_device()
    for _ in range(2):
        gbr.selftest_moe_skip_load(X, Wr, W1, W2, 2, cta, item, LIMIT_NS)
        expect_timeout(gbr)
    assert torch.equal(gbr.moe_layer(X, Wr, W1, None, W2, None), want)


def test_binding_arguments(gbr):
    """What the binding refuses on a GPU tensor, with the exception's type; and it keeps no reference."""
    A, B = (torch.ones(16, 16, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    f, dC, Z = A.float(), A.clone(), A.clone()
    vec = torch.ones(16, device="cuda")

    def refused(kind, fn, *a, **kw):
        with pytest.raises(kind):
            fn(*a, **kw)

    fwd, bwd = gbr.gemm_bias_act, gbr.gemm_bias_act_backward
    for t in (f, A.half()):
        refused(TypeError, fwd, t, B)
        refused(TypeError, fwd, A, t)
        refused(TypeError, fwd, A, B, residual=t)
        refused(TypeError, fwd, A, B, C=t)
        refused(TypeError, bwd, t, A, B)
    refused(TypeError, fwd, A, B, vec.bfloat16())
    refused(TypeError, fwd, A, B, p="0.5")
    for bad in (A[:, :15], A[0], A[None]):
        refused(ValueError, fwd, bad, B)
        refused(ValueError, fwd, A, B, residual=bad)
        refused(ValueError, fwd, A, B, C=bad)
        refused(ValueError, fwd, A, B, Z=bad)
        refused(ValueError, bwd, dC, A, B, dA=bad)
    refused(ValueError, fwd, torch.ones(16, 32, device="cuda", dtype=torch.bfloat16)[:, ::2], B)
    refused(ValueError, fwd, A, B, vec[:8])
    refused(ValueError, fwd, A, B, vec.cpu())
    refused(ValueError, fwd, A, B, torch.ones(32, device="cuda")[::2])
    for act in ("tanh", 1, None, "relu\0"):
        refused(ValueError, fwd, A, B, act=act)
    for seed in (-1, 1 << 64, 0.5, "1", None):
        refused(ValueError, fwd, A, B, seed=seed, p=0.5)
        refused(ValueError, gbr.dropout_add, A, offset=seed)
    refused(ValueError, bwd, dC, A, B, act="relu")
    refused(ValueError, bwd, dC, A, B, needs=(True, True))
    refused(TypeError, bwd, dC, A, B, needs=3)
    refused(ValueError, bwd, dC, A, B, dbias=vec[:8])
    refused(gbr.GbrError, fwd, A, B, p=1.5)
    refused(gbr.GbrError, gbr.dropout_add, A, p=-0.5)
    W1, W2, Wr = A[None].expand(4, 16, 16).contiguous(), A[None].expand(4, 16, 16).contiguous(), f[:, :4].contiguous()
    refused(ValueError, gbr.moe_layer, A, Wr, W1, None, W2, None, gated=True)
    refused(ValueError, gbr.moe_layer, A, f, W1, None, W2, None)
    refused(ValueError, gbr.moe_layer, A, Wr, A, None, W2, None)
    refused(ValueError, gbr.moe_layer, A, Wr, W1, vec, W2, None)
    for k in (-1, 0, 5, 1 << 40):
        refused(gbr.GbrError, gbr.moe_layer, A, Wr, W1, None, W2, None, top_k=k)

    C = torch.empty_like(A)
    held = [sys.getrefcount(t) for t in (A, B, C, Z, vec)]
    needs = (True, False, True)
    for _ in range(20):
        assert fwd(A, B, vec, C=C) is C
        c, z = fwd(A, B, vec, C=C, Z=Z)
        assert c is C and z is Z
        assert gbr.dropout_add(A, A, p=0.5, Y=C) is C
        dA, dB, db = bwd(dC, A, B, Z, act="relu", dA=C, needs=needs)
        assert dA is C and dB is None and db.dtype == torch.float32 and db.shape == (16,)
        assert gbr.moe_layer(A, Wr, W1, None, W2, None, Y=C) is C
        refused(gbr.GbrError, fwd, A, B, vec, C=C, p=1.5)
    del c, z, dA
    assert held == [sys.getrefcount(t) for t in (A, B, C, Z, vec)]


@pytest.mark.parametrize("M,K,N", [(301, 520, 1000), (64, 512, 8192), (2048, 64, 64), (16, 4096, 16),
                                   (1536, 1536, 4096), (300, 4096, 2560)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_gradients_side_by_side(gbr, M, K, N, act):
    """dA and dB may run next to one another: each has the bits of a call for it alone, and what follows the call in
    its stream (an operator whose launch overlaps, or any other kernel) finds both finished."""
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    A, B, dC, Z = (torch.randn(s, generator=g, device="cuda").to(BF) for s in ((M, K), (K, N), (M, N), (M, N)))
    one = gbr.gemm_bias_act_backward(dC, A, B, Z, act=act, needs=(True, False, False))[0]
    two = gbr.gemm_bias_act_backward(dC, A, B, Z, act=act, needs=(False, True, False))[1]
    dA, dB = torch.empty_like(A), torch.empty_like(B)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(20):
        dA.fill_(math.nan)
        dB.fill_(math.nan)
        gbr.gemm_bias_act_backward(dC, A, B, Z, act=act, dA=dA, dB=dB)
        if i % 2:
            a, b = gbr.dropout_add(dA, p=0.0), dB
        else:
            b, a = gbr.dropout_add(dB, p=0.0), dA
        wrong += (a != one).sum() + (b != two).sum()
    assert int(wrong) == 0


@pytest.mark.parametrize("lay", [padded, spaced])
@pytest.mark.parametrize("M,K,N", [(1537, 1031, 1543), (37, 2049, 5003), (4096, 72, 1030)])
def test_strides_large(gbr, lay, M, K, N):
    """The same for products that run on CTA pairs, whose copies are launched together, and for lopsided ones."""
    test_strides(gbr, lay, M, K, N)
