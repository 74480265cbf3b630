"""More of the feed-forward operators' paths on the GPU: the gradients' products in one grid and one after the other,
expert layers of more parts than SMs and of many experts, and rows past 32 bits.  Bars as in test_gpu_operators.py."""
import math
import random

import pytest
import torch

import ffn_reference as ref
from gpu_helpers import load_library, require_gpu
from test_gpu_operators import BF, TWO, close, moe_inputs, normal, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gbr():
    require_gpu()
    return load_library()


def shapes():
    r = random.Random(20)
    out = [(1, 8, 8), (1, 4096, 64), (2, 64, 4096), (8192, 8, 8), (64, 64, 64), (2048, 64, 128), (4096, 512, 512),
           (1000, 2048, 16), (16, 16, 9000), (700, 1032, 264)]
    while len(out) < 40:
        M, K, N = (int(math.exp(r.uniform(math.log(lo), math.log(4000)))) for lo in (1, 8, 8))
        if M * K * N < 2 ** 31:
            out.append((M, -(-K // 8) * 8, -(-N // 8) * 8))
    return out


@pytest.mark.parametrize("M,K,N", shapes())
def test_gradients_together_and_alone(gbr, M, K, N):
    """dA and dB have the bits of a call for each alone, whatever they share a launch with, and are right."""
    g = rng(M + 3 * K + 7 * N)
    A, B, dC, Z = normal(g, (M, K)), normal(g, (K, N), K ** -0.5), normal(g, (M, N)), normal(g, (M, N))
    for act in ("none", "gelu"):
        kw = dict(act=act, p=0.1, seed=3)
        before = gbr.launch_count()
        dA, dB, db = gbr.gemm_bias_act_backward(dC, A, B, Z, **kw)
        assert gbr.launch_count() - before <= 6
        gbr.check_device()
        alone = [gbr.gemm_bias_act_backward(dC, A, B, Z, needs=tuple(j == i for j in range(3)), **kw)[i] for i in range(3)]
        for x, y in zip((dA, dB, db), alone):
            assert torch.equal(x, y)
        rA, rB, _, _ = ref.linear_grad(dC, A, B, Z, act, 0.1, 3, 0)
        close(dA, rA, TWO)
        close(dB, rB, TWO)


def test_versions_of_given_outputs(gbr):
    """A tensor written in place moves its version once a call; a refused call and a new output leave versions alone."""
    A, B = torch.ones(16, 24, device="cuda", dtype=BF), torch.ones(24, 32, device="cuda", dtype=BF)
    C, Z, dA, dB = (torch.zeros(s, device="cuda", dtype=BF) for s in ((16, 32), (16, 32), (16, 24), (24, 32)))
    db, X, Wr = torch.zeros(32, device="cuda"), torch.zeros(16, 24, device="cuda", dtype=BF), torch.ones(24, 2, device="cuda")
    W1, W2 = torch.ones(2, 24, 8, device="cuda", dtype=BF), torch.ones(2, 8, 24, device="cuda", dtype=BF)
    gbr.gemm_bias_act(A, B, C=C, Z=Z)
    gbr.gemm_bias_act_backward(C, A, B, dA=dA, dB=dB, dbias=db)
    gbr.dropout_add(X, Y=X)
    gbr.moe_layer(A, Wr, W1, None, W2, None, Y=dA)
    with pytest.raises(gbr.GbrError):
        gbr.gemm_bias_act(A, B, C=C, p=2.0)
    assert [t._version for t in (A, B, C, Z, dA, dB, db, X, Wr, W1, W2)] == [0, 0, 1, 1, 2, 1, 1, 1, 0, 0, 0]
    assert gbr.dropout_add(X)._version == 0
    w = torch.ones(4, 8, device="cuda", requires_grad=True)
    x = torch.ones(4, 8, device="cuda")
    y = (w * x).sum()
    gbr.dropout_add(x, Y=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        x = torch.ones(4, 8, device="cuda")
    assert gbr.dropout_add(x, p=0.0, Y=x) is x


@pytest.mark.parametrize("top_k", [-1, 0, 5, 1 << 40, 1 << 62])
def test_wrong_top_k_with_routing(gbr, top_k):
    """Refused as such, before the routing's tensors are made in that size."""
    A, W = torch.ones(16, 16, device="cuda", dtype=BF), torch.ones(4, 16, 16, device="cuda", dtype=BF)
    with pytest.raises(gbr.GbrError, match="top_k"):
        gbr.moe_layer(A, torch.ones(16, 4, device="cuda"), W, None, W, None, top_k=top_k, return_routing=True)


def test_no_memory_for_an_output(gbr):
    """Outputs of 2 TB: PyTorch's own error, as for any of its tensors, and the next call works."""
    n = 1 << 20
    A, B = torch.ones(n, 8, device="cuda", dtype=BF), torch.ones(8, n, device="cuda", dtype=BF)
    with pytest.raises(torch.OutOfMemoryError):
        gbr.gemm_bias_act(A, B)
    assert (gbr.gemm_bias_act(A[:16], B[:, :16].contiguous()) == 8).all()
    gbr.check_device()


MOE = [
    # T, D, F, E, top_k, act, gated, biases
    (64, 256, 14336, 64, 8, "relu", False, True),     # more units a part than fit: several parts a CTA
    (64, 256, 14336, 64, 8, "silu", True, True),
    (1, 64, 65536, 2, 2, "gelu", False, True),
    (48, 128, 16384, 40, 7, "gelu_tanh", True, False),
    (40, 512, 72, 250, 8, "silu", True, True),        # four tokens a router cluster, 64 lanes along the experts
    (64, 128, 64, 256, 8, "relu", False, True),
    (33, 8, 8, 129, 1, "gelu", True, True),
    (20, 64, 520, 128, 8, "silu", False, True),
    (64, 1000, 200, 3, 3, "silu", True, True),        # every expert has every token
    (2, 8, 4096, 256, 8, "relu", True, False),
]


@pytest.mark.parametrize("T,D,F,E,top_k,act,gated,biases", MOE)
def test_moe_cuts_and_routers(gbr, T, D, F, E, top_k, act, gated, biases):
    x = moe_inputs(T, D, F, E, gated, biases, 3 * T + D + F)
    Y, ids, w = gbr.moe_layer(*x, top_k=top_k, act=act, gated=gated, return_routing=True)
    gbr.check_device()
    ry, rids, rw = ref.moe(*x, top_k, act, gated)
    assert torch.equal(ids, rids)
    assert (w.double() - rw).abs().max().item() <= 1e-5
    close(Y, ry, TWO)
    for _ in range(10):
        assert torch.equal(Y, gbr.moe_layer(*x, top_k=top_k, act=act, gated=gated))


@pytest.mark.parametrize("chosen", [8, 9, 40, 250])
def test_moe_skewed_routing(gbr, chosen):
    """All tokens on the same 8 experts, or spread over as many as are given: what the scratch has to hold."""
    T, D, F, E, top_k = 64, 64, 8192, 250, 8
    x = moe_inputs(T, D, F, E, False, True, chosen)
    # Column t of X is one for token t alone, so that row t of Wr is its logits.
    x[0].zero_()
    x[0][:, :T] = torch.eye(T, device="cuda").to(BF)
    x[1].copy_(torch.arange(E, 0, -1, device="cuda").float() * -1e-3)
    pick = torch.stack([(torch.arange(top_k) + t * 5) % chosen for t in range(T)]).cuda()
    x[1].scatter_(1, pick, torch.linspace(1.0, 2.0, top_k, device="cuda").expand(T, top_k))
    Y, ids, w = gbr.moe_layer(*x, top_k=top_k, return_routing=True)
    gbr.check_device()
    ry, rids, rw = ref.moe(*x, top_k, "relu", False)
    assert torch.equal(ids, rids) and ids.unique().numel() == chosen
    assert (w.double() - rw).abs().max().item() <= 1e-5
    close(Y, ry, TWO)


def test_linear_mask_and_weights_past_32_bits(gbr):
    """More than 2^31 outputs: the mask of every row against the generator's reference (its first 16 columns; the last
    by the narrow and the whole call of dropout_add), and dB, whose contraction runs along those rows."""
    M, K, N = 270336, 16, 8008
    g = rng(77)
    A, B = normal(g, (M, K)), normal(g, (K, N), K ** -0.5)
    C = gbr.gemm_bias_act(A, B, act="none", p=0.25, seed=8, offset=3)
    keep = ref.keep_mask(M, 16, 0.25, 8, 3, "cuda")[0]
    assert (C[:, :16][~keep] == 0).all()
    # A kept product that is exactly zero is rarer than 2^-16: 16 bf16 products would have to cancel to the bit.
    assert ((C[:, :16] == 0) & keep).sum() <= keep.numel() * 2.0 ** -16
    ones = gbr.dropout_add(torch.ones(M, N, device="cuda", dtype=BF), p=0.25, seed=8, offset=3)
    assert torch.equal(ones[:, :16] != 0, keep)
    dropped = ones == 0
    assert (C[dropped] == 0).all()
    del ones
    dC = C
    dA, dB, db = gbr.gemm_bias_act_backward(dC, A, B, p=0.25, seed=8, offset=3)
    gbr.check_device()
    want, sums, total, scale = 0.0, 0.0, 0.0, 65536 / 49152
    for r in range(0, M, 16896):
        rows = slice(r, r + 16896)
        dz = dC[rows].double().masked_fill(dropped[rows], 0.0) * scale
        close(dA[rows], dz @ B.double().t(), TWO)
        want, sums, total = want + A[rows].double().t() @ dz, sums + dz.sum(0), total + dz.abs().sum(0)
    close(dB, want, TWO)
    assert ((db.double() - sums).abs() <= (2.0 ** -19 + M * 2.0 ** -24) * total).all()
