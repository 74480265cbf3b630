"""residual_norm and its gradients on rows of extreme size, on the GPU against their definitions in 64 bits.

Bars are those of test_gpu_block_operators.py.  They are relative to the sums of the sizes of what is added, so they do not
change when a row and what goes with it are multiplied by a power of ten, as long as nothing leaves fp32's normal range
on the way: with rows of 1e15 (1e-15) roots are 1e-15 (1e15), every product of two of the operands and its mean lies
between 1e-30 and 1e30, and so do the gradients.
"""
import pytest
import torch

import test_gpu_block_operators as block
from test_gpu_block_operators import gbr  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

GRADS = [
    # rows, cols, type, post, gates, pre, residual, scale: one of each kernel and of each way through it
    (5, 257, "fp32", True, 0, True, True, 0.5),         # a row a group of threads
    (7, 31, "bf16", False, 0, True, True, 1.0),
    (6, 264, "bf16", True, 2, False, True, 1.0),        # the norm in front of the sum alone
    (513, 1000, "bf16", True, 0, True, True, 0.25),     # streamed
    (1300, 4096, "bf16", True, 1, True, True, 0.25),    # two vectors a thread
    (700, 1024, "fp32", True, 700, True, True, 1.0),    # a gate an element
    (301, 1001, "bf16", True, 1, True, True, 0.5),      # rows that start anywhere
    (6, 16384, "bf16", True, 1, True, True, 1.0),       # rows cut over a cluster
    (4, 9000, "fp32", True, 4, True, True, 1.0),        # means first
    (5, 9001, "bf16", True, 1, True, True, 0.5),
]


@pytest.mark.parametrize("size", [1e15, 1e-15])
@pytest.mark.parametrize("case", GRADS, ids=["-".join(map(str, c)) for c in GRADS])
def test_gradients_of_large_and_small_rows(gbr, case, size):  # noqa: F811
    """Both terms of each gradient count: dS is as large as what dH brings."""
    a = block.norm_grad_inputs(case)
    a.update(eps=0.0, X=(a["X"].double() * size).to(a["X"].dtype), S=(a["S"].double() * size).to(a["S"].dtype),
             dS=(a["dS"].double() / size).to(a["dS"].dtype))
    block.check_norm_grads(a, gbr.residual_norm_backward(**a))
    gbr.check_device()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("cols", [64, 65, 9000])
@pytest.mark.parametrize("post", [False, True])
def test_sums_over_no_rows_are_zero(gbr, cols, post, dtype):  # noqa: F811
    """Whatever gate and weights hold; and a gate without rows is not read (the buffer behind the pointer has some here)."""
    x = torch.empty(0, cols, device="cuda", dtype=dtype)
    w = torch.full((cols,), float("inf"), device="cuda")
    gate = torch.full((5, cols), float("nan"), device="cuda", dtype=dtype)
    dX, dR, dpost, dgate, dpre = gbr.residual_norm_backward(x, x, x, x, post=w if post else None, gate=gate, pre=w)
    assert dX.shape == dR.shape == x.shape and dgate.shape == gate.shape
    for t in (dgate, dpre) + ((dpost,) if post else ()):
        assert (t == 0).all()
    if post:
        sums = torch.ones(2, cols, device="cuda")
        code = gbr.BF16 if dtype == torch.bfloat16 else gbr.F32_FFMA
        gbr.check(gbr.lib().residual_norm_backward(None, cols, None, cols, None, cols, None, cols, w.data_ptr(), gate.data_ptr(),
                                                   cols, 0, 1.0, w.data_ptr(), 1e-6, None, cols, None, cols,
                                                   sums[0].data_ptr(), None, cols, sums[1].data_ptr(), 0, cols, code,
                                                   torch.cuda.current_stream().cuda_stream))
        assert (sums == 0).all()
    gbr.check_device()


def equal_terms(cols, dtype, **kw):
    """Two rows of one value: each of thousands of roundings of a sum then goes the same way for long, where those of random
    values would cancel."""
    def full(v, shape, t=dtype):
        return torch.full(shape, v, device="cuda", dtype=t)
    return dict({n: full(v, (2, cols)) for n, v in kw.items()}, post=full(0.7, (cols,), torch.float32),
                pre=full(1.1, (cols,), torch.float32), gate=None, scale=1.0, eps=block.EPS)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("cols", [(1 << 22) + 3, 1 << 23])
def test_sums_of_millions_of_columns(gbr, cols, dtype):  # noqa: F811
    """Bars in units u = 2^-24 of a value, the rounding of one operation.  A sum adds at most 16 terms, the runs with two
    roundings, 10 levels over the CTA: 28 u.  A root halves that and has 4 u of its own (2 ulp), eps and the
    mean 1 u: 19 u.
      S      root, five operations: 24 u of m                             below 2^-19 m
      H      S, its root, two products: 24 + 24 + 19 + 2 = 69 u           below 2^-17 m (|H| is at most its m)
      dR     root twice (38), the signed mean (28, its terms two), eight operations: 80 u of m      2^-17 m
      dX     what dR has, and the same once more: 160 u of m               2^-16 m
      dpost, dpre   dR's or less, 19 for the root, two rows: below         2^-17 m
    One after another, 4096 terms of 0.3^2 were off by 2^-15 of their sum.
    """
    a = equal_terms(cols, dtype, X=0.3, R=0.2)
    S, H = gbr.residual_norm(**a)
    s, h, m = block.ref.residual_norm(**a)
    block.within(S, s, 2.0 ** -19 * m, "S")
    block.within(H, h, 2.0 ** -17 * m * block.ref.root(s, a["eps"]) * a["pre"].double(), "H")
    del s, h, m
    # Half of dH and dS the other way: no projection cancels its other term.
    a = equal_terms(cols, dtype, X=0.3, S=0.3, dH=0.7, dS=0.1)
    a["dH"][:, ::2], a["dS"][:, ::2] = -0.2, 0.4
    grads = gbr.residual_norm_backward(**a)
    g, m = block.ref.residual_norm_backward(**a)
    for name, got in zip(block.NAMES, grads):
        if name == "dgate":
            assert got is None
            continue
        block.within(got, g[name], 2.0 ** (-16 if name == "dX" else -17) * m[name], name)
    gbr.check_device()


def test_many_gates_over_no_rows(gbr):  # noqa: F811
    """More of them than one launch's grid has places."""
    x = torch.empty(0, 33, device="cuda", dtype=torch.bfloat16)
    gate = torch.full((140001, 33), float("inf"), device="cuda", dtype=torch.bfloat16)
    view, whole = block.placed(torch.ones_like(gate), 3, 35)
    got = gbr.residual_norm_backward(x, None, x, None, gate=gate, dgate=view)[3]
    assert got is view and not view.any() and (block.others(view, whole) == 5).all()
    gbr.check_device()


FORWARD = [(1, 4096, "bf16", True, 1, True, True, 1.0), (301, 1001, "fp32", True, 7, True, True, 0.25), (2500, 2048, "bf16", True, 1, True, True, 0.5),
           (3, 20000, "fp32", True, 0, True, True, 1.0), (2, 40000, "bf16", True, 1, True, True, 1.0)]


@pytest.mark.parametrize("size", [1e15, 1e-15])
@pytest.mark.parametrize("case", FORWARD, ids=["-".join(map(str, c)) for c in FORWARD])
def test_large_and_small_rows(gbr, case, size):  # noqa: F811
    """A block's output of any size beside a residual stream of it, whose gate brings both together."""
    a = block.norm_inputs(case)
    a.update(eps=0.0, X=(a["X"].double() * size).to(a["X"].dtype), R=(a["R"].double() * size).to(a["R"].dtype))
    if a["gate"] is not None:
        a["gate"] = (a["gate"].double() * size).to(a["gate"].dtype)
    block.check_norm(a, *gbr.residual_norm(**a))
    gbr.check_device()
