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
