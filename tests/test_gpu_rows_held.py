"""Rows sorted by expert and back at sizes where a CTA has several turns of tokens and fetches their places first, and
beyond the choices that it holds.

A CTA of 256 threads (fewer where a token does not fill them) holds 256 choices; there are at most 4 (fp32: 3) CTAs an SM for
bf16 rows, so of 152 SMs at most 608 (456) with rows of 2048 columns and more, and 8 times as many where a token is one
warp's.  With more tokens than those take at once, places are held; with more than 256 choices in a CTA's run of
tokens they are fetched again.

Bars as in test_gpu_block_operators.py: combine (k + 2) 2^-23 of the sizes, dYs 2^-23, dweights 2^-17 of the sizes.
"""
import pytest
import torch

import test_gpu_block_operators as block
from test_gpu_block_operators import gbr  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

HELD = [
    # T, k, D, E, type, struck out
    (8000, 2, 512, 8, "bf16", 0.1), (8000, 2, 512, 8, "fp32", 0.1), (8001, 6, 512, 64, "bf16", 0.25), (8001, 6, 512, 64, "fp32", 0.25),
    (4096, 2, 2048, 8, "bf16", 0.0), (4096, 2, 2048, 8, "fp32", 0.25), (2500, 6, 2048, 64, "bf16", 0.25), (2500, 6, 2048, 64, "fp32", 0.0),
    (3001, 1, 4104, 5, "bf16", 0.5), (1500, 1, 4100, 5, "fp32", 0.0), (2003, 3, 1003, 7, "bf16", 0.25), (3001, 4, 333, 9, "fp32", 0.25),
]
AGAIN = [
    # So many tokens that a CTA's run has more than 256 choices, once or several times.
    (60000, 8, 16, 16, "bf16", 0.2), (400007, 8, 8, 16, "bf16", 0.1), (200000, 8, 9, 16, "fp32", 0.25), (20000, 100, 8, 128, "bf16", 0.25),
    (9000, 255, 8, 256, "bf16", 0.25), (9001, 256, 9, 256, "fp32", 0.25),
]
BEYOND = [(700, 300, 40, 512, "bf16", 0.25), (90, 300, 41, 512, "fp32", 0.25), (3, 1024, 264, 1024, "bf16", 0.0), (5000, 257, 8, 300, "bf16", 0.5)]


def some_choices(T, k, E, masked, seed):
    """A token's choices are different experts, as a router's are, in any order."""
    g = block.rng(seed)
    if T * E <= 1 << 26:
        ids = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].contiguous()
    else:
        ids = (torch.randint(0, E, (T, 1), generator=g, device="cuda") + torch.arange(k, device="cuda")) % E
    ids[torch.rand((T, k), generator=g, device="cuda") < masked] = -1
    return ids


def check(gbr, case, start=0):  # noqa: F811
    T, k, D, E, dt, masked = case
    t, g = block.TYPES[dt], block.rng(7)
    ids = some_choices(T, k, E, masked, 6)
    p, o = gbr.moe_sort(ids, E)
    # The stable order by expert, those that are struck out behind all others.
    keys = torch.where(ids < 0, E, ids).flatten()
    order = keys.sort(stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device="cuda")
    assert torch.equal(p, torch.where(ids < 0, -1, place.view(T, k)).int())
    assert torch.equal(o, torch.searchsorted(keys.sort().values, torch.arange(E + 1, device="cuda")).int())
    on = p >= 0
    at, token = p[on].long(), torch.nonzero(on)[:, 0]

    def matrix(rows):
        m = block.normal(g, (rows, D), 1.0, t)
        return block.placed(m, start, D + 3)[0] if start else m

    X, Ys, dY, R = matrix(T), matrix(T * k), matrix(T), matrix(T)
    w = torch.rand((T, k), generator=g, device="cuda")
    Xs = gbr.moe_dispatch(X, p, o)
    want = torch.zeros(T * k, D, device="cuda", dtype=t)
    want[at] = X[token]
    assert torch.equal(Xs, want)
    Y = gbr.moe_combine(Ys, p, w, residual=R)
    dYs, dw = gbr.moe_combine_backward(dY, Ys, p, o, w)
    wide = torch.zeros(T * k, D, device="cuda", dtype=torch.float64)
    wide[at] = w[on].double()[:, None] * dY[token].double()
    block.within(dYs, wide, 2.0 ** -23 * wide.abs(), "dYs")
    for first in range(0, T, max(1, (1 << 24) // (k * D))):
        s = slice(first, min(T, first + max(1, (1 << 24) // (k * D))))
        rows = Ys.double()[p[s].clamp(min=0).long()] * on[s][..., None]
        term = (w[s].double() * on[s])[..., None] * rows
        m = term.abs().sum(1) + R[s].double().abs()
        block.within(Y[s], term.sum(1) + R[s].double(), (k + 2) * 2.0 ** -23 * m, "Y")
        prod = rows * dY[s].double()[:, None]
        block.within(dw[s], prod.sum(2), 2.0 ** -17 * prod.abs().sum(2), "dweights")
    gbr.check_device()


@pytest.mark.parametrize("start", [0, 3])
@pytest.mark.parametrize("case", HELD + AGAIN + BEYOND, ids=["-".join(map(str, c)) for c in HELD + AGAIN + BEYOND])
def test_rows_of_many_tokens(gbr, case, start):  # noqa: F811
    """`start` 0: contiguous matrices; 3: that many elements behind a boundary of 16 bytes, and three more a row."""
    check(gbr, case, start)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_rows_without_columns(gbr, dtype):  # noqa: F811
    """The products over no columns are zero, and nothing else is written."""
    p, o = gbr.moe_sort(torch.tensor([[0, 1], [1, -1]], device="cuda"), 2)
    x, y, w = torch.empty(2, 0, device="cuda", dtype=dtype), torch.empty(4, 0, device="cuda", dtype=dtype), torch.rand(2, 2, device="cuda")
    dw = torch.ones(2, 2, device="cuda")
    dYs, got = gbr.moe_combine_backward(x, y, p, o, w, dweights=dw)
    assert dYs.shape == (4, 0) and got is dw and not dw.any()
    assert gbr.moe_dispatch(x, p, o).shape == (4, 0) and gbr.moe_combine(y, p, w).shape == (2, 0)
    gbr.check_device()
