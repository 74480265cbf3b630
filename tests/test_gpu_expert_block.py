"""The expert block's two forms, for few tokens and with sorted rows, in turn."""
import pytest
import torch

from test_gpu_block_operators import gbr, normal, rng  # noqa: F401  (gbr: the fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture
def net(gbr):  # noqa: F811
    from mbarrier_gemm_pipelines_gb300 import feed_forward
    return feed_forward.ExpertFeedForward(136, 264, experts=6, top_k=2, act="silu", seed=4)


def test_backward_needs_a_pass_that_kept_its_tensors(gbr, net):  # noqa: F811
    """Not an older one's: neither before any pass nor after one of few tokens."""
    g = rng(1)
    x, dy = normal(g, (40, 136)), normal(g, (40, 136))
    with pytest.raises(RuntimeError):
        net.backward(dy)
    net.forward_sorted(x)
    assert net.backward(dy)["x"].shape == x.shape
    net.forward(normal(g, (40, 136)))
    with pytest.raises(RuntimeError):
        net.backward(dy)
    net.forward_sorted(x)
    with pytest.raises(Exception):
        net.forward_sorted(x[:, :8])
    with pytest.raises(RuntimeError):
        net.backward(dy)
    gbr.check_device()


@pytest.mark.parametrize("what", ["equal", "nan", "infinite"])
def test_both_forms_choose_the_same_experts(gbr, net, what):  # noqa: F811
    """Of equal logits the lowest expert; NaN behind all others.  Biases tell the experts apart.  Bar: each form rounds the
    hidden values, outputs and sums to bf16, 2^-8 relative to the value a rounding."""
    g = rng(2)
    x = normal(g, (50, 136))
    net.b2.copy_(normal(g, net.b2.shape, dtype=torch.float32))
    if what == "equal":
        x[::2] = 0                          # all logits are zero
        net.Wr[:, 3] = net.Wr[:, 1]
    elif what == "nan":
        net.Wr[5, 0], net.Wr[7, 4] = float("nan"), float("nan")
    else:
        x.abs_()
        net.Wr[5, 2] = float("-inf")
    few, many = net.forward(x), net.forward_sorted(x)
    assert torch.isfinite(few.float()).all()
    _, ids, weights, positions, offsets = net._saved[:5]
    assert ids.dtype == torch.int64 and int(offsets[-1]) == 100
    if what == "equal":
        assert (ids[::2] == torch.tensor([0, 1], device="cuda")).all()
    err = (few.double() - many.double()).norm() / few.double().norm()
    assert err <= 4 * 2.0 ** -8
    gbr.check_device()
