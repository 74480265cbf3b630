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
