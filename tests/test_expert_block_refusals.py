"""What the expert block refuses before it computes anything (no GPU)."""
import pytest
import torch


@pytest.mark.parametrize("top_k", [-1, 0, 7, 100])
def test_more_or_fewer_choices_than_experts(top_k):
    from mbarrier_gemm_pipelines_gb300 import feed_forward
    net = object.__new__(feed_forward.ExpertFeedForward)        # __init__ makes its weights on a GPU
    net.Wr, net.top_k, net.gated = torch.zeros(8, 6), top_k, False
    with pytest.raises(ValueError, match="top_k"):
        net.forward_sorted(torch.zeros(70, 8))
    with pytest.raises(ValueError, match="top_k"):
        net.forward(torch.zeros(70, 8))
