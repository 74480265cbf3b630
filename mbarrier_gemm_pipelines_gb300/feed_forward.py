"""A transformer's feed-forward block from the library's operators: a training
step of the dense block and the serving of its mixture-of-experts form.

    y = x + dropout(act(x W1 + b1) W2 + b2)

``FeedForward.forward`` is two ``gemm_bias_act`` calls, the second with dropout
and the residual in its epilogue; ``backward`` is two ``gemm_bias_act_backward``
calls and one ``dropout_add`` without dropout for the sum of the two gradients
of x.  The dropout mask is recomputed from (seed, step), never stored.
``ExpertFeedForward`` serves a few tokens at a time through ``moe_layer``.
Run ``python -m mbarrier_gemm_pipelines_gb300.feed_forward`` for an example of
both on the current GPU.
"""
from __future__ import annotations

import torch

from . import _operators as ops
from ._binding import check_device


def _weights(shape, std, g):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).bfloat16()


class FeedForward:
    def __init__(self, D, F, act="gelu", p=0.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(int(seed))
        self.act, self.p, self.seed = act, p, seed
        self.W1, self.W2 = _weights((D, F), D ** -0.5, g), _weights((F, D), F ** -0.5, g)
        self.b1, self.b2 = torch.zeros(F, device="cuda"), torch.zeros(D, device="cuda")
        self._saved = None

    def forward(self, x, step=0):
        h, z = ops.gemm_bias_act(x, self.W1, self.b1, act=self.act, return_z=True)
        y = ops.gemm_bias_act(h, self.W2, self.b2, residual=x, p=self.p, seed=self.seed, offset=step)
        self._saved = x, h, z, step
        return y

    def backward(self, dy):
        """Gradients of x and of the parameters for dy, by name."""
        x, h, z, step = self._saved
        dh, dW2, db2 = ops.gemm_bias_act_backward(dy, h, self.W2, p=self.p, seed=self.seed, offset=step)
        dx, dW1, db1 = ops.gemm_bias_act_backward(dh, x, self.W1, z, act=self.act)
        ops.dropout_add(dx, dy, p=0.0, Y=dx)
        return {"x": dx, "W1": dW1, "b1": db1, "W2": dW2, "b2": db2}

    def sgd(self, grads, lr):
        for name in ("W1", "b1", "W2", "b2"):
            getattr(self, name).add_(grads[name], alpha=-lr)


class ExpertFeedForward:
    def __init__(self, D, F, experts, top_k=2, act="relu", gated=False, seed=0):
        g = torch.Generator(device="cuda").manual_seed(int(seed))
        self.top_k, self.act, self.gated = top_k, act, gated
        F1 = 2 * F if gated else F
        self.Wr = torch.randn((D, experts), generator=g, device="cuda") * D ** -0.5
        self.W1, self.W2 = _weights((experts, D, F1), D ** -0.5, g), _weights((experts, F, D), F ** -0.5, g)
        self.b1 = torch.zeros(experts, F1, device="cuda")
        self.b2 = torch.zeros(experts, D, device="cuda")

    def forward(self, x):
        return ops.moe_layer(x, self.Wr, self.W1, self.b1, self.W2, self.b2, top_k=self.top_k, act=self.act,
                             gated=self.gated)


def example(steps=20, T=512, D=1024, F=4096):
    """Fits the block to a fixed target by plain gradient steps and serves one token through experts."""
    g = torch.Generator(device="cuda").manual_seed(1)
    block = FeedForward(D, F, act="gelu", p=0.1, seed=7)
    x = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    target = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    losses = []
    for step in range(steps):
        e = block.forward(x, step).float() - target.float()
        losses.append(e.square().mean())
        block.sgd(block.backward((e * (2.0 / T)).bfloat16()), lr=1e-3)
    experts = ExpertFeedForward(D, F, experts=8)
    y = experts.forward(x[:1])
    check_device()
    return [float(v) for v in losses], y


if __name__ == "__main__":
    losses, y = example()
    print("loss %.4f -> %.4f over %d steps; one token through experts: %s"
          % (losses[0], losses[-1], len(losses), list(y.shape)))
