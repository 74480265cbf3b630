"""A transformer's feed-forward block from the library's operators: a training
step of the dense block and of its mixture-of-experts form, and the serving of
both.

    y = x + dropout(act(x W1 + b1) W2 + b2)

``FeedForward.forward`` is two ``gemm_bias_act`` calls, the second with dropout
and the residual in its epilogue; ``backward`` is two ``gemm_bias_act_backward``
calls and one ``dropout_add`` without dropout for the sum of the two gradients
of x.  The dropout mask is recomputed from (seed, step), never stored.

``NormedFeedForward`` puts the block between norms: the block sees norm(x) pre,
and x gains scale * gate * norm(block) post, one ``residual_norm`` call that also
makes the next block's input.

``ExpertFeedForward.forward`` serves a few tokens at a time through ``moe_layer``
and more of them by sorting their rows by expert: ``moe_sort``,
``moe_dispatch``, the experts' products on their runs of rows, ``moe_combine``;
``backward`` goes the same way back.

``FeedForward4Bit`` serves a dense block in microscaled 4-bit floating point.

Run ``python -m mbarrier_gemm_pipelines_gb300.feed_forward`` for an example of
all of them on the current GPU.
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
        self._saved = None

    def forward(self, x):
        if x.shape[0] <= 64:
            self._saved = None              # nothing of an earlier pass for backward
            return ops.moe_layer(x, self.Wr, self.W1, self.b1, self.W2, self.b2, top_k=self.top_k, act=self.act,
                                 gated=self.gated)
        return self.forward_sorted(x)

    def forward_sorted(self, x, live=None):
        """Any number of tokens; `live` [T] (bool) strikes out the others, whose output is zero.  Keeps what backward needs."""
        self._saved = None
        if not 1 <= self.top_k <= self.Wr.shape[1]:
            raise ValueError("top_k must be 1 to %d, the number of experts, got %d" % (self.Wr.shape[1], self.top_k))
        logits = x.float() @ self.Wr
        # As moe_layer chooses: of equal logits the lowest expert, NaN behind all others (topk puts NaN first, ties anyhow).
        ids = (-logits).sort(dim=1, stable=True).indices[:, :self.top_k].contiguous()
        weights = torch.softmax(logits.gather(1, ids), 1)
        if live is not None:
            ids = torch.where(live[:, None], ids, -1)
        positions, offsets = ops.moe_sort(ids, self.Wr.shape[1])
        rows = ops.moe_dispatch(x, positions, offsets)
        runs = offsets.tolist()             # the products' sizes: the one wait for the GPU
        hidden, saved = torch.empty(rows.shape[0], self.W2.shape[1], dtype=x.dtype, device=x.device), []
        out = torch.empty_like(rows)
        for e, (first, last) in enumerate(zip(runs, runs[1:])):
            if first == last:
                saved.append(None)
                continue
            r, h = rows[first:last], hidden[first:last]
            if self.gated:
                F = self.W2.shape[1]
                W, b = self.W1[e], self.b1[e]
                gate = ops.gemm_bias_act(r, W[:, :F], b[:F], act=self.act)
                ops.gemm_bias_act(r, W[:, F:], b[F:], C=h).mul_(gate)
                saved.append(None)
            else:
                saved.append(ops.gemm_bias_act(r, self.W1[e], self.b1[e], act=self.act, C=h, return_z=True)[1])
            ops.gemm_bias_act(h, self.W2[e], self.b2[e], C=out[first:last])
        self._saved = x, ids, weights, positions, offsets, runs, rows, hidden, saved, out
        return ops.moe_combine(out, positions, weights)

    def backward(self, dy):
        """Gradients of x and of the parameters (by name) for dy, after forward_sorted (which forward calls for more than 64
        tokens) of experts that are not gated."""
        if self.gated:
            raise NotImplementedError("gated experts have no backward pass")
        if self._saved is None:
            raise RuntimeError("backward needs forward_sorted before it: forward of up to 64 tokens keeps nothing")
        x, ids, weights, positions, offsets, runs, rows, hidden, saved, out = self._saved
        dout, dweights = ops.moe_combine_backward(dy, out, positions, offsets, weights)
        drows = torch.zeros_like(rows)
        g = {n: torch.zeros_like(getattr(self, n)) for n in ("Wr", "W1", "b1", "W2", "b2")}
        for e, (first, last) in enumerate(zip(runs, runs[1:])):
            if first == last:
                continue
            s = slice(first, last)
            dh = ops.gemm_bias_act_backward(dout[s], hidden[s], self.W2[e], dB=g["W2"][e], dbias=g["b2"][e])[0]
            ops.gemm_bias_act_backward(dh, rows[s], self.W1[e], saved[e], act=self.act, dA=drows[s], dB=g["W1"][e],
                                       dbias=g["b1"][e])
        dx = ops.moe_combine(drows, positions)
        # The router: softmax over the chosen logits.
        dbest = weights * (dweights - (weights * dweights).sum(1, keepdim=True))
        dlogits = torch.zeros(x.shape[0], self.Wr.shape[1], device=x.device)
        dlogits.scatter_(1, ids.clamp(min=0), torch.where(ids >= 0, dbest, 0.0))
        g["Wr"] = x.float().t() @ dlogits
        g["x"] = (dx.float() + dlogits @ self.Wr.t()).to(x.dtype)
        return g


class NormedFeedForward:
    """x + scale * gate * norm(block(norm(x) * pre)) * post, and the norm of that for the next block."""

    def __init__(self, D, F, act="gelu", scale=1.0, eps=1e-6, seed=0):
        self.block, self.scale, self.eps = FeedForward(D, F, act=act, seed=seed), scale, eps
        self.pre, self.post, self.next = (torch.ones(D, device="cuda") for _ in range(3))
        self.gate = torch.ones(1, D, device="cuda", dtype=torch.bfloat16)
        self._saved = None

    def forward(self, x):
        """(the residual stream, the next block's input)."""
        b = self.block
        _, h = ops.residual_norm(x, pre=self.pre, eps=self.eps)
        u, z = ops.gemm_bias_act(h, b.W1, b.b1, act=b.act, return_z=True)
        y = ops.gemm_bias_act(u, b.W2, b.b2)
        s, n = ops.residual_norm(y, x, post=self.post, gate=self.gate, scale=self.scale, pre=self.next, eps=self.eps)
        self._saved = x, h, u, z, y, s
        return s, n

    def backward(self, ds, dn):
        """Gradients of x and of the parameters, by name, for those of both outputs."""
        b = self.block
        x, h, u, z, y, s = self._saved
        dy, dx, dpost, dgate, dnext = ops.residual_norm_backward(ds, dn, y, s, post=self.post, gate=self.gate,
                                                                 scale=self.scale, pre=self.next, eps=self.eps)
        du, dW2, db2 = ops.gemm_bias_act_backward(dy, u, b.W2)
        dh, dW1, db1 = ops.gemm_bias_act_backward(du, h, b.W1, z, act=b.act)
        # x is the sum and the first norm's input at once.
        _, dx, _, _, dpre = ops.residual_norm_backward(dx, dh, None, x, pre=self.pre, eps=self.eps,
                                                       needs=(False, True, False, False, True))
        return {"x": dx, "pre": dpre, "post": dpost, "gate": dgate, "next": dnext, "W1": dW1, "b1": db1, "W2": dW2,
                "b2": db2}


class FeedForward4Bit:
    """A FeedForward's forward pass without dropout, weights and activations in 4 bits."""

    def __init__(self, block):
        self.act, self.b1, self.b2 = block.act, block.b1, block.b2
        self.W1, self.W2 = (ops.quantize_mxfp4(w, transposed=True) for w in (block.W1, block.W2))

    def forward(self, x):
        h = ops.gemm_mxfp4(ops.quantize_mxfp4(x), self.W1, self.b1, act=self.act)
        return ops.gemm_mxfp4(ops.quantize_mxfp4(h), self.W2, self.b2, residual=x)


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


def example_forms(T=512, D=1024, F=4096):
    """A step of the normed block and of the experts with sorted rows, and the dense block served in 4 bits: outputs
    and gradients of x by name."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x, dy = (torch.randn((T, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    normed, experts = NormedFeedForward(D, F, seed=8), ExpertFeedForward(D, F, experts=8, seed=9)
    out = {"normed": normed.forward(x)[0], "normed gradient": normed.backward(dy, dy)["x"],
           "experts": experts.forward(x), "experts' gradient": experts.backward(dy)["x"],
           "4 bits": FeedForward4Bit(FeedForward(D, F, seed=10)).forward(x)}
    check_device()
    return out


if __name__ == "__main__":
    losses, y = example()
    print("loss %.4f -> %.4f over %d steps; one token through experts: %s"
          % (losses[0], losses[-1], len(losses), list(y.shape)))
    print("; ".join("%s %s" % (n, list(t.shape)) for n, t in example_forms().items()))
