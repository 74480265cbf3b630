"""More of the feed-forward operators' paths on the GPU: the gradients' products in one grid and one after the other."""
import math
import random

import pytest
import torch

import ffn_reference as ref
from gpu_helpers import load_library, require_gpu
from test_gpu_operators import BF, TWO, close, normal, rng

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
