"""The `stream` argument of the operators: the results, and whose memory the outputs are made from."""
import math

import pytest
import torch

from gpu_helpers import load_library, require_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def gbr():
    require_gpu()
    return load_library()


def owner(t):
    """Handle of the stream that PyTorch's allocator counts the memory of `t` to."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


def calls(gbr):
    """Every operator with outputs of its own, as functions of the stream."""
    g = torch.Generator(device="cuda").manual_seed(5)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    M, K, N, E = 300, 520, 1000, 4
    A, B, R, Z = normal(M, K).to(BF), normal(K, N, std=K ** -0.5).to(BF), normal(M, N).to(BF), normal(M, N).to(BF)
    bias, x3 = normal(N), normal(3, 5, 1000)
    X, Wr = normal(5, K).to(BF), normal(K, E)
    W1, W2 = normal(E, K, 264, std=K ** -0.5).to(BF), normal(E, 264, K, std=264 ** -0.5).to(BF)
    return [
        lambda s: list(gbr.gemm_bias_act(A, B, bias, residual=R, act="gelu", p=0.1, seed=1, return_z=True, stream=s)),
        lambda s: [gbr.gemm_bias_act(A[:3], B, bias, stream=s)],
        lambda s: list(gbr.gemm_bias_act_backward(R, A, B, Z, act="silu", p=0.1, stream=s)),
        lambda s: [gbr.dropout_add(R, Z, p=0.3, stream=s)],
        lambda s: [gbr.dropout_add(x3, p=0.3, stream=s)],
        lambda s: list(gbr.moe_layer(X, Wr, W1, None, W2, None, return_routing=True, stream=s)),
    ]


@pytest.mark.parametrize("how", ["stream", "handle"])
def test_outputs_belong_to_the_calls_stream(gbr, how):
    side = torch.cuda.Stream()
    for call in calls(gbr):
        want = call(None)
        torch.cuda.synchronize()
        got = call(side if how == "stream" else side.cuda_stream)
        side.synchronize()
        here = torch.cuda.current_stream().cuda_stream
        assert side.cuda_stream != here
        for g, w in zip(got, want):
            assert torch.equal(g, w)
            assert owner(w) == here and owner(g) == side.cuda_stream
        assert torch.cuda.current_stream().cuda_stream == here
    gbr.check_device()


@pytest.mark.parametrize("handle", [0, 1])
def test_null_stream_by_its_handles(gbr, handle):
    """0, and 1 (cudaStreamLegacy), from under another current stream."""
    side = torch.cuda.Stream()
    for call in calls(gbr):
        want = call(None)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = call(handle)
            assert torch.cuda.current_stream() == side
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w) and owner(g) == 0
    gbr.check_device()


def test_refused_calls_leave_the_current_stream(gbr):
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    A = torch.ones(16, 16, device="cuda", dtype=BF)
    for bad in (dict(p=1.5), dict(C=A[:3]), dict(C=A)):
        with pytest.raises((ValueError, gbr.GbrError)):
            gbr.gemm_bias_act(A, A, stream=side, **bad)
        assert torch.cuda.current_stream() == here
    with pytest.raises(AttributeError):
        gbr.gemm_bias_act(A, A, stream="0")


def test_given_outputs_on_another_stream(gbr):
    side = torch.cuda.Stream()
    A = torch.ones(32, 64, device="cuda", dtype=BF)
    B, C = torch.ones(64, 48, device="cuda", dtype=BF), torch.zeros(32, 48, device="cuda", dtype=BF)
    side.wait_stream(torch.cuda.current_stream())
    assert gbr.gemm_bias_act(A, B, C=C, stream=side) is C
    side.synchronize()
    assert (C == 64).all() and math.isclose(C.float().sum().item(), 32 * 48 * 64)


def test_self_tests_outputs(gbr):
    side = torch.cuda.Stream()
    A, B = torch.ones(64, 128, device="cuda", dtype=BF), torch.ones(128, 64, device="cuda", dtype=BF)
    torch.cuda.synchronize()
    # No such CTA: nothing is planted.
    assert owner(gbr.selftest_linear_skip_load(A, B, 100000, 0, 50_000_000, stream=side)) == side.cuda_stream
    side.synchronize()
    gbr.check_device()


@pytest.mark.parametrize("how", ["stream", "handle", "null"])
def test_older_operators_outputs(gbr, how):
    side = torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(6)
    A, B = torch.randn(300, 128, generator=g, device="cuda"), torch.randn(128, 264, generator=g, device="cuda")
    bias, src = torch.randn(264, generator=g, device="cuda"), torch.randn(100, 64, generator=g, device="cuda")
    W, b2, A16, B16 = B[None].repeat(2, 1, 1).to(BF), bias[None].repeat(2, 1), A.to(BF), B.to(BF)
    given, mine = {"stream": (side, side.cuda_stream), "handle": (side.cuda_stream, side.cuda_stream), "null": (0, 0)}[how]
    for call in (lambda s: gbr.gemm_bias_relu(A, B, bias, dtype="ffma", stream=s),
                 lambda s: gbr.gemm_bias_relu(A16, B16, bias, stream=s),
                 lambda s: gbr.gemm_bias_relu_grouped(A16, W, b2, [100, 200], stream=s),
                 lambda s: gbr.staged_copy(src, stream=s)):
        want = call(None)
        torch.cuda.synchronize()
        if how == "null":
            with torch.cuda.stream(side):
                got = call(given)
        else:
            got = call(given)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and owner(got) == mine
    gbr.check_device()
