"""Outputs that the operators make are PyTorch's allocations to whoever watches those, dispatch modes and the profiler.  Results
are the same either way, and with deterministic algorithms asked for."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from test_gpu_block_operators import gbr, normal, rng  # noqa: F401  (gbr: the fixture)

pytestmark = pytest.mark.gpu
F32 = torch.float32


def calls(gbr):  # noqa: F811
    """(name, call, number of outputs) of the operators that make outputs."""
    g = rng(1)
    X, Y, w = normal(g, (40, 64)), normal(g, (40, 64)), 1 + normal(g, (64,), 0.1, F32)
    W, b = normal(g, (64, 64)), normal(g, (64,), 0.1, F32)
    W1, W2, Wr = normal(g, (4, 64, 64), 0.1), normal(g, (4, 64, 64), 0.1), normal(g, (64, 4), 1.0, F32)
    ids = torch.randint(0, 4, (40, 2), generator=g, device="cuda")
    p, o = gbr.moe_sort(ids, 4)
    k = torch.rand((40, 2), generator=g, device="cuda")
    rows = gbr.moe_dispatch(X, p, o)
    Q = gbr.quantize_mxfp4(X)
    return [
        ("dropout_add", lambda: [gbr.dropout_add(X, Y, p=0.25, seed=3)], 1),
        ("gemm_bias_act", lambda: gbr.gemm_bias_act(X, W, b, act="gelu", return_z=True), 2),
        ("gemm_bias_act_backward", lambda: gbr.gemm_bias_act_backward(Y, X, W), 3),
        ("moe_layer", lambda: [gbr.moe_layer(X, Wr, W1, None, W2, None)], 1),
        ("residual_norm", lambda: gbr.residual_norm(X, Y, post=w, pre=w), 2),
        ("residual_norm_backward", lambda: gbr.residual_norm_backward(Y, X, X, Y, post=w, gate=X[:1], pre=w), 5),
        ("moe_sort", lambda: gbr.moe_sort(ids, 4), 2),
        ("moe_dispatch", lambda: [gbr.moe_dispatch(X, p, o)], 1),
        ("moe_combine", lambda: [gbr.moe_combine(rows, p, k, residual=X)], 1),
        ("moe_combine_backward", lambda: gbr.moe_combine_backward(Y, rows, p, o, k), 2),
        ("quantize_mxfp4", lambda: gbr.quantize_mxfp4(X)[:2], 2),
        ("dequantize_mxfp4", lambda: [gbr.dequantize_mxfp4(Q)], 1),
        ("gemm_mxfp4", lambda: [gbr.gemm_mxfp4(Q, Q)], 1),
    ]


class Watch(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.seen = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if func.overloadpacket is torch.ops.aten.empty:
            self.seen.append(tuple(args[0]))
        return func(*args, **(kwargs or {}))


def test_a_dispatch_mode_sees_them(gbr):  # noqa: F811
    for name, call, outputs in calls(gbr):
        want = call()
        with Watch() as watch:
            got = call()
        assert watch.seen == [tuple(t.shape) for t in got] and len(got) == outputs, name
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    gbr.check_device()


def test_the_profiler_sees_them(gbr):  # noqa: F811
    for name, call, outputs in calls(gbr):
        with torch.autograd.profiler.profile(use_cpu=True) as prof:
            call()
        assert sum(e.name == "aten::empty" for e in prof.function_events) == outputs, name
    gbr.check_device()


def test_deterministic_algorithms_change_no_result(gbr):  # noqa: F811
    before = torch.are_deterministic_algorithms_enabled()
    for name, call, _ in calls(gbr):
        want = call()
        torch.use_deterministic_algorithms(True)
        try:
            got = call()
        finally:
            torch.use_deterministic_algorithms(before)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    gbr.check_device()


class Elsewhere(TorchDispatchMode):
    """Gives memory that is not what was asked for."""
    def __init__(self, **how):
        super().__init__()
        self.how = how

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        kwargs = dict(kwargs or {})
        if func.overloadpacket is torch.ops.aten.empty:
            kwargs.update(self.how)
        return func(*args, **kwargs)


def test_a_mode_that_gives_something_else_is_refused(gbr):  # noqa: F811
    """Before its address goes to a kernel."""
    todo = calls(gbr)
    before = gbr.launch_count()
    for how in (dict(device=torch.device("cpu")), dict(device=torch.device("meta")), dict(dtype=torch.float64)):
        for name, call, _ in todo:
            with Elsewhere(**how), pytest.raises((ValueError, TypeError)):
                call()
    assert gbr.launch_count() == before
    gbr.check_device()
