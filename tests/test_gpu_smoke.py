"""smoke() runs every operator of the package."""
import pytest

from gpu_helpers import load_library, require_gpu

pytestmark = pytest.mark.gpu

OPERATORS = ("gemm_bias_relu", "gemm_bias_relu_grouped", "gemm_bias_relu_host", "gemm_bias_relu_tf32_noalloc",
             "staged_copy", "gemm_bias_act", "gemm_bias_act_backward", "dropout_add", "moe_layer")


def test_smoke_runs_every_operator(monkeypatch, capsys):
    require_gpu()
    gbr = load_library()
    import __graft_entry__ as entry
    ran = set()

    def noted(name, fn):
        def call(*a, **kw):
            ran.add(name)
            return fn(*a, **kw)
        return call

    for name in OPERATORS:
        monkeypatch.setattr(gbr, name, noted(name, getattr(gbr, name)))
    entry.smoke()
    assert ran == set(OPERATORS)
    assert "smoke ok" in capsys.readouterr().out
