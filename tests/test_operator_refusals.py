"""The feed-forward operators' checks of arguments (no GPU: every call here is
refused on the host before anything is launched), and the generator of their
dropout mask against its published test vectors."""
import ctypes

import pytest
import torch

import ffn_reference as ref

INVALID, UNSUPPORTED, ALIGN = 1, 2, 3
BASE = 0x7f0000000000          # never dereferenced


@pytest.fixture(scope="module")
def lib():
    import mbarrier_gemm_pipelines_gb300 as gbr
    gbr.build()
    return gbr.lib()


def mb(n):
    return BASE + n * (1 << 20)


def forward(lib, **kw):
    a = dict(A=mb(0), lda=64, B=mb(1), ldb=48, bias=mb(2), R=None, ldr=0, C=mb(3), ldc=48, Z=None, ldz=0,
             M=32, N=48, K=64, dtype=2, act=1, p=0.0, seed=0, offset=0, stream=None)
    a.update(kw)
    return lib.gemm_bias_act(*a.values())


def backward(lib, **kw):
    a = dict(dC=mb(0), lddc=48, A=mb(1), lda=64, B=mb(2), ldb=48, Z=mb(3), ldz=48, dA=mb(4), ldda=64, dB=mb(5),
             lddb=48, dbias=mb(6), M=32, N=48, K=64, dtype=2, act=1, p=0.0, seed=0, offset=0, stream=None)
    a.update(kw)
    return lib.gemm_bias_act_backward(*a.values())


def dropout(lib, **kw):
    a = dict(X=mb(0), ldx=64, R=None, ldr=0, Y=mb(1), ldy=64, rows=32, cols=64, dtype=2, p=0.5, seed=0, offset=0,
             stream=None)
    a.update(kw)
    return lib.dropout_add(*a.values())


def moe(lib, **kw):
    a = dict(X=mb(0), Wr=mb(1), W1=mb(2), b1=None, W2=mb(3), b2=None, Y=mb(4), ids=None, weights=None, T=4, D=64,
             F=128, E=4, top_k=2, act=1, gated=0, dtype=2, stream=None)
    a.update(kw)
    return lib.moe_layer(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=0), UNSUPPORTED), (dict(dtype=1), UNSUPPORTED), (dict(act=5), INVALID), (dict(act=-1), INVALID),
    (dict(p=-0.1), INVALID), (dict(p=1.5), INVALID), (dict(p=float("nan")), INVALID),
    (dict(M=-1), INVALID), (dict(N=1 << 31), INVALID), (dict(K=1 << 31), INVALID),
    (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(C=None), INVALID),
    (dict(lda=63), INVALID), (dict(ldc=47), INVALID), (dict(ldb=-48), INVALID),
    (dict(A=mb(0) + 1), ALIGN), (dict(bias=mb(2) + 2), ALIGN),
    (dict(C=mb(0)), INVALID), (dict(C=mb(1) + 96), INVALID), (dict(Z=mb(3), ldz=48), INVALID),
    (dict(R=mb(3), ldr=56), INVALID), (dict(R=mb(3) + 2, ldr=48), INVALID),
    (dict(Z=mb(2), ldz=48), INVALID),
])
def test_forward(lib, kw, code):
    assert forward(lib, **kw) == code
    assert lib.gbr_last_error() != b""


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=1), UNSUPPORTED), (dict(act=7), INVALID), (dict(p=2.0), INVALID), (dict(K=-1), INVALID),
    (dict(dC=None), INVALID), (dict(Z=None), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID),
    (dict(dA=mb(0)), INVALID), (dict(dB=mb(4)), INVALID), (dict(dbias=mb(5)), INVALID),
    (dict(ldda=63), INVALID), (dict(dbias=mb(6) + 2), ALIGN),
])
def test_backward(lib, kw, code):
    assert backward(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), UNSUPPORTED), (dict(p=-1e-9), INVALID), (dict(rows=-1), INVALID), (dict(X=None), INVALID),
    (dict(Y=None), INVALID), (dict(ldy=63), INVALID), (dict(X=mb(0) + 1), ALIGN), (dict(Y=mb(0) + 2), INVALID),
    (dict(Y=mb(0), ldy=65), INVALID), (dict(R=mb(1), ldr=128), INVALID),
    (dict(dtype=0, X=mb(0) + 2), ALIGN),
])
def test_dropout(lib, kw, code):
    assert dropout(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=0), UNSUPPORTED), (dict(act=9), INVALID), (dict(gated=2), INVALID), (dict(T=65), INVALID),
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(E=257), INVALID), (dict(top_k=0), INVALID),
    (dict(top_k=5), INVALID), (dict(E=64, top_k=9), INVALID), (dict(D=0), INVALID), (dict(F=0), INVALID),
    (dict(D=60), ALIGN), (dict(F=100), ALIGN), (dict(X=mb(0) + 8), ALIGN), (dict(W2=mb(3) + 2), ALIGN),
    (dict(Wr=None), INVALID), (dict(W1=None), INVALID), (dict(Y=mb(0)), INVALID), (dict(ids=mb(4)), INVALID),
    (dict(ids=mb(5), weights=mb(5)), INVALID), (dict(F=1 << 30), INVALID),
])
def test_moe(lib, kw, code):
    assert moe(lib, **kw) == code


def test_empty_calls_launch_nothing(lib):
    assert forward(lib, M=0) == 0 and forward(lib, N=0) == 0
    assert dropout(lib, rows=0) == 0 and dropout(lib, cols=0) == 0
    assert moe(lib, T=0) == 0
    assert backward(lib, dA=None, dB=None, dbias=None) == 0


def test_binding_refuses_cpu_tensors(lib):
    import mbarrier_gemm_pipelines_gb300 as gbr
    a = torch.zeros(8, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        gbr.gemm_bias_act(a, a)
    with pytest.raises(ValueError):
        gbr.gemm_bias_act_backward(a, a, a)
    with pytest.raises(ValueError):
        gbr.dropout_add(a)
    with pytest.raises(ValueError):
        gbr.moe_layer(a, a.float(), a[None], None, a[None], None, top_k=1)
    with pytest.raises(TypeError):
        gbr.dropout_add(a.half())


def test_binding_refuses_other_objects(lib):
    import mbarrier_gemm_pipelines_gb300 as gbr
    for bad in (None, 1, [[1.0]], "A"):
        with pytest.raises(TypeError):
            gbr.gemm_bias_act(bad, bad)
        with pytest.raises(TypeError):
            gbr.gemm_bias_act_backward(bad, bad, bad)
        with pytest.raises(TypeError):
            gbr.dropout_add(bad)
        with pytest.raises(TypeError):
            gbr.moe_layer(bad, bad, bad, None, bad, None)


def test_binding_missing_build(lib, monkeypatch, tmp_path):
    """Without its compiled part the binding raises; it has nothing to fall back to."""
    from mbarrier_gemm_pipelines_gb300 import _build, _operators
    monkeypatch.setattr(_operators, "_ext", None)
    monkeypatch.setattr(_build, "EXT_PATH", str(tmp_path / "absent.so"))
    with pytest.raises(RuntimeError, match="not built"):
        _operators.dropout_add(torch.zeros(2, 2))


@pytest.mark.parametrize("counter,key,out", [
    ((0,) * 4, (0,) * 2, (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_generator_vectors(counter, key, out):
    """The reference generator against the vectors published with the method."""
    assert tuple(ref.philox4x32_10(counter, key)) == out


def test_mask_is_the_generators():
    keep, scale = ref.keep_mask(3, 21, 0.25, (7 << 32) | 5, (9 << 32) | 11)
    for r in range(3):
        for c in range(21):
            w = ref.philox4x32_10((c // 8, r, 11, 9), (5, 7))[c % 8 // 2]
            assert bool(keep[r, c]) == ((w >> 16 if c % 2 else w & 0xFFFF) >= 16384)
    assert scale == 65536 / 49152
