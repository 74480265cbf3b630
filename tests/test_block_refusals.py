"""Checks of arguments of the operators around a feed-forward block (no GPU: every call here is refused on the host, or
empty, before anything is launched)."""
import pytest
import torch

INVALID, UNSUPPORTED, ALIGN = 1, 2, 3
BASE = 0x7f0000000000          # never dereferenced


@pytest.fixture(scope="module")
def lib():
    import mbarrier_gemm_pipelines_gb300 as gbr
    gbr.build()
    return gbr.lib()


def mb(n):
    return BASE + n * (1 << 20)


def norm(lib, **kw):
    a = dict(X=mb(0), ldx=64, R=mb(1), ldr=64, post=mb(2), gate=mb(3), ldg=64, gates=4, scale=1.0, pre=mb(4), eps=1e-6,
             S=mb(5), lds=64, H=mb(6), ldh=64, rows=32, cols=64, dtype=2, stream=None)
    a.update(kw)
    return lib.residual_norm(*a.values())


def norm_backward(lib, **kw):
    a = dict(dS=mb(0), ldds=64, dH=mb(1), lddh=64, X=mb(2), ldx=64, S=mb(3), lds=64, post=mb(4), gate=mb(5), ldg=64,
             gates=4, scale=1.0, pre=mb(6), eps=1e-6, dX=mb(7), lddx=64, dR=mb(8), lddr=64, dpost=mb(9), dgate=mb(10),
             lddg=64, dpre=mb(11), rows=32, cols=64, dtype=2, stream=None)
    a.update(kw)
    return lib.residual_norm_backward(*a.values())


def sort(lib, **kw):
    a = dict(ids=mb(0), choices=64, E=8, positions=mb(1), offsets=mb(2), stream=None)
    a.update(kw)
    return lib.moe_sort(*a.values())


def dispatch(lib, **kw):
    a = dict(X=mb(0), ldx=64, positions=mb(1), offsets=mb(2), E=8, Xs=mb(3), ldxs=64, T=32, k=2, D=64, dtype=2, stream=None)
    a.update(kw)
    return lib.moe_dispatch(*a.values())


def combine(lib, **kw):
    a = dict(Ys=mb(0), ldys=64, rows=64, positions=mb(1), weights=mb(2), R=mb(3), ldr=64, Y=mb(4), ldy=64, T=32, k=2, D=64,
             dtype=2, stream=None)
    a.update(kw)
    return lib.moe_combine(*a.values())


def combine_backward(lib, **kw):
    a = dict(dY=mb(0), lddy=64, Ys=mb(1), ldys=64, positions=mb(2), offsets=mb(3), E=8, weights=mb(4), dYs=mb(5), lddys=64,
             dw=mb(6), T=32, k=2, D=64, dtype=2, stream=None)
    a.update(kw)
    return lib.moe_combine_backward(*a.values())


def quantize(lib, **kw):
    a = dict(X=mb(0), ldx=64, data=mb(1), scales=mb(2), rows=32, cols=64, transposed=0, dtype=2, stream=None)
    a.update(kw)
    return lib.quantize_mxfp4(*a.values())


def dequantize(lib, **kw):
    a = dict(data=mb(0), scales=mb(1), X=mb(2), ldx=64, rows=32, cols=64, dtype=2, stream=None)
    a.update(kw)
    return lib.dequantize_mxfp4(*a.values())


def gemm(lib, **kw):
    a = dict(A=mb(0), As=mb(1), B=mb(2), Bs=mb(3), bias=mb(4), R=None, ldr=0, C=mb(5), ldc=48, M=32, N=48, K=64, act=1,
             stream=None)
    a.update(kw)
    return lib.gemm_mxfp4(*a.values())


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("call,kw,code", [
    (norm, dict(dtype=3), UNSUPPORTED), (norm, dict(rows=-1), INVALID), (norm, dict(cols=1 << 31), INVALID),
    (norm, dict(gates=5), INVALID), (norm, dict(gates=0), INVALID), (norm, dict(gates=-4), INVALID),
    (norm, dict(eps=-1.0), INVALID), (norm, dict(eps=NAN), INVALID), (norm, dict(eps=INF), INVALID),
    (norm, dict(scale=NAN), INVALID), (norm, dict(scale=INF), INVALID), (norm, dict(X=None), INVALID),
    (norm, dict(pre=None), INVALID), (norm, dict(H=None), INVALID), (norm, dict(ldx=63), INVALID),
    (norm, dict(lds=-64), INVALID), (norm, dict(X=mb(0) + 1), ALIGN), (norm, dict(post=mb(2) + 2), ALIGN),
    (norm, dict(S=mb(6)), INVALID), (norm, dict(S=mb(1) + 2), INVALID), (norm, dict(S=mb(1), lds=72), INVALID),
    (norm, dict(H=mb(3)), INVALID), (norm, dict(S=mb(4)), INVALID),
    (norm_backward, dict(dtype=-1), UNSUPPORTED), (norm_backward, dict(gates=3), INVALID),
    (norm_backward, dict(eps=-1e-9), INVALID), (norm_backward, dict(dS=None, pre=None, dpre=None), INVALID),
    (norm_backward, dict(dH=None), INVALID), (norm_backward, dict(S=None), INVALID), (norm_backward, dict(X=None), INVALID),
    (norm_backward, dict(post=None), INVALID), (norm_backward, dict(gate=None), INVALID), (norm_backward, dict(pre=None), INVALID),
    (norm_backward, dict(dX=mb(0)), INVALID), (norm_backward, dict(dR=mb(0)), INVALID), (norm_backward, dict(dgate=mb(5)), INVALID),
    (norm_backward, dict(dpre=mb(9)), INVALID), (norm_backward, dict(lddx=10), INVALID), (norm_backward, dict(dpost=mb(9) + 1), ALIGN),
    (sort, dict(choices=-1), INVALID), (sort, dict(choices=1 << 31), INVALID), (sort, dict(E=0), INVALID),
    (sort, dict(E=1025), INVALID), (sort, dict(ids=None), INVALID), (sort, dict(offsets=None), INVALID),
    (sort, dict(positions=mb(0)), INVALID), (sort, dict(offsets=mb(1) + 252), INVALID), (sort, dict(ids=mb(0) + 4), ALIGN),
    (dispatch, dict(dtype=4), UNSUPPORTED), (dispatch, dict(T=1 << 30, k=2), INVALID), (dispatch, dict(E=0), INVALID),
    (dispatch, dict(X=None), INVALID), (dispatch, dict(offsets=None), INVALID), (dispatch, dict(Xs=mb(0)), INVALID),
    (dispatch, dict(ldxs=63), INVALID), (dispatch, dict(X=mb(0) + 1), ALIGN), (dispatch, dict(Xs=mb(1)), INVALID),
    (combine, dict(rows=-1), INVALID), (combine, dict(Ys=None), INVALID), (combine, dict(positions=None), INVALID),
    (combine, dict(Y=None), INVALID), (combine, dict(Y=mb(0)), INVALID), (combine, dict(Y=mb(3) + 2), INVALID),
    (combine, dict(Y=mb(3), ldy=72), INVALID), (combine, dict(dtype=9), UNSUPPORTED), (combine, dict(weights=mb(2) + 1), ALIGN),
    (combine_backward, dict(weights=None), INVALID), (combine_backward, dict(Ys=None), INVALID),
    (combine_backward, dict(offsets=None), INVALID), (combine_backward, dict(dYs=mb(1)), INVALID),
    (combine_backward, dict(dw=mb(4)), INVALID), (combine_backward, dict(E=2000), INVALID), (combine_backward, dict(k=-1), INVALID),
    (quantize, dict(dtype=7), UNSUPPORTED), (quantize, dict(transposed=2), INVALID), (quantize, dict(X=None), INVALID),
    (quantize, dict(data=mb(1) + 8), ALIGN), (quantize, dict(scales=mb(2) + 4), ALIGN), (quantize, dict(ldx=63), INVALID),
    (quantize, dict(data=mb(0)), INVALID), (quantize, dict(scales=mb(1)), INVALID), (quantize, dict(transposed=1, ldx=31), INVALID),
    (dequantize, dict(X=mb(0)), INVALID), (dequantize, dict(data=None), INVALID), (dequantize, dict(scales=mb(1) + 1), ALIGN),
    (gemm, dict(act=5), INVALID), (gemm, dict(M=-1), INVALID), (gemm, dict(K=1 << 31), INVALID), (gemm, dict(A=None), INVALID),
    (gemm, dict(Bs=None), INVALID), (gemm, dict(C=None), INVALID), (gemm, dict(A=mb(0) + 8), ALIGN),
    (gemm, dict(Bs=mb(3) + 1), ALIGN), (gemm, dict(C=mb(0)), INVALID), (gemm, dict(C=mb(3)), INVALID),
    (gemm, dict(C=mb(4)), INVALID), (gemm, dict(ldc=47), INVALID), (gemm, dict(C=mb(5) + 1), ALIGN),
    (gemm, dict(R=mb(5), ldr=56), INVALID), (gemm, dict(R=mb(5) + 2, ldr=48), INVALID),
])
def test_refused(lib, call, kw, code):
    assert call(lib, **kw) == code
    assert lib.gbr_last_error() != b""


@pytest.mark.parametrize("call,kw", [
    (norm, dict(cols=1 << 30)), (norm_backward, dict(cols=(1 << 31) - 1)), (dispatch, dict(D=1 << 30)), (combine, dict(D=1 << 30)),
    (combine_backward, dict(D=(1 << 31) - 1)), (quantize, dict(cols=1 << 30)), (quantize, dict(rows=1 << 30, transposed=1)),
    (dequantize, dict(cols=(1 << 31) - 1)), (gemm, dict(M=1 << 30)), (gemm, dict(N=(1 << 31) - 1)), (gemm, dict(K=1 << 30)),
])
def test_rows_longer_than_kernels_count_are_refused(lib, call, kw):
    assert call(lib, **kw) == INVALID
    assert b"2^30" in lib.gbr_last_error()


def test_empty_calls_launch_nothing(lib):
    before = lib.gbr_launch_count()
    assert norm(lib, rows=0, gates=0) == 0 and norm(lib, cols=0) == 0 and norm(lib, S=None, H=None) == 0
    assert norm_backward(lib, cols=0) == 0
    assert norm_backward(lib, dX=None, dR=None, dpost=None, dgate=None, dpre=None) == 0
    assert dispatch(lib, T=0) == 0 and dispatch(lib, k=0) == 0 and dispatch(lib, D=0) == 0
    assert combine(lib, T=0) == 0 and combine(lib, D=0) == 0
    assert combine_backward(lib, T=0) == 0 and combine_backward(lib, dYs=None, dw=None) == 0
    assert quantize(lib, rows=0) == 0 and quantize(lib, cols=0) == 0 and dequantize(lib, rows=0) == 0
    assert gemm(lib, M=0) == 0 and gemm(lib, N=0) == 0
    assert lib.gbr_launch_count() == before


def test_sizes_of_4_bit_matrices(lib):
    assert lib.mxfp4_data_bytes(3, 33) == 3 * 2 * 16 and lib.mxfp4_scale_bytes(129, 129) == 2 * 2 * 512
    assert lib.mxfp4_data_bytes(0, 7) == 0 and lib.mxfp4_scale_bytes(5, 0) == 0
    assert lib.mxfp4_data_bytes(-1, 7) == -1 and lib.mxfp4_scale_bytes(5, 1 << 31) == -1
    assert lib.mxfp4_data_bytes((1 << 31) - 1, (1 << 31) - 1) == ((1 << 31) - 1) * (1 << 26) * 16


def every(gbr, a, f, i):
    """Each operator with bf16 a, fp32 f and int i in the places of its tensors."""
    Q = gbr.Mxfp4(i.byte(), i.byte(), 32)
    return [
        (lambda: gbr.residual_norm(a, a)), (lambda: gbr.residual_norm_backward(a, None, None, None)),
        (lambda: gbr.moe_sort(i, 4)), (lambda: gbr.moe_dispatch(a, i.int(), i.int()[0])),
        (lambda: gbr.moe_combine(a, i.int())), (lambda: gbr.moe_combine_backward(a, a, i.int(), i.int()[0], f)),
        (lambda: gbr.quantize_mxfp4(a)), (lambda: gbr.dequantize_mxfp4(Q)), (lambda: gbr.gemm_mxfp4(Q, Q)),
    ]


def test_binding_refuses_cpu_tensors(lib):
    import mbarrier_gemm_pipelines_gb300 as gbr
    a = torch.zeros(8, 8)
    for call in every(gbr, a.bfloat16(), a, a.long()):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gbr.residual_norm(a.half()), lambda: gbr.moe_dispatch(a.half(), a.int(), a.int()[0]),
                 lambda: gbr.moe_combine(a.double(), a.int()), lambda: gbr.quantize_mxfp4(a.half())):
        with pytest.raises(TypeError):
            call()


def test_binding_refuses_other_objects(lib):
    import mbarrier_gemm_pipelines_gb300 as gbr
    for bad in (None, 1, [[1.0]], "A"):
        Q = gbr.Mxfp4(bad, bad, 32)
        for call in (lambda: gbr.residual_norm(bad), lambda: gbr.moe_sort(bad, 4), lambda: gbr.moe_dispatch(bad, bad, bad),
                     lambda: gbr.moe_combine(bad, bad), lambda: gbr.moe_combine_backward(bad, bad, bad, bad, bad),
                     lambda: gbr.quantize_mxfp4(bad), lambda: gbr.dequantize_mxfp4(Q), lambda: gbr.gemm_mxfp4(Q, Q)):
            with pytest.raises(TypeError):
                call()
    with pytest.raises(ValueError):
        gbr.residual_norm_backward(None, None, None, None)
