"""The self tests' operands are checked for shape before their addresses go to a kernel (no GPU: refused on the host)."""
import pytest
import torch


@pytest.fixture(scope="module")
def gbr():
    import mbarrier_gemm_pipelines_gb300 as gbr
    gbr.build()
    return gbr


def blocks(gbr, rows, columns):
    return gbr.Mxfp4(torch.zeros(rows, (columns + 31) // 32 * 16, dtype=torch.uint8),
                     torch.zeros((rows + 127) // 128, (columns + 127) // 128, 512, dtype=torch.uint8), columns)


def test_4_bit_operands(gbr):
    A, B = blocks(gbr, 20, 512), blocks(gbr, 300, 512)
    for a, b in ((A, blocks(gbr, 300, 256)), (blocks(gbr, 20, 1024), B), (A._replace(columns=2048), B),
                 (A, B._replace(scales=B.scales[:2])), (A._replace(scales=A.scales[:, :3]), B), (A, B._replace(data=B.data[0]))):
        with pytest.raises(ValueError, match="shape"):
            gbr.selftest_mxfp4_skip_load(a, b, 0, 0, 1000)
    with pytest.raises(ValueError, match="CUDA"):
        gbr.selftest_mxfp4_skip_load(A, B, 0, 0, 1000)


def test_linear_operands(gbr):
    A = torch.zeros(16, 64, dtype=torch.bfloat16)
    for rows in (32, 128):
        with pytest.raises(ValueError, match="shape"):
            gbr.selftest_linear_skip_load(A, torch.zeros(rows, 48, dtype=torch.bfloat16), 0, 0, 1000)


def test_expert_operands(gbr):
    D, F, E = 64, 128, 4
    good = dict(X=torch.zeros(3, D).bfloat16(), Wr=torch.zeros(D, E), W1=torch.zeros(E, D, F).bfloat16(),
                W2=torch.zeros(E, F, D).bfloat16())
    for name, shape in (("Wr", (D, E - 1)), ("W1", (E, D, F // 2)), ("W2", (E, F, D // 2)), ("X", (3, 2 * D))):
        with pytest.raises(ValueError, match="shape"):
            gbr.selftest_moe_skip_load(**dict(good, **{name: torch.zeros(shape).to(good[name].dtype)}), top_k=2, cta=0, item=0,
                                       limit_ns=1000)
