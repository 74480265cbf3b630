"""Scale and eps of the norms that fp32 does not hold (no GPU: refused on the host, or empty)."""
import pytest

import test_block_refusals as refusals
from test_block_refusals import INVALID, lib  # noqa: F401  (lib: the fixture)


@pytest.mark.parametrize("call", [refusals.norm, refusals.norm_backward])
@pytest.mark.parametrize("kw", [dict(scale=1e39), dict(scale=-1e300), dict(eps=1e39), dict(eps=1e-60), dict(eps=5e-324)])
def test_beyond_fp32(lib, call, kw):  # noqa: F811
    assert call(lib, **kw) == INVALID
    assert b"fp32" in lib.gbr_last_error()


@pytest.mark.parametrize("kw", [dict(scale=3e38), dict(scale=-3e38), dict(scale=0.0), dict(scale=1e-60), dict(eps=0.0),
                                dict(eps=3e38), dict(eps=1e-44)])
def test_within_fp32(lib, kw):  # noqa: F811
    """Accepted; without columns nothing is launched."""
    assert refusals.norm(lib, cols=0, **kw) == 0 and refusals.norm_backward(lib, cols=0, **kw) == 0
