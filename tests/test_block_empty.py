"""Calls of the operators around a block whose matrices have no columns or no rows (no GPU: nothing is launched)."""
import test_block_refusals as refusals
from test_block_refusals import INVALID, lib  # noqa: F401  (lib: the fixture)


def test_gradient_rows_without_columns_need_no_offsets(lib):  # noqa: F811
    """No element of dYs is written then, so the offsets, which say where its zero rows begin, are not read."""
    before = lib.gbr_launch_count()
    assert refusals.combine_backward(lib, D=0, offsets=None, dw=None) == 0
    assert refusals.combine_backward(lib, D=0, dw=None) == 0
    assert lib.gbr_launch_count() == before
    assert refusals.combine_backward(lib, offsets=None) == INVALID
    assert refusals.combine_backward(lib, offsets=None, dw=None) == INVALID
