"""Limits of the step's operators that hold only where their reason does."""

import pytest

from cross_rank_collective_amd import step as S
from tests.test_step_cpu import BF16, F32, INVALID, NONE, OK, UNSUPPORTED, ffngrad, rows


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_slopes_alone_have_no_widest_row(dtype):
    """The limits are those of matrices that products read: without products there
    are none."""
    wide = S.PTORED_FFN_MAX_PITCH // (4 if dtype == F32 else 2) + 8
    alone = dict(F=wide, dt=dtype, x=NONE, w_gate=NONE, w_up=NONE, dx=NONE, dw_gate=NONE, dw_up=NONE,
                 **{k: rows(n, wide) for n, k in enumerate(("dy", "gate", "up", "dgate", "dup"))})
    assert ffngrad(T=0, **alone) == OK
    # with rows (and nothing launched here: half an element off is found later)
    assert ffngrad(T=2, **{**alone, "dy": rows(0, wide, 1)}) == INVALID
    narrow = {k: rows(n, wide) for n, k in enumerate(("dy", "gate", "up", "dgate", "dup"))}
    assert ffngrad(T=2, **{**alone, "F": 16, **narrow, "dy": rows(0, wide, 1)}) == INVALID
    # a product that reads them
    assert ffngrad(T=2, **{**alone, "dw_up": rows(11, 8), "x": rows(6, 8)}) == UNSUPPORTED
    assert ffngrad(T=2, **{**alone, "F": 16, **narrow, "dw_up": rows(11, 8), "x": rows(6, 8)}) == UNSUPPORTED
    assert ffngrad(T=2, **{**alone, "F": 1 << 60, "dy": rows(0, 1), "D": 0}) == INVALID  # a pitch below the columns
