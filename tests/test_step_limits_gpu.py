"""The step's operators on the GPU past the limits that hold for products only."""

import pytest
import torch

import cross_rank_collective_amd as crc
from tests import step_reference as R
from tests.block_reference import close
from tests.test_step_gpu import BF16, F32, Room, put, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_slopes_of_the_widest_rows(dtype):
    wide = (1 << 22) // dtype.itemsize + 9
    dy, g, u = (rand(3, wide, seed=s, dtype=dtype) for s in (1, 2, 3))
    dg, du = Room(3, wide, dtype, 5, 1), Room(3, wide, dtype, 5, 1)
    crc.gated_ffn_backward(*(put(t, 5, 1) for t in (dy, g, u)), dg.t, du.t)
    want = R.gated_slopes(dy, g, u, "silu")
    close(dg.t, *want["dgate"], "dgate")
    close(du.t, *want["dup"], "dup")
    dg.check("dgate")
    du.check("dup")
