"""The step's operators on the GPU at the ends of binary32's range."""

import pytest
import torch

import cross_rank_collective_amd as crc
from tests.block_reference import ROW, U
from tests.test_step_gpu import BF16, F32

pytestmark = pytest.mark.gpu


def layer_norm(x, bias):
    """mean, rstd and z of one row."""
    z, mean, rstd = torch.empty_like(x), *(torch.empty(x.shape[0], device="cuda") for _ in range(2))
    crc.layer_norm([], x, None, z, bias=bias, mean=mean, rstd=rstd)
    return mean, rstd, z


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [16, 200, 1001, 4096, 16381])
def test_layer_norm_sums_pass_the_range_both_ways(cols, dtype):
    """Partial sums of +inf and -inf, whose sum is a NaN that the row does not hold."""
    x = torch.full((2, cols), 3e38, dtype=dtype)
    x[:, cols // 2:] *= -1
    x[1] = x[1].flip(0)
    bias = torch.arange(cols, device="cuda", dtype=F32) / 256
    mean, rstd, z = layer_norm(x.cuda(), bias)
    want = x.double().mean(1)
    # each quotient by the columns and each addition rounds
    bound = U * (ROW + 2) * x.double().abs().mean(1)
    assert bool(((mean.cpu().double() - want).abs() <= bound).all()), mean
    assert bool((rstd == 0).all())  # the variance passes the range
    assert torch.equal(z, bias.to(dtype).expand(2, cols))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [16, 200, 1001, 4096, 16381])
def test_layer_norm_differences_pass_the_range(cols, dtype):
    """Elements further from the mean than binary32 reaches."""
    x = torch.full((2, cols), -3e38, dtype=dtype)
    x[:, 3::8] = 3e38
    x[1] *= -1
    bias = torch.arange(cols, device="cuda", dtype=F32) / 256
    mean, rstd, z = layer_norm(x.cuda(), bias)
    want = x.double().mean(1)
    bound = U * (ROW + 2) * x.double().abs().mean(1)
    assert bool(((mean.cpu().double() - want).abs() <= bound).all()), mean
    assert bool((rstd == 0).all())
    assert torch.equal(z, bias.to(dtype).expand(2, cols))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_norm_specials_among_large_elements(dtype):
    """What a row holds is not taken for a sum past the range."""
    x = torch.full((4, 1000), 3e38, dtype=dtype)
    x[:, 500:] *= -1
    x[0, 7], x[1, 7], x[2, 7] = float("nan"), float("inf"), -float("inf")
    x[3, 7], x[3, 8] = float("inf"), -float("inf")
    mean, rstd, z = layer_norm(x.cuda(), torch.zeros(1000, device="cuda"))
    assert bool(z.isnan().all()) and bool(rstd.isnan().all())
    assert bool(mean[[0, 3]].isnan().all()) and not bool(mean[1:3].isfinite().any())
