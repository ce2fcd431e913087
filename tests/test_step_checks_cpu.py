"""That the checks of ``test_step_kernels_gpu.py`` tell products of fewer bits from
those of binary32: mistakes planted in products made here, on the CPU."""

import pytest
import torch

from tests.test_step_kernels_gpu import apart, same

PAIRS = [(0, 0), (0, 1), (1, 0), (0, 2), (2, 0), (1, 1)]


def pieces(v):
    """float32 as the exact sum of three bfloat16, truncated."""
    out = []
    for _ in range(3):
        p = (v.view(torch.int32) & -65536).view(torch.float32)
        out.append(p.double())
        v = v - p
    return out


def product(a, b, pairs):
    x, y = pieces(a), pieces(b)
    return sum(x[i] @ y[j].t() for i, j in pairs).float()


def whole(gen, bits, *shape):
    return (2 * torch.randint(-(1 << bits) // 2, (1 << bits) // 2, shape, generator=gen) + 1).float()


def cases(gen):
    """(checks of one product each): of random numbers, and of one product a sum."""
    a, b = (torch.randn(60, 1000, generator=gen) for _ in range(2))
    yield lambda pairs: apart(product(a, b, pairs), a.double() @ b.double().t(), 1000, "random")
    for n, m in ((24, 0), (12, 12), (0, 24)):
        value = lambda k, *s: whole(gen, k - 1, *s) if k else 2.0 ** torch.randint(-4, 5, s, generator=gen)  # noqa: E731
        p, q = torch.zeros(60, 100), value(m, 60, 100)
        p.scatter_(1, torch.randint(0, 100, (60, 1), generator=gen), value(n, 60, 1))
        yield lambda pairs, p=p, q=q: same(product(p, q, pairs), p, q, f"{n} by {m} bits")


def test_six_products_of_pieces_pass():
    for check in cases(torch.Generator().manual_seed(1)):
        check(PAIRS)


@pytest.mark.parametrize("left_out", PAIRS)
def test_a_product_of_pieces_that_is_left_out_is_found(left_out):
    found = 0
    for check in cases(torch.Generator().manual_seed(1)):
        try:
            check([p for p in PAIRS if p != left_out])
        except AssertionError:
            found += 1
    assert found >= 2 or (left_out == (1, 1) and found >= 1)


@pytest.mark.parametrize("dtype,running", [(torch.bfloat16, torch.float16), (torch.float16, torch.float16),
                                           (torch.bfloat16, torch.bfloat16)])
def test_running_sums_of_16_bits_are_found(dtype, running):
    gen = torch.Generator().manual_seed(2)
    a, b = whole(gen, 6, 40, 640).to(dtype), (whole(gen, 6, 50, 640) / 256).to(dtype)
    total = torch.zeros(40, 50)
    for k in range(0, 640, 64):
        total = (total + a[:, k:k + 64].float() @ b[:, k:k + 64].float().t()).to(running).float()
    same((a.double() @ b.double().t()).to(dtype), a, b, "as it should be")
    with pytest.raises(AssertionError, match="elements"):
        same(total.to(dtype), a, b, "running sums")
