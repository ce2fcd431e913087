"""Every kernel of the feed-forward block's products on the GPU, at the sizes of
``step_sizes.py``: against 64-bit products, to the last bit where sums are exact in
binary32, and rows of NaN that stay alone."""

import math

import pytest
import torch

import cross_rank_collective_amd as crc
from tests import step_reference as R
from tests.block_reference import U
from tests.step_sizes import CASES
from tests.test_step_gpu import ACTS, BF16, F16, F32, Room

pytestmark = pytest.mark.gpu

RUNS = [(dtype, *case) for bits, *case in CASES for dtype in ([F32] if bits == 32 else [BF16, F16])]
IDS = ["-".join(str(v).replace("torch.", "") for v in r) for r in RUNS]


def close(got, want, bound, what):
    """As ``block_reference.close``, on the GPU: half a step of got's type and the bound."""
    t, g = got.dtype, got.double()
    tol = bound + torch.finfo(t).eps / 2 * (want.abs() + bound) + torch.finfo(t).tiny * torch.finfo(t).eps / 2
    assert bool(g.isfinite().all()), f"{what}: not finite"
    over = float(((g - want).abs() - tol).max())
    assert over <= 0, f"{what}: off by {over} more than the bound"


def apart(got, want, terms, what):
    """The relative distance of sums of `terms` products in binary32.

    Rounding a running sum moves it by at most U times itself; of terms of random
    signs the sum of j has the size of sqrt(j) of them, and the errors of all
    additions, independent as they are, that of U sqrt(terms^2 / 2) of them: U
    sqrt(terms / 2) of the whole.  Each product is rounded (U) or lacks the pieces
    below 2^-21 = 8 U of it, and the result is rounded (U).  Operands of 16 bits in
    place of 24 would leave some 2^-16 = 256 U."""
    far = float((got.double() - want).norm() / want.norm())
    assert far <= U * (math.sqrt(terms / 2) + 10), f"{what}: {far / U:.0f} U of {terms} terms"


class Data:
    """A call's matrices, every one in rows of its own buffer with `pad` elements behind."""

    def __init__(self, dtype, rows, cols, wide, pad, call, seed=0):
        self.dtype, self.pad, self.call = dtype, pad, call
        self.rows, self.cols, self.wide = rows, cols, wide
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)

    def put(self, value):
        return Room(*value.shape, self.dtype, self.pad, 0, value).t

    def normal(self, *shape, scale=1.0):
        return self.put(torch.randn(*shape, generator=self.gen, device="cuda") * scale)

    def whole(self, *shape, most, unit=1.0):
        """Odd whole numbers of up to `most`, times a power of two."""
        v = torch.randint(-(most + 1) // 2, most // 2 + 1, shape, generator=self.gen, device="cuda")
        return self.put((2 * v + 1).float() * unit)

    def room(self, *shape, dtype=None, value=None):
        return Room(*shape, dtype or self.dtype, self.pad, 0, value)

    def forward(self, x, wg, wu, act="silu"):
        out = [self.room(self.rows, self.wide) for _ in range(3)]
        crc.gated_ffn(x, wg, wu, out[0].t, activation=act, gate=out[1].t, up=out[2].t)
        return out

    def backward(self, dy, g, u, x, wg, wu, act="silu", dw_type=None, add=None):
        """{name: room}: dgate and dup, and what the call wants."""
        rows, cols, wide = self.rows, self.cols, self.wide
        out = {k: self.room(rows, wide) for k in ("dg", "du")}
        kw = {}
        if "i" in self.call:
            out["dx"] = self.room(rows, cols)
            kw.update(w_gate=wg, w_up=wu, dx=out["dx"].t)
        for k, name in (("g", "dw_gate"), ("u", "dw_up")):
            if k in self.call:
                out[name] = self.room(wide, cols, dtype=dw_type, value=add)
                kw.update({"x": x, name: out[name].t})
        crc.gated_ffn_backward(dy, g, u, out["dg"].t, out["du"].t, activation=act, accumulate=add is not None, **kw)
        return out

    def products(self, dg, du, x, wg, wu):
        """{name: (a, b, terms)}: what an output is the product a b^T of."""
        pairs = {}
        if "i" in self.call:
            pairs["dx"] = torch.cat([dg, du], 1), torch.cat([wg, wu], 0).t(), 2 * self.wide
        for k, name, d in (("g", "dw_gate", dg), ("u", "dw_up", du)):
            if k in self.call:
                pairs[name] = d.t(), x.t(), self.rows
        return pairs


@pytest.mark.parametrize("dtype,rows,cols,wide,pad,call", RUNS, ids=IDS)
def test_products(dtype, rows, cols, wide, pad, call):
    d = Data(dtype, rows, cols, wide, pad, call)
    exact = dtype != F32
    x, act = d.normal(rows, cols), ACTS[wide % 3]
    wg, wu = (d.normal(wide, cols, scale=cols ** -0.5) for _ in range(2))
    if call == "forward":
        want = R.gated_ffn(x, wg, wu, act)
        y, g, u = d.forward(x, wg, wu, act)
        for k, r in (("y", y), ("gate", g), ("up", u)):
            close(r.t, *want[k], k)
            if dtype == F32 and k != "y" and cols > 1:
                apart(r.t, want[k][0], cols, k)
            r.check(k)
        return
    dy, g, u = (d.normal(rows, wide) for _ in range(3))
    dw_type = F32 if rows % 2 else dtype
    add = None
    if wide % 2 == 0 and call != "i":
        add = torch.randn(wide, cols, generator=d.gen, device="cuda").to(dw_type)
    out = d.backward(dy, g, u, x, wg, wu, act, dw_type, add)
    want = R.gated_slopes(dy, g, u, act)
    close(out["dg"].t, *want["dgate"], "dgate")
    close(out["du"].t, *want["dup"], "dup")
    for k, (a, b, terms) in d.products(out["dg"].t, out["du"].t, x, wg, wu).items():
        value, bound = R.product(a, b, exact)
        if out[k].t.dtype == F32 and add is None and terms > 1:
            apart(out[k].t, value, terms, k)
        if add is not None and k != "dx":
            value, bound = value + add.double(), bound + U * (value.abs() + add.double().abs())
        close(out[k].t, value, bound, k)
    for k, r in out.items():
        r.check(k)


def same(got, a, b, what):
    """got is a b^T, rounded once."""
    want = (a.double() @ b.double().t()).to(got.dtype)
    assert bool(want.isfinite().all()) and bool((want != 0).any())
    off = (got != want).nonzero()
    assert off.numel() == 0, (f"{what}: {off.shape[0]} of {got.numel()} elements, the first at {off[0].tolist()}: "
                              f"{float(got[tuple(off[0])])!r}, want {float(want[tuple(off[0])])!r}")


@pytest.mark.parametrize("dtype,rows,cols,wide,pad,call", RUNS, ids=IDS)
def test_sums_that_are_exact(dtype, rows, cols, wide, pad, call):
    """Whole numbers whose products and running sums binary32 holds exactly, in any
    order: at most 127 x 127 a product, so that 8 times the size of a sum of 8192 of
    random signs, 127^2 / 3 sqrt(8192), is 2^22 (and of the gradients', 224 x 127 and
    16384, 2^23).  The outputs are the sums rounded once, to the bit.  16-bit types
    hold neither the products nor the sums."""
    d = Data(dtype, rows, cols, wide, pad, call, seed=1)
    most = 127 if dtype != F32 else 31
    unit = 2.0 ** -8  # keeps sums in f16's range
    x = d.whole(rows, cols, most=most)
    wg, wu = (d.whole(wide, cols, most=15 if call != "forward" else most, unit=unit) for _ in range(2))
    if call == "forward":
        _, g, u = d.forward(x, wg, wu)
        same(g.t, x, wg, "gate")
        same(u.t, x, wu, "up")
        return
    # f(32) = 32 and f'(32) = 1 to the bit
    dy, u = d.whole(rows, wide, most=7), d.whole(rows, wide, most=7)
    g = d.put(torch.full((rows, wide), 32.0, device="cuda"))
    x = d.put(x * unit)
    for dw_type in {dtype, F32}:
        out = d.backward(dy, g, u, x, wg, wu, dw_type=dw_type)
        assert torch.equal(out["dg"].t, dy * u) and torch.equal(out["du"].t, 32 * dy)
        for k, (a, b, _) in d.products(out["dg"].t, out["du"].t, x, wg, wu).items():
            same(out[k].t, a, b, k)


def one_each(d, rows, cols, values):
    """A matrix with one value a row, at columns all over."""
    t = torch.zeros(rows, cols, device="cuda")
    at = torch.randint(0, cols, (rows, 1), generator=d.gen, device="cuda")
    return d.put(t.scatter_(1, at, values))


@pytest.mark.parametrize("dtype,rows,cols,wide,pad,call", [r for r in RUNS if r[0] == F32],
                         ids=[i for r, i in zip(RUNS, IDS) if r[0] == F32])
def test_every_bit_of_float32_counts(dtype, rows, cols, wide, pad, call):
    """Sums of one product, exact in 24 bits: all 24 bits of one operand by a power of
    two of the other, either way round, and 12 bits of each."""
    d = Data(dtype, rows, cols, wide, pad, call, seed=2)
    bits = lambda n, *s: d.whole(*s, most=(1 << n) - 1)  # noqa: E731
    power = lambda *s: d.put(2.0 ** torch.randint(-4, 5, s, generator=d.gen, device="cuda"))  # noqa: E731
    if call == "forward":
        for n, m in ((24, 0), (12, 12), (0, 24)):
            x = one_each(d, rows, cols, bits(n, rows, 1) if n else power(rows, 1))
            wg, wu = (bits(m, wide, cols) if m else power(wide, cols) for _ in range(2))
            _, g, u = d.forward(x, wg, wu)
            same(g.t, x, wg, "gate")
            same(u.t, x, wu, "up")
        return
    g, ones = (d.put(torch.full((rows, wide), v, device="cuda")) for v in (32.0, 1.0))
    for n, m in ((24, 0), (12, 12), (0, 24)):
        wg, wu = (bits(m, wide, cols) if m else power(wide, cols) for _ in range(2))
        value = lambda *s: bits(n, *s) if n else power(*s)  # noqa: E731
        # the input's: one feature a token, of one of the two projections
        if "i" in call:
            dy, none = one_each(d, rows, wide, value(rows, 1)), d.put(0 * ones)
            alone = Data(dtype, rows, cols, wide, pad, "i")
            out = alone.backward(dy, g, none, None, wg, wu)  # u = 0: dgate = 0, dup = 32 dy
            same(out["dx"].t, out["du"].t, wu.t(), "dx by up")
            out = alone.backward(dy, none, ones, None, wg, wu)  # f(0) = 0, f'(0) = 1/2: dup = 0
            same(out["dx"].t, out["dg"].t, wg.t(), "dx by gate")
        # the weights': one token a feature
        x = bits(m, rows, cols) if m else power(rows, cols)
        dy = d.put(one_each(d, wide, rows, value(wide, 1)).t())
        for k in "gu":
            if k in call:
                out = Data(dtype, rows, cols, wide, pad, k).backward(dy, g, ones, x, wg, wu)
                name = "dw_gate" if k == "g" else "dw_up"
                same(out[name].t, out["dg" if k == "g" else "du"].t.t(), x.t(), name)


@pytest.mark.parametrize("dtype,rows,cols,wide,pad,call", RUNS, ids=IDS)
def test_what_is_not_finite_stays_in_its_row(dtype, rows, cols, wide, pad, call):
    d = Data(dtype, rows, cols, wide, pad, call, seed=3)
    x, dy = d.normal(rows, cols), d.normal(rows, wide)
    wg, wu = (d.normal(wide, cols, scale=cols ** -0.5) for _ in range(2))
    nan, inf = math.nan, math.inf
    if call == "forward":
        y = d.forward(x, wg, wu)[0].t.clone()
        x[0, -1], wg[-1, 0] = nan, nan
        keep = torch.ones(rows, wide, dtype=torch.bool, device="cuda")
        if rows > 2:
            x[rows // 2] = inf
        z = d.forward(x, wg, wu)[0].t
        assert bool(z[0].isnan().all()) and bool(z[:, -1].isnan().all())
        if rows > 2:
            assert not bool(z[rows // 2].isfinite().any())
            keep[rows // 2] = False
        keep[0], keep[:, -1] = False, False
        assert torch.equal(y[keep], z[keep])
        return
    g, u = d.normal(rows, wide), d.normal(rows, wide)
    a = d.backward(dy, g, u, x, wg, wu)
    dy2, x2 = d.put(dy), d.put(x)
    dy2[0, -1] = nan  # the first token's gradient, the last feature's
    x2[-1, 0] = nan   # the first column of the weights'
    b = d.backward(dy2, g, u, x2, wg, wu)
    for k, r in b.items():
        bad = r.t.isnan()
        want = torch.zeros_like(bad)
        if k in ("dg", "du"):
            want[0, -1] = True
        elif k == "dx":
            want[0] = True
        else:
            want[-1], want[:, 0] = True, True
        assert torch.equal(bad, want), k
        assert torch.equal(r.t[~bad], a[k].t[~bad]), k


@pytest.mark.parametrize("small", ["x", "w"])
@pytest.mark.parametrize("dtype,rows,cols,wide,pad,call", [
    (F32, 1605, 2944, 2131, 0, "forward"), (F32, 137, 1280, 5760, 0, "gu"), (F32, 971, 1152, 6720, 0, "i"),
    (F32, 1798, 789, 131, 0, "forward"), (F32, 34, 114, 44, 1, "forward"), (F32, 157, 42, 137, 0, "igu"),
    (BF16, 839, 16, 4856, 0, "forward"), (BF16, 18, 556, 54, 5, "forward"), (BF16, 2, 300, 100, 0, "forward"),
    (BF16, 292, 47, 234, 5, "igu")])
def test_operands_near_the_least(dtype, rows, cols, wide, pad, call, small):
    """Operands down to the least of their type's: of F32 what lies below 2^-133 may be
    left out, of 16-bit types nothing."""
    d = Data(dtype, rows, cols, wide, pad, call, seed=4)
    least = 2.0 ** (-118 if dtype == F32 else -128)
    lost = 2.0 ** -133 if dtype == F32 else 0.0
    a, b = (least, 1.0) if small == "x" else (1.0, least)
    x = d.normal(rows, cols, scale=a)
    wg, wu = (d.normal(wide, cols, scale=b) for _ in range(2))

    def check(got, p, q, terms, left, right, what):
        value, bound = R.product(p, q, dtype != F32)
        # a step of the least numbers for each rounding on the way
        bound = bound + 2 * terms * 2.0 ** -149
        if left:
            bound = bound + lost * q.double().abs().sum(1)
        if right:
            bound = bound + lost * p.double().abs().sum(1, keepdim=True)
        close(got, value, bound, what)

    if call == "forward":
        _, g, u = d.forward(x, wg, wu)
        check(g.t, x, wg, cols, small == "x", small == "w", "gate")
        check(u.t, x, wu, cols, small == "x", small == "w", "up")
        return
    # the gradients of the projections small in the place of the weights, and the input
    dy = d.normal(rows, wide, scale=b if "i" not in call else a)
    out = d.backward(dy, d.put(torch.full((rows, wide), 4.0, device="cuda")), d.normal(rows, wide), x, wg, wu)
    for k, (p, q, terms) in d.products(out["dg"].t, out["du"].t, x, wg, wu).items():
        check(out[k].t, p, q, terms, True, True, k)
