"""The step's operators on the GPU against 64-bit references: layer norm, the
gated feed-forward block, gradient clipping."""

import math

import pytest
import torch

import cross_rank_collective_amd as crc
from tests import step_reference as R
from tests.block_reference import close

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]
MARK = 0x5A


def rand(*shape, seed=0, scale=1.0, dtype=F32):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(dtype)


class Room:
    """A rows x cols matrix inside a buffer of marked bytes: `pad` elements
    behind each row, `lead` elements before the first."""

    def __init__(self, rows, cols, dtype, pad=0, lead=0, value=None):
        es = dtype.itemsize
        n = (lead + rows * (cols + pad) + 7) * es
        self.bytes = torch.full((n + 64,), MARK, dtype=torch.uint8, device="cuda")
        flat = self.bytes[:n].view(dtype)
        self.t = flat[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        if value is not None:
            self.t.copy_(value)

    def check(self, what):
        """Nothing but the matrix's own elements was written."""
        if self.t.numel():
            self.t.view(torch.int32 if self.t.element_size() == 4 else torch.int16).copy_(
                torch.full_like(self.t, 0).view(torch.int32 if self.t.element_size() == 4 else torch.int16)
                .fill_(0x5A5A5A5A if self.t.element_size() == 4 else 0x5A5A))
        assert bool((self.bytes == MARK).all()), f"{what}: bytes around it were written"


def put(t, pad=0, lead=0):
    return Room(*t.shape, t.dtype, pad, lead, t).t


# ---------------------------------------------------------------- layer norm

LN_SHAPES = [
    # rows, cols, ranks, pad, lead
    (1, 8, 0, 0, 0), (1, 1, 1, 0, 0), (3, 7, 2, 1, 1), (5, 64, 0, 0, 0), (2, 513, 1, 3, 1),
    (300, 1000, 3, 0, 0), (64, 2501, 8, 3, 1), (7, 4096, 5, 8, 0), (2, 8193, 1, 0, 3),
    (2, 16384, 9, 0, 0), (1, 16381, 2, 1, 1),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,ranks,pad,lead", LN_SHAPES)
def test_layer_norm(rows, cols, ranks, pad, lead, dtype):
    x = rand(rows, cols, seed=1, dtype=dtype) + rand(rows, 1, seed=2, scale=3).to(dtype)
    parts = [rand(rows, cols, seed=3 + r, dtype=dtype) for r in range(ranks)]
    wt = F32 if rows % 2 else dtype
    w, b = 1 + rand(cols, seed=20, scale=0.3), rand(cols, seed=21, scale=0.3)
    w, b = w.to(wt), b.to(wt)
    want = R.layer_norm(parts, x, w, b, 1e-5)
    x_out, z = Room(rows, cols, dtype, pad, lead), Room(rows, cols, dtype, pad, lead)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    crc.layer_norm([put(p, pad, lead) for p in parts], put(x, pad, lead), x_out.t, z.t,
                   weight=w.cuda(), bias=b.cuda(), mean=mean, rstd=rstd)
    got = {"x_out": x_out.t, "mean": mean, "rstd": rstd, "z": z.t}
    for k, v in got.items():
        close(v, *want[k], k)
    x_out.check("x_out")
    z.check("z")


def test_layer_norm_without_weights_in_place():
    x, y = rand(9, 1000, seed=1), rand(9, 1000, seed=2)
    want = R.layer_norm([y], x, None, None, 0.0)
    gx, gy = x.cuda(), y.cuda()
    crc.layer_norm([gy], gx, gx, gy, eps=0.0)  # x' over x, z over the partial
    close(gx, *want["x_out"], "x_out")
    close(gy, *want["z"], "z")


@pytest.mark.parametrize("dtype", TYPES)
def test_layer_norm_mean_far_from_zero(dtype):
    """A row's mean of 1000 times its spread: the differences keep their digits."""
    x = (rand(17, 1500, seed=5) + 1000.0).to(dtype)
    want = R.layer_norm([], x, None, None, 1e-5)
    z = torch.empty_like(x, device="cuda")
    mean, rstd = torch.empty(17, device="cuda"), torch.empty(17, device="cuda")
    crc.layer_norm([], x.cuda(), None, z, mean=mean, rstd=rstd)
    for k, v in {"z": z, "mean": mean, "rstd": rstd}.items():
        close(v, *want[k], k)


def test_layer_norm_range_and_nan():
    cols = 4096
    x = rand(6, cols, seed=7)
    x[0] *= 1e37  # the sum passes binary32's range only by its partial sums' sizes
    x[0] += 2e37
    x[1] = 3.0  # no spread
    x[2, 5] = math.nan
    x[3, 9] = math.inf
    x[4] *= 1e-30
    z, mean, rstd = torch.empty(6, cols, device="cuda"), torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    crc.layer_norm([], x.cuda(), None, z, mean=mean, rstd=rstd, eps=1e-5)
    assert bool(torch.isnan(z[2]).all()) and bool(torch.isnan(z[3]).all())
    assert bool((z[1] == 0).all()) and float(mean[1]) == 3.0
    assert abs(float(mean[0]) / float(x[0].double().mean()) - 1) < 1e-5
    assert float(rstd[0]) == 0.0  # the variance passes the range
    close(mean[4:], *(t[4:] for t in R.layer_norm([], x, None, None, 1e-5)["mean"]), "mean")
    y = rand(3, cols, seed=8) * 2e18  # squares' sum passes the range, their mean does not
    want = R.layer_norm([], y, None, None, 1e-5)
    z = torch.empty(3, cols, device="cuda")
    crc.layer_norm([], y.cuda(), None, z)
    close(z, want["z"][0], 2 * want["z"][1], "z")  # another rounding a square: v / D


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad,lead", [
    (1, 8, 0, 0), (1, 1, 0, 0), (4, 7, 1, 1), (300, 1000, 0, 0), (257, 2501, 3, 1), (2000, 520, 8, 0),
    (9, 8193, 0, 1), (300, 16384, 0, 0), (5000, 64, 0, 0)])
def test_layer_norm_backward(rows, cols, pad, lead, dtype):
    dz, dxo = rand(rows, cols, seed=1, dtype=dtype), rand(rows, cols, seed=2, dtype=dtype)
    x = rand(rows, cols, seed=3, dtype=dtype) + rand(rows, 1, seed=4).to(dtype)
    mean = x.double().mean(1).float()
    rstd = (x.double().var(1, correction=0) + 1e-5).rsqrt().float()
    wt = F32 if rows % 2 else dtype
    w = (1 + rand(cols, seed=5, scale=0.3)).to(wt)
    want = R.layer_norm_backward(dz, dxo, x, mean, rstd, w)
    dx, dw, db = Room(rows, cols, dtype, pad, lead), Room(1, cols, wt), Room(1, cols, wt)
    args = [put(t, pad, lead) for t in (dz, dxo, x)]
    crc.layer_norm_backward(*args, mean.cuda(), rstd.cuda(), dx.t, weight=w.cuda(), dweight=dw.t[0],
                            dbias=db.t[0])
    close(dx.t, *want["dx"], "dx")
    close(dw.t[0], *want["dweight"], "dweight")
    close(db.t[0], *want["dbias"], "dbias")
    for r in (dx, dw, db):
        r.check("a gradient")
    # without what is optional, over dz itself
    want = R.layer_norm_backward(dz, None, x, mean, rstd, None)
    crc.layer_norm_backward(args[0], None, args[2], mean.cuda(), rstd.cuda(), args[0])
    close(args[0], *want["dx"], "dx over dz")


def test_layer_norm_gradient_by_differences():
    """Against differences of the forward formula in 64 bits."""
    rows, cols = 3, 40
    x, dz = rand(rows, cols, seed=1).double(), rand(rows, cols, seed=2).double()
    w = (1 + rand(cols, seed=3, scale=0.3)).double()

    def loss(x, w):
        m = x.mean(1, keepdim=True)
        return ((x - m) * ((x - m).square().mean(1, keepdim=True) + 1e-5) ** -0.5 * w * dz).sum()

    dx, dw = torch.empty(rows, cols, device="cuda"), torch.empty(cols, device="cuda")
    z, mean, rstd = torch.empty(rows, cols, device="cuda"), *(torch.empty(rows, device="cuda") for _ in "12")
    gx = x.float().cuda()
    crc.layer_norm([], gx, None, z, weight=w.float().cuda(), mean=mean, rstd=rstd)
    crc.layer_norm_backward(dz.float().cuda(), None, gx, mean, rstd, dx, weight=w.float().cuda(), dweight=dw)
    h = 1e-5
    for t, g in ((x, dx), (w, dw)):
        flat = t.view(-1)
        for i in range(0, flat.numel(), 7):
            keep = float(flat[i])
            flat[i] = keep + h
            up = loss(x, w)
            flat[i] = keep - h
            down = loss(x, w)
            flat[i] = keep
            # differences in 64 bits: h^2 of a third derivative of order 1; the kernel: some 100 U
            assert abs(float((up - down) / (2 * h)) - float(g.view(-1)[i])) < 2e-5


# ---------------------------------------------------------------- feed-forward

FFN_SHAPES = [
    # rows, cols, wide, pad, lead
    (1, 8, 8, 0, 0), (1, 1, 1, 0, 0), (2, 3, 5, 1, 1), (7, 64, 64, 0, 0), (33, 72, 40, 8, 8),
    (129, 200, 136, 0, 0), (128, 256, 256, 0, 0), (65, 1003, 251, 1, 0), (300, 77, 333, 0, 1),
    (17, 4096, 96, 0, 0), (1, 1024, 1000, 0, 0), (5, 515, 129, 3, 1), (16, 512, 512, 0, 0),
    (48, 640, 320, 0, 0), (100, 130, 6, 0, 0), (40, 6, 200, 2, 0),
]
ACTS = ["silu", "gelu", "gelu_tanh"]


def ffn_inputs(rows, cols, wide, dtype, seed=0):
    x = rand(rows, cols, seed=seed + 1, dtype=dtype)
    scale = 2.0 / math.sqrt(cols)
    return (x, rand(wide, cols, seed=seed + 2, scale=scale, dtype=dtype),
            rand(wide, cols, seed=seed + 3, scale=scale, dtype=dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,wide,pad,lead", FFN_SHAPES)
def test_gated_ffn(rows, cols, wide, pad, lead, dtype):
    x, wg, wu = ffn_inputs(rows, cols, wide, dtype)
    act = ACTS[rows % 3]
    want = R.gated_ffn(x, wg, wu, act)
    outs = {k: Room(rows, wide, dtype, pad, lead) for k in ("y", "gate", "up")}
    args = [put(t, pad, lead) for t in (x, wg, wu)]
    crc.gated_ffn(*args, outs["y"].t, activation=act, gate=outs["gate"].t, up=outs["up"].t)
    for k, v in outs.items():
        close(v.t, *want[k], k)
    alone = Room(rows, wide, dtype, pad, lead)
    crc.gated_ffn(*args, alone.t, activation=act)
    assert torch.equal(alone.t, outs["y"].t)
    for k, v in outs.items():
        v.check(k)
    alone.check("y alone")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,wide,pad,lead", FFN_SHAPES)
def test_gated_ffn_backward(rows, cols, wide, pad, lead, dtype):
    x, wg, wu = ffn_inputs(rows, cols, wide, dtype)
    g, u, dy = (rand(rows, wide, seed=s, scale=1.5, dtype=dtype) for s in (11, 12, 13))
    act = ACTS[cols % 3]
    want = R.gated_slopes(dy, g, u, act)
    dw_type = F32 if wide % 2 else dtype
    dg, du = Room(rows, wide, dtype, pad, lead), Room(rows, wide, dtype, pad, lead)
    dx = Room(rows, cols, dtype, pad, lead)
    dwg, dwu = Room(wide, cols, dw_type, pad, lead), Room(wide, cols, dw_type, pad, lead)
    gx, gwg, gwu, gg, gu, gdy = (put(t, pad, lead) for t in (x, wg, wu, g, u, dy))
    crc.gated_ffn_backward(gdy, gg, gu, dg.t, du.t, activation=act, x=gx, w_gate=gwg, w_up=gwu,
                           dx=dx.t, dw_gate=dwg.t, dw_up=dwu.t)
    close(dg.t, *want["dgate"], "dgate")
    close(du.t, *want["dup"], "dup")
    hg, hu = dg.t.cpu(), du.t.cpu()  # the products take them as rounded
    exact = dtype != F32
    pairs = torch.cat([hg, hu], 1), torch.cat([wg, wu], 0).t()
    close(dx.t, *R.product(*pairs, exact), "dx")
    close(dwg.t, *R.product(hg.t(), x.t(), exact), "dw_gate")
    close(dwu.t, *R.product(hu.t(), x.t(), exact), "dw_up")
    # one weight alone, added to what is there; slopes over their own inputs
    add = rand(wide, cols, seed=14, dtype=dw_type)
    one = put(add, pad, lead)
    crc.gated_ffn_backward(gdy, gg, gu, gg, gu, activation=act, x=gx, dw_up=one, accumulate=True)
    assert torch.equal(gg, dg.t) and torch.equal(gu, du.t)
    value, bound = R.product(hu.t(), x.t(), exact)
    close(one, value + add.double(), bound + R.U * (value.abs() + add.double().abs()), "accumulated")
    for r in (dg, du, dx, dwg, dwu):
        r.check("a gradient")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,wide", [(5, 264, 24), (5, 250, 24), (200, 264, 24), (200, 1003, 24), (64, 264, 200),
                                            (64, 250, 200), (200, 1000, 200), (200, 1003, 511), (700, 264, 200)])
def test_gated_ffn_both_gradients(rows, cols, wide, dtype):
    """All gradients of one call, sums of either kind split among workgroups or not,
    added to what is there; both weights' and one alone."""
    x, wg, wu = ffn_inputs(rows, cols, wide, dtype)
    g, u, dy = (rand(rows, wide, seed=s, dtype=dtype) for s in (21, 22, 23))
    add = [rand(wide, cols, seed=24 + i) for i in range(2)]
    exact = dtype != F32
    on = [t.cuda() for t in (dy, g, u, x, wg, wu)]
    for which in ((0, 1), (0,), (1,)):
        dg, du, dx = Room(rows, wide, dtype), Room(rows, wide, dtype, 8), Room(rows, cols, dtype, 8)
        dw = [Room(wide, cols, F32, 4, 0, add[i]) if i in which else None for i in range(2)]
        crc.gated_ffn_backward(on[0], on[1], on[2], dg.t, du.t, x=on[3], w_gate=on[4], w_up=on[5], dx=dx.t,
                               dw_gate=dw[0].t if dw[0] else None, dw_up=dw[1].t if dw[1] else None,
                               accumulate=True)
        hg, hu = dg.t.cpu(), du.t.cpu()
        pairs = torch.cat([hg, hu], 1), torch.cat([wg, wu], 0).t()
        close(dx.t, *R.product(*pairs, exact), "dx")
        for i in which:
            value, bound = R.product((hg, hu)[i].t(), x.t(), exact)
            close(dw[i].t, value + add[i].double(), bound + R.U * (value.abs() + add[i].double().abs()), f"dw {i}")
        for r in (dg, du, dx, *(dw[i] for i in which)):
            r.check("a gradient")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,cols,wide", [(1000, 520, 2056), (2048, 2048, 512), (520, 1032, 4096)])
def test_gated_ffn_tiles(rows, cols, wide, dtype):
    """Sizes at which tiles of every shape and splits of the sums are taken."""
    x, wg, wu = ffn_inputs(rows, cols, wide, dtype)
    y, g, u = (torch.empty(rows, wide, dtype=dtype, device="cuda") for _ in range(3))
    crc.gated_ffn(x.cuda(), wg.cuda(), wu.cuda(), y, gate=g, up=u)
    want = R.gated_ffn(x, wg, wu, "silu")
    for k, v in {"y": y, "gate": g, "up": u}.items():
        close(v, *want[k], k)
    dy = rand(rows, wide, seed=9, dtype=dtype).cuda()
    dx, dwg, dwu = (torch.empty_like(t, device="cuda") for t in (x, wg, wu))
    crc.gated_ffn_backward(dy, g, u, g, u, x=x.cuda(), w_gate=wg.cuda(), w_up=wu.cuda(), dx=dx,
                           dw_gate=dwg, dw_up=dwu)
    hg, hu = g.cpu(), u.cpu()
    close(dx, *R.product(torch.cat([hg, hu], 1), torch.cat([wg, wu], 0).t(), True), "dx")
    close(dwg, *R.product(hg.t(), x.t(), True), "dw_gate")
    close(dwu, *R.product(hu.t(), x.t(), True), "dw_up")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 40, 100, 300])
def test_gated_ffn_pitches_of_their_own(rows, dtype):
    """Every matrix in rows of another pitch, some at multiples of 16 bytes and
    some not."""
    cols, wide = 264, 200
    x, wg, wu = ffn_inputs(rows, cols, wide, dtype)
    want = R.gated_ffn(x, wg, wu, "silu")
    for step in (8, 1):
        y, g, u = (Room(rows, wide, dtype, step * (4 + i)) for i in range(3))
        gx, gwg, gwu = (put(t, step * (1 + i)) for i, t in enumerate((x, wg, wu)))
        crc.gated_ffn(gx, gwg, gwu, y.t, gate=g.t, up=u.t)
        for k, v in {"y": y, "gate": g, "up": u}.items():
            close(v.t, *want[k], k)
        dy = put(rand(rows, wide, seed=9, dtype=dtype), step * 7)
        dg, du, dx = Room(rows, wide, dtype, step * 8), Room(rows, wide, dtype, step * 9), Room(rows, cols, dtype, 3)
        dwg, dwu = Room(wide, cols, dtype, 5), Room(wide, cols, dtype, 6)
        crc.gated_ffn_backward(dy, g.t, u.t, dg.t, du.t, x=gx, w_gate=gwg, w_up=gwu, dx=dx.t,
                               dw_gate=dwg.t, dw_up=dwu.t)
        hg, hu, exact = dg.t.cpu(), du.t.cpu(), dtype != F32
        close(dx.t, *R.product(torch.cat([hg, hu], 1), torch.cat([wg, wu], 0).t(), exact), "dx")
        close(dwg.t, *R.product(hg.t(), x.t(), exact), "dw_gate")
        close(dwu.t, *R.product(hu.t(), x.t(), exact), "dw_up")
        for r in (y, g, u, dg, du, dx, dwg, dwu):
            r.check("an output")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,wide", [(1, 1024, 40), (3, 257, 17), (13, 2545, 65), (16, 128, 16), (7, 384, 300),
                                            (1, 9, 3), (16, 4100, 33)])
def test_gated_ffn_few_rows_between_words(rows, cols, wide, dtype):
    """Rows of few tokens and of weights that begin between two words, with NaN in
    the elements that share words with them."""
    x, wg, wu = ffn_inputs(rows, cols, wide, dtype)
    want = R.gated_ffn(x, wg, wu, "silu")
    for pads, leads in (((1, 1, 1), (0, 0, 0)), ((1, 2, 1), (1, 1, 1)), ((2, 1, 3), (0, 1, 1)), ((8, 8, 8), (1, 0, 1))):
        held = []
        for t, pad, lead in zip((x, wg, wu), pads, leads):
            ld = t.shape[1] + pad
            room = torch.full((lead + t.shape[0] * ld + 8,), math.nan, dtype=dtype, device="cuda")
            held.append(room[lead:lead + t.shape[0] * ld].view(t.shape[0], ld)[:, :t.shape[1]])
            held[-1].copy_(t)
        y, g, u = (Room(rows, wide, dtype, 1) for _ in range(3))
        crc.gated_ffn(*held, y.t, gate=g.t, up=u.t)
        for k, v in {"y": y, "gate": g, "up": u}.items():
            close(v.t, *want[k], k)
            v.check(k)


# ---------------------------------------------------------------- clipping

def grads_of(shapes, dtype, seed=0, scale=1.0):
    return [rand(*s, seed=seed + i, scale=scale, dtype=dtype) for i, s in enumerate(shapes)]


SHAPES = [(1,), (7,), (64, 64), (1000,), (33, 257), (3, 5, 7), (4097,), (128, 1000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("most", [1e9, 3.0])
def test_grad_clip(dtype, most):
    grads = grads_of(SHAPES, dtype)
    n = R.norm(grads)
    norm = torch.full((1,), -1.0, device="cuda")
    dev = [g.cuda() for g in grads]
    crc.grad_clip(dev, most, norm)
    close(norm, torch.tensor([n], dtype=torch.float64), torch.zeros(1, dtype=torch.float64), "norm")
    for i, (g, d) in enumerate(zip(grads, dev)):
        close(d, *R.scaled(g, n, most), f"gradient {i}")


def test_grad_clip_mixed_types_into_float32():
    grads = [rand(*s, seed=i, dtype=TYPES[i % 3]) for i, s in enumerate(SHAPES * 20)]  # several launches
    n = R.norm(grads)
    dev, outs = [g.cuda() for g in grads], [torch.empty(g.shape, device="cuda") for g in grads]
    norm = torch.zeros((), device="cuda")
    crc.grad_norm(dev, norm)
    close(norm, torch.tensor(n, dtype=torch.float64), torch.zeros((), dtype=torch.float64), "norm")
    crc.grad_scale(dev, norm, 2.0, outs=outs)
    for i, (g, d, o) in enumerate(zip(grads, dev, outs)):
        assert torch.equal(g, d.cpu())
        close(o, *R.scaled(g, n, 2.0), f"gradient {i}")


def test_grad_clip_rows_with_gaps_and_other_orders():
    rooms = [Room(5, 3, F32, 2, 1), Room(300, 130, BF16, 7, 3), Room(2, 9000, F16, 1, 1), Room(1, 4096, F32)]
    grads = []
    for i, r in enumerate(rooms):
        r.t.copy_(rand(*r.t.shape, seed=i, dtype=r.t.dtype))
        grads.append(r.t)
    grads.append(rand(40, 30, seed=8).cuda().t())            # columns first
    grads.append(rand(4, 6, 10, seed=9).cuda().transpose(0, 1))  # dense, in another order
    grads.append(rand(50, 8, seed=10).cuda()[:, 3:4])        # single elements, spaced
    grads.append(rand(6, 8, 12, seed=11).cuda()[:, :, :5])   # rows of two dimensions
    grads.append(torch.empty(0, 5, device="cuda"))
    before = [g.cpu().clone() for g in grads]
    n = R.norm(before)
    norm = torch.zeros(1, device="cuda")
    crc.grad_clip(grads, 1.0, norm)
    close(norm, torch.tensor([n], dtype=torch.float64), torch.zeros(1, dtype=torch.float64), "norm")
    for i, (b, g) in enumerate(zip(before, grads)):
        close(g, *R.scaled(b, n, 1.0), f"gradient {i}")
    for i, r in enumerate(rooms):
        r.check(f"gradient {i}")


def test_grad_norm_range_and_specials():
    norm = torch.zeros(1, device="cuda")
    big, small = torch.full((1000,), 1e30, device="cuda"), torch.full((1000,), 1e-30, device="cuda")
    for g in (big, small):
        crc.grad_norm([g], norm)
        want = float(g[0].double()) * math.sqrt(1000)
        assert abs(float(norm) / want - 1) < 2.0 ** -23
    crc.grad_norm([], norm)
    assert float(norm) == 0.0
    crc.grad_norm([small, small], norm)  # listed twice, counts twice
    assert abs(float(norm) / (1e-30 * math.sqrt(2000)) - 1) < 1e-6
    huge = torch.full((1000,), 3e38, device="cuda")
    crc.grad_norm([huge], norm)
    assert math.isinf(float(norm))  # the norm itself passes binary32's range
    bad = torch.ones(5, device="cuda")
    bad[2] = math.nan
    ones = torch.ones(3, device="cuda")
    crc.grad_clip([ones, bad], 1.0, norm)
    assert math.isnan(float(norm)) and bool(torch.isnan(ones).all()) and bool(torch.isnan(bad).all())
    bad = torch.ones(5, device="cuda")
    bad[2] = math.inf
    ones = torch.ones(3, device="cuda")
    crc.grad_clip([ones, bad], 1.0, norm)
    assert math.isinf(float(norm)) and bool((ones == 0).all())
    assert bad.isnan().tolist() == [False, False, True, False, False]
    ones = torch.ones(3, device="cuda")
    crc.grad_clip([ones], 0.0, norm)
    assert bool((ones == 0).all())
    zeros = torch.zeros(3, device="cuda")
    crc.grad_clip([zeros], 0.0, norm)
    assert float(norm) == 0.0 and bool((zeros == 0).all())
    ones = torch.ones(3, device="cuda")
    crc.grad_clip([ones], math.inf, norm)
    assert bool((ones == 1).all())
