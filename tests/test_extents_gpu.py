"""Calls whose matrices are column ranges of one buffer, on the GPU: the same
results as with buffers of their own, and nothing written between."""

import pytest
import torch

import cross_rank_collective_amd as crc
from tests.test_step_gpu import F16, TYPES, rand

pytestmark = pytest.mark.gpu


class Halves:
    """Two rows x cols matrices, and `gap` marked columns behind each, in one buffer."""

    MARK = 7.0

    def __init__(self, rows, cols, dtype, gap=0, values=(None, None)):
        self.room = torch.full((rows, 2 * (cols + gap)), self.MARK, dtype=dtype, device="cuda")
        self.t = self.room[:, :cols], self.room[:, cols + gap:2 * cols + gap]
        self.gaps = self.room[:, cols:cols + gap], self.room[:, 2 * cols + gap:]
        for t, v in zip(self.t, values):
            if v is not None:
                t.copy_(v)

    def check(self, *want):
        for t, w in zip(self.t, want):
            assert torch.equal(t, w)
        assert all(bool((g == self.MARK).all()) for g in self.gaps)


SHAPES = [(3, 131, 45), (300, 264, 136), (40, 1001, 77), (700, 520, 515)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gap", [0, 3])
@pytest.mark.parametrize("rows,cols,wide", SHAPES)
def test_feed_forward(rows, cols, wide, gap, dtype):
    r = lambda *s, k, **kw: rand(*s, seed=k, dtype=dtype, **kw).cuda()  # noqa: E731
    x, dy = r(rows, cols, k=1), r(rows, wide, k=2)
    wg, wu = (r(wide, cols, k=k, scale=cols ** -0.5) for k in (3, 4))
    y, g, u, dg, du = (torch.empty_like(dy) for _ in range(5))
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    w2 = Halves(wide, cols, dtype, gap, (wg, wu))
    x2 = Halves(rows, cols, dtype, gap, (x, None))
    # the weights' and x's rows begin as they do in the halves, so that the same kernel runs
    wg, wu = (Halves(wide, cols, dtype, gap, (wg, wu)).t[i] for i in range(2))
    x = Halves(rows, cols, dtype, gap, (x, None)).t[0]
    kept = Halves(rows, wide, dtype, gap)
    crc.gated_ffn(x, wg, wu, y, gate=kept.t[0], up=kept.t[1])
    g, u = (t.clone() for t in kept.t)
    crc.gated_ffn(x, wg, wu, dg, gate=du, up=dx.new_empty(rows, wide))
    assert torch.equal(y, dg) and torch.equal(g, du)
    kept.check(g, u)
    sep = [Halves(rows, wide, dtype, gap, (t, None)).t[0] for t in (g, u)]
    sep[1] = Halves(rows, wide, dtype, gap, (None, u)).t[1]
    dw = [Halves(wide, cols, dtype, gap).t[i] for i in range(2)]
    crc.gated_ffn_backward(dy, *sep, *sep, x=x, w_gate=wg, w_up=wu, dx=dx, dw_gate=dw[0], dw_up=dw[1])
    dw2 = Halves(wide, cols, dtype, gap)
    crc.gated_ffn_backward(dy, *kept.t, *kept.t, x=x2.t[0], w_gate=w2.t[0], w_up=w2.t[1], dx=x2.t[1],
                           dw_gate=dw2.t[0], dw_up=dw2.t[1])
    kept.check(*sep)
    x2.check(x, dx)
    dw2.check(*dw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 64), (5, 131), (300, 1001), (70, 4096)])
def test_boundaries(rows, cols, dtype):
    r = lambda *s, k: rand(*s, seed=k, dtype=dtype).cuda()  # noqa: E731
    x, part, dz = r(rows, cols, k=1), r(rows, cols, k=2), r(rows, cols, k=3)
    w = torch.ones(cols, device="cuda")
    x_out, z, dx = (torch.empty_like(x) for _ in range(3))
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    for gap in (0, 1):
        crc.layer_norm([part], x, x_out, z, weight=w, mean=mean, rstd=rstd)
        two = Halves(rows, cols, dtype, gap)
        ins = Halves(rows, cols, dtype, gap, (x, part))
        crc.layer_norm([ins.t[1]], ins.t[0], *two.t, weight=w)
        two.check(x_out, z)
        crc.layer_norm([ins.t[1]], *ins.t[:1], *ins.t, weight=w)  # over what was read
        ins.check(x_out, z)
        dw, dw2 = torch.empty_like(w), torch.empty_like(w)
        crc.layer_norm_backward(dz, None, x_out, mean, rstd, dx, weight=w, dweight=dw)
        two = Halves(rows, cols, dtype, gap, (dz, None))
        crc.layer_norm_backward(two.t[0], None, x_out, mean, rstd, two.t[1], weight=w, dweight=dw2)
        two.check(dz, dx)
        assert torch.equal(dw, dw2)
        # the boundary with a root-mean-square norm
        crc.block_norm([part], x, x_out, z, pre_weight=w.to(dtype), pre_rstd=rstd)
        two = Halves(rows, cols, dtype, gap)
        crc.block_norm([part], x, *two.t, pre_weight=w.to(dtype))
        two.check(x_out, z)
        crc.block_norm_backward(dz, None, x_out, rstd, dx, pre_weight=w.to(dtype))
        two = Halves(rows, cols, dtype, gap, (dz, None))
        crc.block_norm_backward(two.t[0], None, x_out, rstd, two.t[1], pre_weight=w.to(dtype))
        two.check(dz, dx)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(5, 131), (300, 1001), (64, 512)])
def test_a_checkpoint_with_its_scales_behind_each_row(rows, cols, dtype):
    x = rand(rows, cols, seed=1, dtype=dtype).cuda()
    apart = crc.checkpoint_empty(rows, cols)
    crc.checkpoint_pack(x, apart)
    blocks = apart.scales.shape[1]
    room = torch.full((rows, cols + blocks + 3), 77, dtype=torch.uint8, device="cuda")
    kept = crc.Checkpoint(room.view(torch.int8)[:, :cols], room[:, cols:cols + blocks])
    crc.checkpoint_pack(x, kept)
    assert torch.equal(kept.q, apart.q) and torch.equal(kept.scales, apart.scales)
    assert bool((room[:, cols + blocks:] == 77).all())
    out, want = torch.empty_like(x), torch.empty_like(x)
    crc.checkpoint_unpack(apart, want)
    crc.checkpoint_unpack(kept, out)
    assert torch.equal(out, want)


def test_a_column_that_is_shared_is_refused():
    room = torch.zeros(6, 40, device="cuda", dtype=F16)
    x = torch.zeros(6, 20, device="cuda", dtype=F16)
    crc.layer_norm([], x, room[:, :20], room[:, 20:])
    with pytest.raises(crc.PtoredError, match="(?i)overlap"):
        crc.layer_norm([], x, room[:, :20], room[:, 19:39])
    with pytest.raises(crc.PtoredError, match="(?i)overlap"):  # rows that run into the next ones
        crc.layer_norm([], room[:, 30:].as_strided((5, 20), (40, 1), 30), room[:5, :20], None)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,many", [(5, 3, 2), (64, 131, 3), (300, 40, 90), (7, 1000, 4)])
def test_clipping_of_column_slices(rows, cols, many, dtype):
    """Slices of one fused gradient, clipped in place and into slices of another."""
    fused = rand(rows, many * cols, seed=1, dtype=dtype).cuda()
    # each in a buffer of its own, in rows that lie as the slices do
    parts = [fused.clone()[:, i * cols:(i + 1) * cols] for i in range(many)]
    norm, want = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    crc.grad_clip(parts, 1.0, want)
    for out_type in {dtype, torch.float32}:
        into = torch.full((rows, many * cols + 2), 7.0, dtype=out_type, device="cuda")
        outs = [into[:, 1 + i * cols:1 + (i + 1) * cols] for i in range(many)]
        crc.grad_clip(list(fused.split(cols, 1)), 1.0, norm, outs=outs)
        assert torch.equal(norm, want)
        for o, p in zip(outs, parts):
            assert torch.equal(o.to(dtype), p)
        assert bool((into[:, 0] == 7).all() and (into[:, -1] == 7).all())
    crc.grad_clip(list(fused.split(cols, 1)), 1.0, norm)
    assert torch.equal(norm, want) and torch.equal(fused, torch.cat(parts, 1))
    with pytest.raises(crc.PtoredError, match="(?i)overlap"):
        crc.grad_clip([fused[:, :cols + 1], fused[:, cols:]], 1.0, norm)
