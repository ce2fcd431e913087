"""The step's operators without a GPU: refusals of the C ABI in their order,
workspace queries, the extension module and the 64-bit reference itself."""

import ctypes
import math

import pytest
import torch

import cross_rank_collective_amd as crc
from cross_rank_collective_amd import step as S
from cross_rank_collective_amd.block import ptored_rows
from tests import step_reference as R

OK, INVALID, UNSUPPORTED, OVERLAP = 0, -1, -2, -3
F32, BF16, F16, I32 = 0, 1, 2, 3
BIG = 1 << 62


def at(k):
    """A made-up device address, far from the others."""
    return 0x100000000 + k * 0x10000000


def rows(k, ld, off=0):
    return ptored_rows(at(k) + off, ld)


NONE = ptored_rows()


# ---------------------------------------------------------------- layer norm

def ln(rows_=0, cols=8, parts=(), part_ld=8, x=rows(1, 8), x_out=NONE, z=NONE, w=None, b=None,
       eps=1e-5, dt=F32, wdt=F32, mean=None, rstd=None, nranks=None):
    p = S.ptored_layer_norm_params(rows_, cols, w, b, eps, dt, wdt)
    n = len(parts) if nranks is None else nranks
    return S.ptored_layer_norm(list(parts), n, part_ld, p, x, x_out, z, mean, rstd, 0)


def test_layer_norm_refusals():
    assert ln() == OK  # no rows: nothing is launched
    assert ln(cols=0, rows_=4, x=rows(1, 0)) == OK
    for bad in (dict(rows_=-1), dict(cols=-1), dict(x=NONE), dict(eps=-1.0), dict(eps=math.nan),
                dict(nranks=-1), dict(nranks=65), dict(parts=[0]), dict(rows_=4, x=rows(1, 7)),
                dict(rows_=4, parts=[at(3)], part_ld=7), dict(rows_=4, z=rows(2, 7)),
                dict(rows_=BIG, cols=BIG)):
        assert ln(**bad) == INVALID, bad
    for bad in (dict(dt=I32), dict(dt=7), dict(dt=BF16, wdt=F16), dict(cols=16385, x=rows(1, 16385))):
        assert ln(**bad) == UNSUPPORTED, bad
    # order: shapes, then types, then alignment, then overlaps
    assert ln(rows_=4, x=rows(1, 7), dt=I32) == INVALID
    assert ln(rows_=4, x=rows(1, 8, 2)) == INVALID  # half an element off
    assert ln(rows_=4, w=at(5) + 2) == INVALID
    assert ln(rows_=4, x_out=rows(1, 8, 4)) == OVERLAP
    assert ln(rows_=4, z=rows(2, 8), x_out=rows(2, 8)) == OVERLAP  # two outputs
    assert ln(rows_=4, z=rows(1, 9)) == OVERLAP  # x in another pitch
    assert ln(rows_=4, mean=at(1)) == OVERLAP
    assert ln(rows_=4, z=rows(2, 8), rstd=at(2) + 8) == OVERLAP


def lngrad(rows_=0, cols=8, dz=rows(1, 8), dxo=NONE, x=rows(2, 8), mean=at(3), rstd=at(4), dx=rows(5, 8),
           dw=None, db=None, ws=None, nbytes=0, dt=F32, wdt=F32, w=None):
    p = S.ptored_layer_norm_params(rows_, cols, w, None, math.nan, dt, wdt)  # eps is not read
    return S.ptored_layer_norm_backward(p, dz, dxo, x, mean, rstd, dx, dw, db, ws, nbytes, 0)


def test_layer_norm_backward_refusals():
    assert lngrad() == OK
    for bad in (dict(dz=NONE), dict(x=NONE), dict(mean=None), dict(rstd=None), dict(rows_=-1),
                dict(rows_=4, dz=rows(1, 7)), dict(rows_=4, dxo=rows(6, 1))):
        assert lngrad(**bad) == INVALID, bad
    assert lngrad(dt=I32) == UNSUPPORTED
    st, need = S.ptored_layer_norm_backward_workspace(4, 8)
    assert st == OK and need > 0
    assert lngrad(rows_=4, dw=at(6)) == INVALID  # no workspace
    assert lngrad(rows_=4, dw=at(6), ws=at(7), nbytes=need // 64) == INVALID
    assert lngrad(rows_=4, dw=at(6), ws=at(7) + 8, nbytes=need) == INVALID  # not at 16 bytes
    assert lngrad(rows_=4, dw=at(6), ws=at(1), nbytes=need) == OVERLAP
    assert lngrad(rows_=4, dw=at(1), ws=at(7), nbytes=need) == OVERLAP
    assert lngrad(rows_=4, dx=rows(3, 8)) == OVERLAP
    assert lngrad(rows_=4, dx=rows(2, 9)) == OVERLAP
    assert lngrad(rows_=4, dx=NONE) == OK  # nothing is wanted
    assert S.ptored_layer_norm_backward_workspace(4, 16385)[0] == UNSUPPORTED
    assert S.ptored_layer_norm_backward_workspace(-1, 4)[0] == INVALID


# ---------------------------------------------------------------- feed-forward

def ffn(T=0, D=8, F=16, x=rows(1, 8), wg=rows(2, 8), wu=rows(3, 8), y=rows(4, 16), gate=NONE, up=NONE,
        dt=BF16, act=0, ws=None, nbytes=0):
    return S.ptored_gated_ffn(S.ptored_ffn_params(T, D, F, dt, act), x, wg, wu, y, gate, up, ws, nbytes, 0)


def test_gated_ffn_refusals():
    assert ffn() == OK
    assert ffn(T=3, F=0, y=rows(4, 0)) == OK
    for bad in (dict(T=-1), dict(x=NONE), dict(wg=NONE), dict(wu=NONE), dict(y=NONE),
                dict(T=2, x=rows(1, 7)), dict(T=2, y=rows(4, 15)), dict(T=2, gate=rows(5, 3)),
                dict(T=BIG, D=BIG)):
        assert ffn(**bad) == INVALID, bad
    for bad in (dict(dt=I32), dict(act=3), dict(act=-1), dict(D=1 << 22, x=rows(1, 1 << 22), wg=rows(2, 1 << 22),
                                                            wu=rows(3, 1 << 22)),
                dict(T=2, x=rows(1, (1 << 21) + 8)), dict(F=(1 << 21) + 1, y=rows(4, 1 << 22))):
        assert ffn(**bad) == UNSUPPORTED, bad
    assert ffn(T=2, x=rows(1, 8, 1)) == INVALID
    assert ffn(T=2, y=rows(1, 16)) == OVERLAP
    assert ffn(T=2, y=rows(2, 16)) == OVERLAP
    assert ffn(T=2, gate=rows(4, 16)) == OVERLAP
    assert ffn(T=2, gate=rows(5, 16), up=rows(5, 16, 8)) == OVERLAP
    # too many tiles for a launch
    assert ffn(T=1 << 40, F=1 << 20, y=rows(4, 1 << 20)) in (INVALID, UNSUPPORTED)
    # few tokens and features split the columns: the workspace is checked
    st, need = S.ptored_gated_ffn_workspace(1, 8192, 16, BF16)
    assert st == OK and need > 0
    few = dict(T=1, D=8192, F=16, x=rows(1, 8192), wg=rows(2, 8192), wu=rows(3, 8192))
    assert ffn(**few) == INVALID
    assert ffn(**few, ws=at(6) + 4, nbytes=need) == INVALID
    assert ffn(**few, ws=at(6), nbytes=need - 1) == INVALID
    assert ffn(**few, ws=at(2), nbytes=need) == OVERLAP
    assert S.ptored_gated_ffn_workspace(1, 8, 8, I32)[0] == UNSUPPORTED
    assert S.ptored_gated_ffn_workspace(-1, 8, 8, F32)[0] == INVALID


def ffngrad(T=0, D=8, F=16, dt=BF16, act=0, **io):
    full = dict(dy=rows(1, 16), gate=rows(2, 16), up=rows(3, 16), dgate=rows(4, 16), dup=rows(5, 16),
                x=rows(6, 8), w_gate=rows(7, 8), w_up=rows(8, 8), dx=rows(9, 8), dw_gate=rows(10, 8),
                dw_up=rows(11, 8), dw_dtype=dt, accumulate=0, workspace=at(12), workspace_bytes=1 << 27)
    full.update(io)
    g = S.ptored_ffn_grad_io()
    for k, v in full.items():
        setattr(g, k, v)
    return S.ptored_gated_ffn_backward(S.ptored_ffn_params(T, D, F, dt, act), g, 0)


def test_gated_ffn_backward_refusals():
    for k in ("dy", "gate", "up", "dgate", "dup", "x", "w_gate", "w_up"):
        assert ffngrad(T=2, **{k: NONE}) == INVALID, k
    for k in ("dy", "gate", "up", "dgate", "dup"):
        assert ffngrad(T=2, **{k: rows(20, 15)}) == INVALID, k
    for k in ("x", "w_gate", "w_up", "dx", "dw_gate", "dw_up"):
        assert ffngrad(T=2, **{k: rows(20, 7)}) == INVALID, k
    assert ffngrad(T=2, dt=I32) == UNSUPPORTED
    assert ffngrad(T=2, act=9) == UNSUPPORTED
    assert ffngrad(T=2, dw_dtype=F16) == UNSUPPORTED
    assert ffngrad(T=2, x=rows(6, 1 << 22)) == UNSUPPORTED
    assert ffngrad(T=2, dy=rows(1, 16, 1)) == INVALID
    assert ffngrad(T=2, dgate=rows(4, 16), dup=rows(4, 16)) == OVERLAP
    assert ffngrad(T=2, dgate=rows(2, 17)) == OVERLAP
    for k in ("dx", "dw_gate", "dw_up"):
        for other in (1, 2, 4, 6, 7):
            assert ffngrad(T=2, **{k: rows(other, 8)}) == OVERLAP, (k, other)
    # a split product's workspace
    st, need = S.ptored_gated_ffn_backward_workspace(4096, 64, 64, BF16)
    assert st == OK and need > 0
    wide = {k: rows(n, 64) for n, k in enumerate(("dy", "gate", "up", "dgate", "dup", "x", "w_gate",
                                                  "w_up", "dx", "dw_gate", "dw_up"), 1)}
    assert ffngrad(T=4096, D=64, F=64, **wide, workspace=None) == INVALID
    assert ffngrad(T=4096, D=64, F=64, **wide, workspace_bytes=16) == INVALID
    assert ffngrad(T=4096, D=64, F=64, **wide, workspace=at(12) + 8) == INVALID
    assert ffngrad(T=4096, D=64, F=64, **wide, workspace=at(1)) == OVERLAP


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_workspaces_cover_every_call(dtype):
    """Queries grow with nothing unreasonable: at most 32 bits for each of a few
    splits of the outputs."""
    for T in (1, 7, 16, 17, 64, 128, 1000, 8192):
        for D in (8, 100, 1024, 5120):
            for F in (8, 130, 2048, 12288):
                _, n = S.ptored_gated_ffn_workspace(T, D, F, dtype)
                assert 0 <= n <= 64 * 2 * T * (F + 3) * 4
                _, n = S.ptored_gated_ffn_backward_workspace(T, D, F, dtype)
                assert 0 <= n <= 2048 * 4 * max(T * (D + 3), 2 * F * (D + 3))
                assert n <= 1 << 30


# ---------------------------------------------------------------- clipping

def grads(*entries):
    t = (S.ptored_grad * max(1, len(entries)))()
    for e, v in zip(t, entries):
        e.data, e.out, e.rows, e.cols, e.ld, e.out_ld, e.dtype, e.out_dtype = v
    return t, len(entries)


def clip(*entries, most=1.0, norm=at(30), ws=at(31), nbytes=1 << 24, count=None):
    t, n = grads(*entries)
    return S.ptored_grad_clip(t, n if count is None else count, most, norm, ws, nbytes, 0)


def scale(*entries, most=1.0, norm=at(30), ws=at(31), nbytes=1 << 24):
    t, n = grads(*entries)
    return S.ptored_grad_scale(t, n, norm, most, ws, nbytes, 0)


def dense(k, n, dt=F32, out=None, odt=None):
    return (at(k), at(k if out is None else out), 1, n, n, n, dt, dt if odt is None else odt)


def test_gradient_refusals():
    assert scale() == OK  # nothing to scale
    assert scale((0, 0, 0, 5, 5, 5, F32, F32)) == OK
    for bad in (dict(most=-1.0), dict(most=math.nan), dict(norm=None), dict(norm=at(30) + 2)):
        assert scale(dense(1, 8), **bad) == INVALID, bad
    assert clip(dense(1, 8), count=-1) == INVALID
    assert scale((0, at(1), 1, 8, 8, 8, F32, F32)) == INVALID
    assert scale((at(1), 0, 1, 8, 8, 8, F32, F32)) == INVALID
    assert scale((at(1), at(1), 2, 8, 7, 8, F32, F32)) == INVALID
    assert scale((at(1), at(1), 2, 8, 8, 7, F32, F32)) == INVALID
    assert scale((at(1), at(1), -1, 8, 8, 8, F32, F32)) == INVALID
    assert scale((at(1) + 2, at(1) + 2, 1, 8, 8, 8, F32, F32)) == INVALID
    assert scale(dense(1, 8, I32)) == UNSUPPORTED
    assert scale(dense(1, 8, BF16, 2, F16)) == UNSUPPORTED
    assert scale(dense(1, 1 << 40)) == UNSUPPORTED
    assert scale((at(1), at(1), 2, 8, 1 << 28, 1 << 28, F32, F32)) == UNSUPPORTED
    assert scale((at(1), at(1), 1 << 31, 8, 8, 8, F32, F32)) == UNSUPPORTED
    assert clip(dense(1, 8), ws=None) == INVALID
    assert clip(dense(1, 8), nbytes=0) == INVALID
    assert clip(dense(1, 8), ws=at(31) + 8) == INVALID
    # what is written overlaps nothing
    assert scale(dense(1, 8), dense(1, 8)) == OVERLAP  # the same one twice, in place
    assert scale(dense(1, 8), dense(2, 8, out=1)) == OVERLAP
    assert scale(dense(1, 8, out=3), dense(2, 8, out=3)) == OVERLAP
    assert scale(dense(1, 8, BF16, 1, F32)) == OVERLAP  # wider, over itself
    assert scale((at(1), at(1), 2, 8, 8, 9, F32, F32)) == OVERLAP  # in place in another pitch
    assert scale(dense(1, 8), norm=at(1) + 4) == OVERLAP
    assert clip(dense(1, 8), norm=at(1)) == OVERLAP
    assert clip(dense(1, 8), ws=at(1)) == OVERLAP
    assert clip(dense(1, 8), norm=at(31)) == OVERLAP
    t, n = grads(dense(1, 8), dense(1, 8))
    assert S.ptored_grad_norm(t, n, at(1), at(31), 1 << 20, 0) == OVERLAP  # the norm on a gradient
    assert S.ptored_grad_norm(t, n, at(31), at(31), 1 << 20, 0) == OVERLAP
    st, need = S.ptored_grad_norm_workspace(t, n)
    assert st == OK and need == 16
    assert S.ptored_grad_norm_workspace(*grads(dense(1, 8, I32)))[0] == UNSUPPORTED
    assert S.ptored_grad_norm_workspace(t, -1)[0] == INVALID
    many = [dense(k, 100) for k in range(200)]
    st, need = S.ptored_grad_norm_workspace(*grads(*many))
    assert st == OK and need == 200 * 8 + 200 * 48  # partial sums and the table
    assert scale(*many, ws=None) == INVALID


# ---------------------------------------------------------------- Python's side

def test_the_extension_leaves_what_does_not_fit():
    from cross_rank_collective_amd import block as K

    K._torch is None and K._init()
    x, w, n = torch.zeros(4, 64), torch.ones(64), torch.zeros(1)
    none = [None]
    calls = {
        "layer_norm": [[x], x, x, x, w, w, 1e-5, *none * 3],
        "layer_norm_backward": [x, x, x, w[:4], w[:4], x, *none * 5],
        "gated_ffn": [x, x, x, x[:, :4], 0, *none * 4],
        "gated_ffn_backward": [x, x, x, x, x, 0, *none * 6, False, *none * 2],
        "grad_norm": [[x], n, *none * 2],
        "grad_scale": [[x], n, 1.0, *none * 3],
        "grad_clip": [[x], 1.0, n, *none * 3],
    }
    for name, args in calls.items():
        call = getattr(K._native, name)
        assert call(*args) is None, name
        assert call() is None and call(*args, None) is None, name
        assert call(*["no tensor"] * len(args)) is None, name
        for i in range(len(args)):
            assert call(*args[:i], object(), *args[i + 1:]) is None, (name, i)


def test_tensors_that_are_refused_without_a_gpu():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        crc.layer_norm([], x, x, x)
    with pytest.raises(ValueError, match="activation"):
        crc.gated_ffn(x, x, x, x, activation="relu")
    with pytest.raises(ValueError, match="GPU"):
        crc.gated_ffn(x, torch.zeros(5, 8), torch.zeros(5, 8), torch.zeros(4, 5))
    with pytest.raises(ValueError, match="norm"):
        crc.grad_clip([x], 1.0, torch.zeros(1))
    with pytest.raises(ValueError, match="norm"):
        crc.grad_norm([x], torch.zeros(2))
    with pytest.raises(crc.PtoredError):
        crc.layer_norm_backward_workspace(4, 1 << 20)


def test_how_gradients_lie():
    t = torch.zeros(6, 8, 12)
    assert S._runs(t) == (1, 576, 576)
    assert S._runs(t[:, :, :5]) == (48, 5, 12)
    assert S._runs(t[:, :4, :5]) is None
    assert S._runs(t[:, 0]) == (6, 12, 96)
    assert S._runs(t[0, :, 3]) == (8, 1, 12)
    assert S._runs(t[0].t()) is None and S._dense(t[0].t())
    assert not S._dense(t[:, :, :5]) and S._dense(t.permute(2, 0, 1))
    assert S._runs(torch.zeros(5, 1).expand(5, 4)) is None
    assert not S._dense(torch.zeros(5, 1).expand(5, 4))
    assert S._runs(torch.zeros(3, 1, 4)[:, :, 1:2]) == (3, 1, 4)


# ---------------------------------------------------------------- the reference

@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_reference_slopes_against_differences(name):
    g = torch.linspace(-9, 9, 181, dtype=torch.float64)
    h = 1e-5
    (up, _), _ = R.activation(name, g + h)
    (down, _), _ = R.activation(name, g - h)
    (f, ef), (slope, es) = R.activation(name, g)
    assert float(((up - down) / (2 * h) - slope).abs().max()) < 1e-9
    want = {"silu": torch.nn.functional.silu(g), "gelu": torch.nn.functional.gelu(g),
            "gelu_tanh": torch.nn.functional.gelu(g, approximate="tanh")}[name]
    assert float((f - want).abs().max()) < 1e-12
    assert bool((ef < 1e-4 * (1 + f.abs())).all()) and bool((es < 1e-4 * (1 + slope.abs())).all())


def test_reference_layer_norm_against_torch():
    x, y = torch.randn(5, 40, dtype=torch.float64), torch.randn(5, 40, dtype=torch.float64)
    w, b = torch.randn(40, dtype=torch.float64), torch.randn(40, dtype=torch.float64)
    got = R.layer_norm([y], x, w, b, 1e-5)
    want = torch.nn.functional.layer_norm(x + y, (40,), w, b, 1e-5)
    assert float((got["z"][0] - want).abs().max()) < 1e-12
    v, dz = (x + y).requires_grad_(), torch.randn(5, 40, dtype=torch.float64)
    wl = w.clone().requires_grad_()
    bl = b.clone().requires_grad_()
    torch.nn.functional.layer_norm(v, (40,), wl, bl, 1e-5).backward(dz)
    g = R.layer_norm_backward(dz, None, v.detach(), got["mean"][0], got["rstd"][0], w)
    for k, want in {"dx": v.grad, "dweight": wl.grad, "dbias": bl.grad}.items():
        assert float((g[k][0] - want).abs().max()) < 1e-12, k
