"""Calls of the step's operators as programs make them: on other streams, captured
in graphs, through either way from Python, at offsets past 32 bits, together."""

import importlib.util
import math
import os

import pytest
import torch

import cross_rank_collective_amd as crc
from cross_rank_collective_amd import block as K
from tests import step_reference as R
from tests.block_reference import close
from tests.test_step_gpu import BF16, F16, F32, TYPES, ffn_inputs, put, rand

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Step:
    """Every operator once, on buffers of its own."""

    def __init__(self, rows=70, cols=264, wide=136, dtype=BF16, seed=0, many=3, workspaces=True):
        r = lambda *s, k=0, **kw: rand(*s, seed=seed + k, **kw).cuda()  # noqa: E731
        self.parts = [r(rows, cols, k=i, dtype=dtype) for i in range(2)]
        self.x, self.dz, self.dxo = (r(rows, cols, k=10 + i, dtype=dtype) for i in range(3))
        self.w, self.b = 1 + r(cols, k=20, scale=0.1), r(cols, k=21, scale=0.1)
        self.wg, self.wu = (r(wide, cols, k=22 + i, scale=cols ** -0.5, dtype=dtype) for i in range(2))
        self.dy = r(rows, wide, k=25, dtype=dtype)
        new = torch.empty_like
        self.out = {k: new(self.x) for k in ("x_out", "z", "dz_in", "dx")}
        self.out |= {k: torch.empty(rows, device="cuda") for k in ("mean", "rstd")}
        self.out |= {k: new(self.dy) for k in ("y", "g", "u", "dg", "du")}
        self.out |= {"dw": new(self.w), "db": new(self.b), "dwg": new(self.wg), "dwu": new(self.wu),
                     "norm": torch.empty(1, device="cuda")}
        # gradients clipped into tensors of their own, many enough for a table
        grads = [self.out["dwg"], self.out["dwu"], self.out["dw"], self.out["db"]]
        self.grads = grads + [r(5 + i, k=30 + i) for i in range(many)]
        self.clipped = [new(g) for g in self.grads]
        self.out |= {f"clipped{i}": t for i, t in enumerate(self.clipped)}
        self.ws = {}
        if workspaces:
            room = lambda n: torch.empty(max(16, n), dtype=torch.uint8, device="cuda")  # noqa: E731
            self.ws = {"ln": room(crc.layer_norm_backward_workspace(rows, cols)),
                       "ffn": room(crc.gated_ffn_workspace(rows, cols, wide, self.dy.dtype)),
                       "ffngrad": room(crc.gated_ffn_backward_workspace(rows, cols, wide, self.dy.dtype)),
                       "clip": room(1 << 20)}

    def run(self, stream=None):
        o, ws = self.out, self.ws.get
        crc.layer_norm(self.parts, self.x, o["x_out"], o["z"], weight=self.w, bias=self.b, mean=o["mean"],
                       rstd=o["rstd"], stream=stream)
        crc.gated_ffn(o["z"], self.wg, self.wu, o["y"], gate=o["g"], up=o["u"], workspace=ws("ffn"), stream=stream)
        crc.gated_ffn_backward(self.dy, o["g"], o["u"], o["dg"], o["du"], x=o["z"], w_gate=self.wg,
                               w_up=self.wu, dx=o["dz_in"], dw_gate=o["dwg"], dw_up=o["dwu"],
                               workspace=ws("ffngrad"), stream=stream)
        crc.layer_norm_backward(o["dz_in"], self.dxo, o["x_out"], o["mean"], o["rstd"], o["dx"],
                                weight=self.w, dweight=o["dw"], dbias=o["db"], workspace=ws("ln"), stream=stream)
        crc.grad_clip(self.grads, 0.5, o["norm"], outs=self.clipped, workspace=ws("clip"), stream=stream)

    def take(self):
        got = {k: v.clone() for k, v in self.out.items()}
        for v in self.out.values():
            v.fill_(math.nan)
        return got


def same(a, b, what):
    for k, v in a.items():
        assert torch.equal(v, b[k]), f"{what}: {k}"
        assert not bool(torch.isnan(v).any()), f"{what}: {k} was not written"


SIZES = [dict(), dict(rows=1, cols=4096, wide=64, many=100), dict(rows=9, cols=131, wide=45, dtype=F32),
         dict(rows=600, cols=520, wide=1032, dtype=F16, many=200)]


@pytest.mark.parametrize("size", SIZES)
def test_streams_graphs_and_repeats(size):
    step = Step(**size)
    step.run()
    want = step.take()
    step.run()
    same(step.take(), want, "again")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    same(step.take(), want, "another stream")
    torch.cuda.synchronize()
    step.run(stream=side.cuda_stream)
    side.synchronize()
    same(step.take(), want, "a stream's handle")
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step.run()
    torch.cuda.synchronize()
    x0 = step.x.clone()
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        same(step.take(), want, f"replay {i}")
        step.x.mul_(0.5)  # other inputs: the replay takes what is there
        graph.replay()
        torch.cuda.synchronize()
        got = step.take()
        step.run()  # and eager work in between
        same(got, step.take(), f"replay {i} of other inputs")
        step.x.copy_(x0)


def test_two_streams_at_once():
    steps = [Step(seed=s, rows=300, cols=1024, wide=512, many=80, workspaces=False) for s in (0, 1000)]
    want = []
    for s in steps:
        s.run()
        want.append(s.take())
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, q in zip(steps, streams):
            with torch.cuda.stream(q):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        same(s.take(), w, "side by side")


@pytest.mark.parametrize("size", SIZES)
def test_both_ways_from_python(size, monkeypatch):
    step = Step(**size)
    step.run()
    want = step.take()
    made = []

    def look(name, stream, *args):
        made.append(name)
        return False

    monkeypatch.setattr(K, "_native_call", look)
    step.run()
    same(step.take(), want, "Python's own way")
    assert set(made) == {"layer_norm", "layer_norm_backward", "gated_ffn", "gated_ffn_backward", "grad_clip"}


def test_tensors_that_fit_are_called_natively(monkeypatch):
    step = Step()
    native = K._native_call
    outcomes = []

    def look(name, *args):
        outcomes.append((name, native(name, *args)))
        return outcomes[-1][1]

    monkeypatch.setattr(K, "_native_call", look)
    step.run()
    crc.grad_norm(step.grads, step.out["norm"])
    crc.grad_scale(step.grads, step.out["norm"], 1.0)
    assert len(outcomes) == 7 and all(done for _, done in outcomes), outcomes


@pytest.mark.parametrize("native", [True, False])
def test_outputs_count_as_changed_in_place(native, monkeypatch):
    if not native:
        monkeypatch.setattr(K, "_native_call", lambda *a: False)
    step = Step()
    before = {k: v._version for k, v in step.out.items()}
    inputs = {k: getattr(step, k)._version for k in ("x", "dz", "wg", "dy", "w")}
    step.run()
    assert all(v._version > before[k] for k, v in step.out.items()), "an output"
    assert inputs == {k: getattr(step, k)._version for k in inputs}
    held = [g._version for g in step.grads]
    crc.grad_norm(step.grads, step.out["norm"])
    assert held == [g._version for g in step.grads]
    crc.grad_scale(step.grads, step.out["norm"], 1.0)
    assert all(g._version > h for g, h in zip(step.grads, held))


def test_refused_tensors():
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    n = torch.zeros(1, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        crc.layer_norm([], x, None, torch.empty(4, 63, device="cuda"))
    with pytest.raises(ValueError):
        crc.layer_norm([x[:3]], x, None, x)
    with pytest.raises(TypeError):
        crc.layer_norm([], x, None, x, weight=w.half())
    with pytest.raises(ValueError, match="cuda"):
        crc.layer_norm([], x, None, x, weight=w.cpu())
    with pytest.raises(ValueError, match="overlap"):
        crc.layer_norm([], x[:1].expand(4, 64), None, x)
    with pytest.raises(ValueError, match="column stride"):
        crc.gated_ffn(torch.randn(64, 4, device="cuda").t(), x, x, torch.empty(4, 4, device="cuda"))
    with pytest.raises(crc.PtoredError, match="(?i)overlap"):
        crc.layer_norm([], x, x[:, :64], x)
    with pytest.raises(crc.PtoredError, match="(?i)overlap"):
        crc.gated_ffn(x, x, x, x[:, :4])
    y = torch.randn(4, 5, device="cuda")
    with pytest.raises(ValueError, match="needs w_gate"):
        crc.gated_ffn_backward(y, y, y, y.clone(), y.clone(), dx=x)
    with pytest.raises(ValueError, match="need x"):
        crc.gated_ffn_backward(y, y, y, y.clone(), y.clone(), dw_up=torch.empty(5, 64, device="cuda"))
    with pytest.raises(TypeError):
        crc.gated_ffn_backward(y.half(), y.half(), y.half(), y.half(), y.half(), x=x.half(),
                               dw_up=torch.empty(5, 64, device="cuda", dtype=BF16))
    with pytest.raises(ValueError, match="lie in"):
        crc.grad_clip([x.view(4, 8, 8)[:, :4, :5]], 1.0, n)
    with pytest.raises(ValueError, match="one tensor for each"):
        crc.grad_clip([x], 1.0, n, outs=[])
    with pytest.raises(ValueError, match="shape"):
        crc.grad_clip([x], 1.0, n, outs=[w])
    with pytest.raises(ValueError, match="type or float32"):
        crc.grad_clip([x], 1.0, n, outs=[torch.empty(4, 64, device="cuda", dtype=BF16)])
    with pytest.raises(TypeError):
        crc.grad_clip([x.long()], 1.0, n)
    with pytest.raises(TypeError):
        crc.grad_clip([None], 1.0, n)
    with pytest.raises(ValueError, match="cuda"):
        crc.grad_clip([x.cpu()], 1.0, n)
    with pytest.raises(crc.PtoredError, match="(?i)overlap"):
        crc.grad_clip([x, x[:2]], 1.0, n)
    with pytest.raises(crc.PtoredError):
        crc.grad_clip([x], -1.0, n)
    crc.grad_clip([x], 1.0, n, workspace=torch.empty(4, device="cuda"))  # one sum of 8 bytes fits
    with pytest.raises(crc.PtoredError):
        crc.grad_clip([x], 1.0, n, workspace=torch.empty(1, device="cuda"))


def test_empty_tensors():
    e = lambda *s, **kw: torch.zeros(*s, device="cuda", **kw)  # noqa: E731
    crc.layer_norm([], e(0, 8), e(0, 8), e(0, 8))
    crc.layer_norm([], e(4, 0), e(4, 0), e(4, 0))
    dw, db = torch.ones(8, device="cuda"), torch.ones(8, device="cuda")
    crc.layer_norm_backward(e(0, 8), None, e(0, 8), e(0), e(0), e(0, 8), dweight=dw, dbias=db)
    assert float(dw.abs().sum() + db.abs().sum()) == 0
    y = torch.ones(4, 5, device="cuda")
    crc.gated_ffn(e(4, 0), e(5, 0), e(5, 0), y)
    assert float(y.abs().sum()) == 0
    crc.gated_ffn(e(0, 8), e(5, 8), e(5, 8), e(0, 5))
    crc.gated_ffn(e(4, 8), e(0, 8), e(0, 8), e(4, 0))
    dwg = torch.ones(5, 8, device="cuda")
    crc.gated_ffn_backward(e(0, 5), e(0, 5), e(0, 5), e(0, 5), e(0, 5), x=e(0, 8), dw_gate=dwg,
                           accumulate=True)
    assert float(dwg.sum()) == 40
    crc.gated_ffn_backward(e(0, 5), e(0, 5), e(0, 5), e(0, 5), e(0, 5), x=e(0, 8), dw_gate=dwg)
    assert float(dwg.abs().sum()) == 0
    dx = torch.ones(4, 8, device="cuda")
    crc.gated_ffn_backward(e(4, 0), e(4, 0), e(4, 0), e(4, 0), e(4, 0), w_gate=e(0, 8), w_up=e(0, 8), dx=dx)
    assert float(dx.abs().sum()) == 0
    dg, du = e(4, 5), e(4, 5)
    g, u, dy = rand(4, 5, seed=1), rand(4, 5, seed=2), rand(4, 5, seed=3)
    crc.gated_ffn_backward(dy.cuda(), g.cuda(), u.cuda(), dg, du, x=e(4, 0), dw_gate=e(5, 0))
    close(dg, *R.gated_slopes(dy, g, u, "silu")["dgate"], "dgate without columns")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [3, 20, 90, 700])
def test_a_row_of_nan_stays_alone(rows, dtype):
    """A token with NaN, and one with infinities, change no other token's outputs, a
    feature with NaN no other feature's."""
    cols, wide = 520, 264
    x, wg, wu = ffn_inputs(rows, cols, wide, dtype)
    y, z = (torch.empty(rows, wide, dtype=dtype, device="cuda") for _ in range(2))
    crc.gated_ffn(x.cuda(), wg.cuda(), wu.cuda(), y)
    x[1, 7], x[2] = math.nan, math.inf
    wg[5, 3] = math.nan
    crc.gated_ffn(x.cuda(), wg.cuda(), wu.cuda(), z)
    keep = torch.ones(rows, wide, dtype=torch.bool, device="cuda")
    keep[1], keep[2], keep[:, 5] = False, False, False
    assert torch.equal(y[keep], z[keep])
    assert bool(torch.isnan(z[1]).all()) and bool(torch.isnan(z[:, 5]).all())
    assert not bool(torch.isfinite(z[2]).any())


def test_overflow_of_f16():
    """Gradients of projections past f16's range are infinities, as rounded."""
    g, u, dy = (torch.full((3, 8), v, dtype=F16, device="cuda") for v in (4.0, 200.0, 400.0))
    dg, du = torch.empty_like(g), torch.empty_like(g)
    crc.gated_ffn_backward(dy, g, u, dg, du)
    assert bool(torch.isinf(dg).all()) and bool(torch.isfinite(du).all())


def far(rows, cols, ld, dtype, value=None):
    """A rows x cols matrix in rows of `ld` elements."""
    room = torch.empty(rows * ld, dtype=dtype, device="cuda")
    t = room.view(rows, ld)[:, :cols]
    if value is not None:
        t.copy_(value)
    return t


def test_layer_norm_of_rows_past_32_bits():
    rows, cols, ld = 5, 520, 1 << 30  # 2 GiB a row
    x, y, dz = (rand(rows, cols, seed=s, dtype=BF16) for s in (1, 2, 3))
    gx, gy = far(rows, cols, ld, BF16, x), far(rows, cols, ld, BF16, y)
    out, z = far(rows, cols, ld, BF16), far(rows, cols, ld, BF16)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    crc.layer_norm([gy], gx, out, z, mean=mean, rstd=rstd)
    want = R.layer_norm([y], x, None, None, 1e-5)
    for k, v in {"x_out": out, "z": z, "mean": mean, "rstd": rstd}.items():
        close(v, *want[k], k)
    gy.copy_(dz)
    dw = torch.empty(cols, device="cuda")
    kept = out.cpu()
    crc.layer_norm_backward(gy, None, out, mean, rstd, z, dweight=dw)
    want = R.layer_norm_backward(dz, None, kept, mean.cpu(), rstd.cpu(), None)
    close(z, *want["dx"], "dx")
    close(dw, *want["dweight"], "dweight")


@pytest.mark.parametrize("dtype,rows", [(BF16, 1100), (BF16, 100), (BF16, 9), (F32, 1100)])
def test_gated_ffn_of_rows_past_32_bits(dtype, rows):
    """Every matrix in the largest pitch: 4 MiB a row, and outputs in a larger one."""
    cols, wide = 72, 1100
    ld = (1 << 22) // dtype.itemsize
    x, wg, wu = ffn_inputs(rows, cols, wide, dtype)
    gx, gwg, gwu = (far(*t.shape, ld, dtype, t) for t in (x, wg, wu))
    y = far(rows, wide, ld + 8, dtype)
    g, u = (torch.empty(rows, wide, dtype=dtype, device="cuda") for _ in range(2))
    crc.gated_ffn(gx, gwg, gwu, y, gate=g, up=u)
    want = R.gated_ffn(x, wg, wu, "silu")
    for k, v in {"y": y, "gate": g, "up": u}.items():
        close(v, *want[k], k)
    dy = rand(rows, wide, seed=7, dtype=dtype)
    y.copy_(dy)
    dg = far(rows, wide, ld, dtype)
    dx, dwu = torch.empty_like(x, device="cuda"), torch.empty_like(wu, device="cuda")
    dwg = far(wide, cols, ld, dtype)
    crc.gated_ffn_backward(y, g, u, dg, u, x=gx, w_gate=gwg, w_up=gwu, dx=dx, dw_gate=dwg, dw_up=dwu)
    hg, hu, exact = dg.cpu(), u.cpu(), dtype != F32
    close(dx, *R.product(torch.cat([hg, hu], 1), torch.cat([wg, wu], 0).t(), exact), "dx")
    close(dwg, *R.product(hg.t(), x.t(), exact), "dw_gate")
    close(dwu, *R.product(hu.t(), x.t(), exact), "dw_up")


def test_gradients_past_32_bits():
    n = (1 << 31) + 4099  # elements, of 16 bits
    norm = torch.zeros(1, device="cuda")
    t = torch.full((n,), 0.5, dtype=BF16, device="cuda")
    t[-1] = 3.0
    crc.grad_clip([t], 1.0, norm)
    want = math.sqrt(0.25 * (n - 1) + 9.0)
    assert abs(float(norm) / want - 1) < 2.0 ** -23
    for at in (0, 12345, (1 << 31) - 1, 1 << 31, n - 2):
        assert abs(float(t[at]) * want / 0.5 - 1) < 2.0 ** -8, at
    assert abs(float(t[-1]) * want / 3.0 - 1) < 2.0 ** -8
    del t
    rows = far(5, 1000, 1 << 27, F32, rand(5, 1000, seed=3))  # 512 MiB a row
    ref = rows.cpu()
    crc.grad_clip([rows], 1.0, norm)
    close(rows, *R.scaled(ref, R.norm([ref]), 1.0), "rows")


def test_layer_norm_of_many_rows():
    rows = 300_000
    x = rand(rows, 24, seed=1, dtype=F16)
    z, mean, rstd = torch.empty_like(x, device="cuda"), *(torch.empty(rows, device="cuda") for _ in "12")
    crc.layer_norm([], x.cuda(), None, z, mean=mean, rstd=rstd)
    close(z, *R.layer_norm([], x, None, None, 1e-5)["z"], "z")
    dz = rand(rows, 24, seed=2, dtype=F16)
    dx, db = torch.empty_like(z), torch.empty(24, device="cuda")
    crc.layer_norm_backward(dz.cuda(), None, x.cuda(), mean, rstd, dx, dbias=db)
    want = R.layer_norm_backward(dz, None, x, mean.cpu(), rstd.cpu(), None)
    close(dx, *want["dx"], "dx")
    close(db, want["dbias"][0], 2 * want["dbias"][1], "dbias")  # chunks of 300 rows, not 256


def test_kept_in_8_bits_between():
    """The input kept packed: ``checkpoint_wgrad`` takes the projections' gradients."""
    x, wg, wu = ffn_inputs(200, 264, 136, BF16)
    g, u, dy = (rand(200, 136, seed=s, dtype=BF16).cuda() for s in (11, 12, 13))
    kept = crc.checkpoint_empty(200, 264)
    crc.checkpoint_pack(x.cuda(), kept)
    back, dw = torch.empty_like(x, device="cuda"), torch.empty(136, 264, device="cuda")
    dwp = torch.empty_like(dw)
    crc.checkpoint_unpack(kept, back)
    dg, du = torch.empty_like(g), torch.empty_like(g)
    crc.gated_ffn_backward(dy, g, u, dg, du, x=back, dw_up=dw)
    crc.checkpoint_wgrad(du, kept, dwp)
    value, bound = R.product(du.cpu().t(), back.cpu().t(), True)
    close(dw, value, bound, "from what was unpacked")
    close(dwp, value, bound, "from the packed input")


@pytest.mark.parametrize("dtype,ranks,tokens", [("bfloat16", 2, 257), ("float32", 3, 65), ("float16", 1, 300)])
def test_ffn_step_example(dtype, ranks, tokens):
    """A whole training step: every output and gradient against autograd in float32."""
    spec = importlib.util.spec_from_file_location("ffn_step", os.path.join(ROOT, "examples", "ffn_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    apart = example.main(["--tokens", str(tokens), "--width", "264", "--wide", "480", "--ranks", str(ranks),
                          "--dtype", dtype])
    assert len(apart) == 7 + 3 * ranks
    # Each tensor that passes from one operator to the next is rounded to the type,
    # by at most half a step, and some ten of them meet in the last gradient: each
    # adds at most half a step of what it is part of, relative to its size.
    half = torch.finfo(getattr(torch, dtype)).eps / 2
    # float32: sums of up to 480 terms of products, both sides' own
    most = 10 * half if dtype != "float32" else 480 * half
    for name, distance in apart.items():
        assert distance < most, (name, distance)
