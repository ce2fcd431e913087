"""Block-boundary operators and 8-bit checkpoints on the GPU against the 64-bit
reference (tests/block_reference.py), within bounds derived from the roundings
that the formulas leave; nothing outside the outputs is written."""

import sys

import pytest
import torch

import cross_rank_collective_amd as crc
from tests import block_reference as R

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


class Room:
    """A rows x cols tensor inside a larger buffer filled with one byte: `pad`
    elements between rows, `skip` elements before the first."""

    def __init__(self, rows, cols, dtype, pad=0, skip=0, value=None):
        es = torch.empty(0, dtype=dtype).element_size()
        self.buf = torch.full(((64 + skip + rows * (cols + pad) + 64) * es,), 0xA5,
                              dtype=torch.uint8, device="cuda")
        self.t = self.buf.view(dtype).as_strided((rows, cols), (cols + pad, 1), 64 + skip)
        if value is not None:
            self.t.copy_(value)

    def rest_untouched(self):
        copy = self.buf.clone()
        es = self.t.element_size()
        inside = copy.view(self.t.dtype).as_strided(self.t.shape, self.t.stride(),
                                                    self.t.storage_offset())
        inside.copy_(torch.full((es,), 0xA5, dtype=torch.uint8, device="cuda")
                     .view(self.t.dtype).expand(self.t.shape))
        return bool((copy == 0xA5).all())


def draw(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, dtype=torch.float64) * scale


def make(dtype, rows, cols, ranks, post, groups, pre, w32, seed, pad=0, skip=0, offset=0.0):
    """Inputs rounded to their types, on both sides."""
    gen = torch.Generator().manual_seed(seed)
    ty = TYPES[dtype]
    wt = torch.float32 if w32 else ty
    mid = 1.0 - offset
    c = {"x": (draw(gen, rows, cols) * torch.exp(draw(gen, cols, scale=0.7))).to(ty),
         "parts": [draw(gen, rows, cols).to(ty) for _ in range(ranks)],
         "w1": (mid + draw(gen, cols, scale=0.3)).to(wt) if post else None,
         "w2": (mid + draw(gen, cols, scale=0.3)).to(wt) if pre else None,
         "gate": (0.5 + draw(gen, groups, cols, scale=0.5)).to(ty) if groups else None}
    g = {"x": Room(rows, cols, ty, pad, skip, c["x"]).t,
         "parts": [Room(rows, cols, ty, pad, (skip + r) % 5, y).t for r, y in enumerate(c["parts"])],
         "w1": c["w1"].cuda() if post else None, "w2": c["w2"].cuda() if pre else None,
         "gate": Room(groups, cols, ty, pad, skip, c["gate"]).t if groups else None}
    return c, g


def norms(g):
    return {"post_weight": g["w1"], "gate": g["gate"], "pre_weight": g["w2"]}


def check_rest(rooms):
    for name, r in rooms.items():
        assert r.rest_untouched(), f"{name}: bytes outside the output were written"


FORWARD = [
    # dtype, rows, cols, ranks, post, gate rows, pre, 32-bit weights, pad, skip, offset
    ("bf16", 1, 8192, 8, False, 0, True, False, 0, 0, 0.0),
    ("bf16", 1, 1, 1, True, 1, True, True, 0, 0, 0.0),
    ("f32", 1, 1, 2, True, 1, True, True, 3, 1, 1.0),
    ("f16", 3, 7, 3, True, 3, True, False, 1, 1, 0.0),
    ("bf16", 4, 8, 2, True, 2, True, True, 0, 0, 1.0),
    ("bf16", 5, 31, 1, True, 1, True, False, 5, 3, 0.0),
    ("f32", 6, 33, 5, True, 3, True, True, 2, 1, 0.0),
    ("bf16", 9, 511, 4, True, 9, True, True, 1, 1, 0.0),
    ("f16", 16, 512, 7, True, 4, True, False, 8, 0, 1.0),
    ("f32", 7, 513, 2, True, 0, True, True, 0, 2, 0.0),
    ("bf16", 65, 2053, 3, True, 5, True, True, 3, 7, 0.0),
    ("f16", 33, 4096, 2, True, 1, True, True, 0, 0, 0.0),
    ("f32", 12, 4100, 9, True, 12, True, True, 0, 0, 0.0),
    ("bf16", 5, 8200, 2, True, 1, True, True, 0, 0, 0.0),
    ("f32", 3, 8193, 2, True, 3, True, True, 1, 0, 0.0),
    ("bf16", 3, 16384, 2, True, 1, True, False, 0, 0, 0.0),
    ("f16", 2, 16383, 3, True, 2, True, True, 1, 1, 0.0),
    ("f32", 3, 16384, 2, True, 1, True, True, 0, 0, 0.0),
    ("f32", 2, 16381, 2, True, 1, True, True, 3, 3, 0.0),
    ("bf16", 10, 768, 64, True, 2, True, True, 0, 0, 0.0),
    ("bf16", 10, 96, 0, False, 0, True, True, 0, 0, 0.0),
    ("f32", 10, 100, 2, True, 1, False, True, 0, 0, 0.0),
    ("bf16", 10, 100, 2, False, 1, False, True, 0, 0, 0.0),
    ("f16", 300, 1000, 2, False, 300, True, True, 0, 0, 0.0),
]


@pytest.mark.parametrize("case", FORWARD, ids=lambda c: "-".join(map(str, c)))
def test_forward(case):
    dtype, rows, cols, ranks, post, groups, pre, w32, pad, skip, offset = case
    say("forward", *case)
    ty = TYPES[dtype]
    c, g = make(dtype, rows, cols, ranks, post, groups, pre, w32, 11, pad, skip, offset)
    kw = dict(branch_scale=0.6, residual_scale=1.2, weight_offset=offset, eps=EPS)
    out = {"x_out": Room(rows, cols, ty, pad, (skip + 1) % 8)}
    nb = (cols + 31) // 32
    kept = {"x_kept": (Room(rows, cols, torch.int8, pad, skip), Room(rows, nb, torch.uint8, 1, 3))}
    vec = {"post_rstd": Room(1, rows, torch.float32)} if post else {}
    if ranks:
        out["h"] = Room(rows, cols, ty, 0, skip)
        kept["h_kept"] = (Room(rows, cols, torch.int8, 0, 1), Room(rows, nb, torch.uint8))
    if pre:
        out["z"] = Room(rows, cols, ty, pad + 1, skip)
        kept["z_kept"] = (Room(rows, cols, torch.int8, 3, 2), Room(rows, nb, torch.uint8, 0, 1))
        vec["pre_rstd"] = Room(1, rows, torch.float32)
    crc.block_norm(g["parts"], g["x"], **norms(g), **{k: r.t for k, r in out.items()},
                   **{k: (q.t, s.t) for k, (q, s) in kept.items()},
                   **{k: r.t[0] for k, r in vec.items()}, **kw)
    torch.cuda.synchronize()
    want = R.forward(c["parts"], c["x"], c["w1"], c["gate"], c["w2"], eps=EPS, offset=offset,
                     alpha=0.6, beta=1.2)
    for name, room in out.items():
        R.close(room.t, *want[name], name)
    for name, key in (("post_rstd", "r1"), ("pre_rstd", "r2")):
        if name in vec:
            R.close(vec[name].t[0], *want[key], name)
    # the 8-bit forms are exactly those of the outputs as rounded
    for name, (q, s) in kept.items():
        wq, ws = R.pack(out[{"x_kept": "x_out", "h_kept": "h", "z_kept": "z"}[name]].t.cpu())
        assert torch.equal(q.t.cpu(), wq) and torch.equal(s.t.cpu(), ws), name
    check_rest({**out, **vec, **{k + str(i): r for k, p in kept.items() for i, r in enumerate(p)}})
    # with fewer outputs the others keep their bits
    if pre:
        z = Room(rows, cols, ty, 0, 0)
        crc.block_norm(g["parts"], g["x"], z=z.t, **norms(g), **kw)
        assert torch.equal(z.t, out["z"].t)
    # in place on the residual stream, z over a part
    if pre and ranks and pad == 0:
        x = g["x"].clone()
        parts = [p.clone() for p in g["parts"]]
        crc.block_norm(parts, x, x, parts[-1], **norms(g), **kw)
        assert torch.equal(x, out["x_out"].t) and torch.equal(parts[-1], out["z"].t)


def test_forward_rows_do_not_touch_each_other():
    """Zeros, infinities, NaN and huge values stay in their rows."""
    rows, cols = 9, 1000
    c, g = make("bf16", rows, cols, 2, True, 1, True, True, 5)
    y = c["parts"][0]
    y[1], c["parts"][1][1], c["x"][1] = 0, 0, 0
    y[2, 7], y[3, 9], y[4, 0] = float("inf"), float("nan"), -float("inf")
    c["x"][5, 3] = float("inf")
    y[6] *= 1e30  # squares pass binary32's range
    c["x"][7] *= 1e-30
    g["parts"] = [p.cuda() for p in c["parts"]]
    x, z, xo = c["x"].cuda(), torch.empty_like(c["x"], device="cuda"), torch.empty_like(c["x"], device="cuda")
    k = crc.checkpoint_empty(rows, cols)
    crc.block_norm(g["parts"], x, xo, z, **norms(g), eps=EPS, x_kept=k)
    want = R.forward(c["parts"], c["x"], c["w1"], c["gate"], c["w2"], eps=EPS, offset=0.0,
                     alpha=1.0, beta=1.0)
    for i in (0, 1, 7, 8):
        R.close(xo[i], want["x_out"][0][i], want["x_out"][1][i], f"row {i}")
        R.close(z[i], want["z"][0][i], want["z"][1][i], f"row {i}")
    assert torch.isfinite(xo[6]).all() and torch.equal(xo[6].cpu(), c["x"][6])  # r1 = 0: no branch
    for i in (2, 3, 4):
        assert torch.isnan(xo[i]).any()
    assert torch.isnan(z[5]).any()
    q, s = R.pack(xo.cpu())
    assert torch.equal(k.q.cpu(), q) and torch.equal(k.scales.cpu(), s)


BACKWARD = [
    # dtype, rows, cols, post, gate rows, pre, 32-bit weights, packed, pad, skip, offset, dx_out
    ("bf16", 1, 1, True, 1, True, True, False, 0, 0, 0.0, True),
    ("f32", 1, 37, True, 1, True, True, False, 1, 1, 0.0, True),
    ("bf16", 3, 64, True, 3, True, False, True, 0, 0, 1.0, True),
    ("f16", 6, 65, True, 2, True, True, True, 1, 3, 0.0, True),
    ("f32", 8, 100, True, 4, True, True, True, 2, 1, 0.0, False),
    ("bf16", 64, 511, True, 8, True, True, False, 1, 1, 0.0, True),
    ("f16", 257, 96, True, 1, True, False, False, 0, 0, 0.0, True),
    ("bf16", 1025, 160, True, 1, True, True, True, 0, 0, 0.0, True),
    ("f32", 2100, 40, True, 1050, True, True, False, 0, 0, 0.0, True),  # gate rows in pairs
    ("bf16", 4200, 33, True, 600, True, True, True, 1, 0, 0.0, True),  # seven rows a gate row
    ("f16", 3000, 24, True, 3000, True, True, False, 0, 0, 0.0, True),
    ("bf16", 6000, 16, True, 2, True, True, False, 0, 0, 0.0, True),
    ("f32", 33, 2501, True, 3, True, True, False, 3, 2, 0.0, True),
    ("bf16", 20, 4096, True, 1, True, True, True, 0, 0, 0.0, True),
    ("bf16", 5, 8200, True, 1, True, True, False, 0, 0, 0.0, True),
    ("f32", 4, 8193, True, 2, True, True, True, 0, 1, 0.0, True),
    ("f16", 3, 16383, True, 3, True, True, True, 0, 1, 0.0, True),
    ("bf16", 3, 16384, True, 1, True, False, False, 0, 0, 0.0, True),
    ("f32", 3, 16384, True, 1, True, True, False, 0, 0, 0.0, True),
    ("bf16", 40, 128, False, 1, True, True, False, 0, 0, 0.0, True),
    ("bf16", 40, 128, False, 0, True, True, True, 0, 0, 0.0, True),
    ("f32", 40, 130, True, 0, False, True, False, 0, 0, 0.0, True),
    ("f16", 40, 130, False, 4, False, True, True, 0, 0, 0.0, True),
    ("bf16", 40, 130, True, 0, True, False, True, 0, 0, 0.0, False),
]


def grad_case(case, seed=21):
    dtype, rows, cols, post, groups, pre, w32, packed, pad, skip, offset, has_dxo = case
    ty = TYPES[dtype]
    c, g = make(dtype, rows, cols, 1, post, groups, pre, w32, seed, pad, skip, offset)
    gen = torch.Generator().manual_seed(seed + 1)
    c["dz"] = draw(gen, rows, cols).to(ty) if pre else None
    c["dxo"] = draw(gen, rows, cols, scale=0.5).to(ty) if has_dxo else None
    c["r1"] = (0.5 + torch.rand(rows, generator=gen)).float() if post else None
    c["r2"] = (0.5 + torch.rand(rows, generator=gen)).float() if pre else None
    c["h"] = c["parts"][0] if post or groups else None
    c["xo"] = c["x"] if pre else None
    acts = {}
    for name, key in (("x_out", "xo"), ("h", "h")):
        v = c[key]
        if v is None:
            acts[name] = None
        elif packed:
            q, s = R.pack(v.float())
            c[key] = R.unpack(q, s)
            acts[name] = (Room(rows, cols, torch.int8, pad, skip, q).t,
                          Room(rows, s.shape[1], torch.uint8, 1, 1, s).t)
        else:
            acts[name] = Room(rows, cols, ty, pad, skip, v).t
    ins = {n: Room(rows, cols, ty, pad, skip, c[n]).t if c[n] is not None else None
           for n in ("dz", "dxo")}
    vec = {n: c[n].cuda() if c[n] is not None else None for n in ("r1", "r2")}
    return c, g, acts, ins, vec


def run_backward(case, g, acts, ins, vec, **over):
    dtype, rows, cols, post, groups, pre, w32, packed, pad, skip, offset, _ = case
    ty = TYPES[dtype]
    wt = torch.float32 if w32 else ty
    out = {"dx": Room(rows, cols, ty, pad, skip), "dh": Room(rows, cols, ty, pad + 1, 0)}
    if post:
        out["dw1"] = Room(1, cols, wt)
    if pre:
        out["dw2"] = Room(1, cols, wt)
    if groups:
        out["dgate"] = Room(groups, cols, ty, pad, 1)
    kw = dict(dx=out["dx"].t, dh=out["dh"].t, h=acts["h"], post_rstd=vec["r1"],
              dpost_weight=out["dw1"].t[0] if post else None,
              dpre_weight=out["dw2"].t[0] if pre else None,
              dgate=out["dgate"].t if groups else None, branch_scale=0.6, residual_scale=1.2,
              weight_offset=offset, **norms(g))
    crc.block_norm_backward(ins["dz"], ins["dxo"], acts["x_out"], vec["r2"], **{**kw, **over})
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("case", BACKWARD, ids=lambda c: "-".join(map(str, c)))
def test_backward(case):
    say("backward", *case)
    dtype, rows, cols, post, groups, pre, w32, packed, pad, skip, offset, _ = case
    c, g, acts, ins, vec = grad_case(case)
    out = run_backward(case, g, acts, ins, vec)
    want = R.backward(c["dz"], c["dxo"], c["xo"], c["h"], c["r1"], c["r2"], c["w1"], c["gate"],
                      c["w2"], offset=offset, alpha=0.6, beta=1.2)
    for name, room in out.items():
        v, b = want[name]
        R.close(room.t, v.view(room.t.shape), b.view(room.t.shape), name)
    check_rest(out)
    # again: the same bits; and with fewer outputs, the others keep theirs
    again = run_backward(case, g, acts, ins, vec)
    for name, room in out.items():
        assert torch.equal(room.t, again[name].t), name
    few = run_backward(case, g, acts, ins, vec, dgate=None, dpost_weight=None, dpre_weight=None)
    assert torch.equal(few["dx"].t, out["dx"].t)
    assert torch.equal(few["dh"].t, out["dh"].t)
    # in place over the gradients
    if pre and ins["dxo"] is not None:
        run_backward(case, g, acts, ins, vec, dx=ins["dxo"], dh=ins["dz"])
        assert torch.equal(ins["dxo"], out["dx"].t) and torch.equal(ins["dz"], out["dh"].t)


def test_backward_with_a_gate_whose_gradient_is_not_wanted():
    """Chunks then cross gate rows."""
    case = ("bf16", 3000, 40, True, 10, True, True, False, 0, 0, 0.0, True)
    c, g, acts, ins, vec = grad_case(case)
    full = run_backward(case, g, acts, ins, vec)
    some = run_backward(case, g, acts, ins, vec, dgate=None)
    for name in ("dx", "dh"):
        assert torch.equal(full[name].t, some[name].t)
    want = R.backward(c["dz"], c["dxo"], c["xo"], c["h"], c["r1"], c["r2"], c["w1"], c["gate"],
                      c["w2"], offset=0.0, alpha=0.6, beta=1.2)
    for name in ("dw1", "dw2"):
        R.close(some[name].t[0], *want[name], name)


@pytest.mark.parametrize("rows,gate_rows", [(0, 3), (0, 0)])
def test_no_rows_give_zero_gradients(rows, gate_rows):
    cols = 40
    x = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(cols, device="cuda")
    dw1, dw2 = torch.full_like(w, 7), torch.full_like(w, 7)
    gate = torch.ones(gate_rows, cols, device="cuda", dtype=torch.bfloat16) if gate_rows else None
    dg = torch.full_like(gate, 7) if gate_rows else None
    r = torch.empty(0, device="cuda")
    crc.block_norm([x], x.clone(), x.clone(), post_weight=w, gate=gate)
    crc.block_norm_backward(x, x.clone(), x.clone(), r, x.clone(), x.clone(), h=x.clone(),
                            post_rstd=r, post_weight=w, pre_weight=w, gate=gate, dgate=dg,
                            dpost_weight=dw1, dpre_weight=dw2)
    assert not dw1.any() and not dw2.any() and (dg is None or not dg.any())
    dw = torch.full((5, cols), 7.0, device="cuda")
    k = crc.checkpoint_empty(rows, cols)
    dy = torch.empty(rows, 5, device="cuda")
    crc.checkpoint_wgrad(dy, k, dw, accumulate=True)
    assert (dw == 7).all()
    crc.checkpoint_wgrad(dy, k, dw)
    assert not dw.any()
    crc.checkpoint_pack(x, k)
    crc.checkpoint_unpack(k, x)


def test_gradient_against_differences_of_the_forward_kernels():
    """Directional derivatives of c_z z + c_x x' in float32: central
    differences with step s are off by s^2 of the third derivative (about
    1e-4 here) and by the outputs' rounding over s (1e-7 sqrt(n) / s)."""
    torch.manual_seed(2)
    t, d = 4, 48
    v = {"x": torch.randn(t, d), "h": torch.randn(t, d), "w1": 1 + 0.2 * torch.randn(d),
         "w2": 1 + 0.2 * torch.randn(d), "gate": torch.randn(2, d)}
    v = {k: a.cuda() for k, a in v.items()}
    cz, cx = torch.randn(t, d).cuda(), torch.randn(t, d).cuda()
    r1, r2 = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")

    def run(v):
        xo, z = torch.empty(t, d, device="cuda"), torch.empty(t, d, device="cuda")
        crc.block_norm([v["h"]], v["x"], xo, z, post_weight=v["w1"], gate=v["gate"],
                       pre_weight=v["w2"], branch_scale=0.8, residual_scale=1.1, eps=1e-5,
                       post_rstd=r1, pre_rstd=r2)
        return xo, z

    xo, _ = run(v)
    g = {k: torch.empty_like(a) for k, a in v.items()}
    crc.block_norm_backward(cz, cx, xo, r2, g["x"], g["h"], h=v["h"], post_rstd=r1,
                            post_weight=v["w1"], gate=v["gate"], pre_weight=v["w2"],
                            dpost_weight=g["w1"], dgate=g["gate"], dpre_weight=g["w2"],
                            branch_scale=0.8, residual_scale=1.1)

    def loss(v):
        xo, z = run(v)
        return (xo.double() * cx + z.double() * cz).sum()

    step = 5e-3
    for k, a in v.items():
        way = torch.randn_like(a)
        want = (loss({**v, k: a + step * way}) - loss({**v, k: a - step * way})) / (2 * step)
        got = (g[k].double() * way).sum()
        size = (g[k].double().abs() * way.abs()).sum()
        assert abs(got - want) < 1e-3 * size, k


PACK = [("bf16", 1, 1, 0, 0), ("f32", 1, 31, 0, 1), ("f16", 3, 32, 1, 1), ("bf16", 5, 33, 3, 5),
        ("f32", 4, 64, 0, 0), ("f32", 7, 130, 2, 3), ("bf16", 70, 1003, 1, 7), ("f16", 257, 96, 0, 0),
        ("bf16", 33, 20000, 0, 0), ("f32", 2, 40001, 1, 0)]


@pytest.mark.parametrize("case", PACK, ids=lambda c: "-".join(map(str, c)))
def test_pack_and_unpack(case):
    dtype, rows, cols, pad, skip = case
    say("pack", *case)
    ty = TYPES[dtype]
    gen = torch.Generator().manual_seed(4)
    v = (draw(gen, rows, cols) * torch.exp(draw(gen, cols, scale=2.0))).to(ty)
    if rows > 2:
        v[0] = 0
        v[1, cols // 2] = float("nan")
        v[2, 0] = float("inf")
        v[2, -1] = -0.0
    if dtype != "f16" and rows > 3:  # the ends of the exponents
        v[3] = torch.finfo(ty).max * torch.linspace(-1, 1, cols)
        v[-1] = torch.finfo(ty).tiny * torch.linspace(0, 3, cols)
    x = Room(rows, cols, ty, pad, skip, v).t
    q = Room(rows, cols, torch.int8, pad + 2, skip)
    s = Room(rows, (cols + 31) // 32, torch.uint8, 1, 1)
    crc.checkpoint_pack(x, (q.t, s.t))
    wq, ws = R.pack(v.float())
    assert torch.equal(s.t.cpu(), ws)
    assert torch.equal(q.t.cpu(), wq)
    want = R.unpack(wq, ws)
    for name, t in TYPES.items():
        out = Room(rows, cols, t, pad, (skip + 3) % 8)
        crc.checkpoint_unpack((q.t, s.t), out.t)
        R.close(out.t, want, torch.zeros_like(want), f"unpacked to {name}")
        if name != "f16":
            assert torch.equal(out.t.cpu().double().nan_to_num(7.25e-9), want.nan_to_num(7.25e-9))
        check_rest({"out": out})
    check_rest({"q": q, "scales": s})


WGRAD = [
    # dtype, rows, outs, cols, pad, skip, dw of dy's type, accumulate
    ("bf16", 1, 1, 1, 0, 0, False, False), ("f32", 1, 3, 40, 1, 1, True, True),
    ("bf16", 63, 128, 128, 0, 0, False, False), ("bf16", 64, 128, 128, 0, 0, True, False),
    ("bf16", 65, 129, 127, 1, 1, False, True), ("f16", 100, 17, 300, 3, 1, False, False),
    ("f16", 128, 256, 160, 0, 0, True, True), ("f32", 130, 200, 97, 0, 0, False, False),
    ("bf16", 2000, 200, 136, 0, 0, False, True), ("bf16", 5000, 33, 65, 7, 3, True, True),
    ("f16", 3001, 130, 140, 1, 0, False, False), ("f32", 1111, 64, 64, 0, 0, False, True),
    ("bf16", 256, 1000, 1500, 0, 0, False, False),
]


@pytest.mark.parametrize("case", WGRAD, ids=lambda c: "-".join(map(str, c)))
def test_wgrad(case):
    dtype, rows, outs, cols, pad, skip, same, acc = case
    say("wgrad", *case)
    ty = TYPES[dtype]
    gen = torch.Generator().manual_seed(8)
    dy = draw(gen, rows, outs).to(ty)
    q, s = R.pack((draw(gen, rows, cols) * torch.exp(draw(gen, cols))).float())
    old = draw(gen, outs, cols, scale=3.0).to(ty if same else torch.float32)
    dw = Room(outs, cols, old.dtype, pad, skip, old)
    args = (Room(rows, outs, ty, pad, skip, dy).t,
            (Room(rows, cols, torch.int8, pad, skip + 1, q).t, Room(rows, s.shape[1], torch.uint8, 1, 0, s).t),
            dw.t)
    crc.checkpoint_wgrad(*args, accumulate=acc)
    want, bound = R.wgrad(dy, q, s)
    if acc:
        want, bound = want + old.double(), bound + R.U * (want.abs() + old.double().abs())
    R.close(dw.t, want, bound, "dw")
    check_rest({"dw": dw})
    first = dw.t.clone()
    dw.t.copy_(old)
    crc.checkpoint_wgrad(*args, accumulate=acc)
    assert torch.equal(dw.t, first)


def test_wgrad_non_finite_values():
    """An infinity or a NaN of dy reaches its row of dw, a NaN block of x its
    columns, and neither anything else; f32's largest values do not overflow
    on their way through bfloat16."""
    for dtype, ty in TYPES.items():
        rows, outs, cols = 70, 40, 96
        gen = torch.Generator().manual_seed(3)
        dy, x = draw(gen, rows, outs).to(ty), draw(gen, rows, cols).float()
        dy[5, 3], dy[6, 4], dy[7, 20] = float("inf"), float("nan"), -float("inf")
        dy[8, 9] = torch.finfo(ty).max
        if dtype == "f32":
            dy[9, 11] = torch.tensor([0x7F800001], dtype=torch.int32).view(torch.float32)[0]
        x[:, 1] = 1.0
        x[8] /= 4
        x[10, 40] = float("nan")
        q, s = R.pack(x)
        want, bound = R.wgrad(dy, q, s)
        dw = torch.empty(outs, cols, device="cuda")
        crc.checkpoint_wgrad(dy.cuda(), (q.cuda(), s.cuda()), dw)
        finite = torch.isfinite(want)
        assert torch.equal(torch.isnan(dw.cpu()), torch.isnan(want)), dtype
        assert torch.equal(torch.isinf(dw.cpu()), torch.isinf(want)), dtype
        R.close(dw.cpu()[finite], want[finite], bound[finite], dtype)


def test_streams_graphs_and_workspaces():
    """The step on a side stream and replayed from a graph gives the eager
    bits; replays alternate with eager work."""
    t, d, o = 200, 1024, 192
    gen = torch.Generator().manual_seed(6)
    ty = torch.bfloat16
    parts = [draw(gen, t, d).to(ty).cuda() for _ in range(3)]
    x = draw(gen, t, d).to(ty).cuda()
    dz, dxo, dy = (draw(gen, t, n).to(ty).cuda() for n in (d, d, o))
    w1, w2 = ((1 + draw(gen, d, scale=0.2)).float().cuda() for _ in range(2))
    gate = draw(gen, 1, d).to(ty).cuda()

    def room():
        b = {n: torch.zeros(t, d, dtype=ty, device="cuda") for n in ("xo", "z", "dx", "dh")}
        b |= {"dw1": torch.zeros(d, device="cuda"), "dw2": torch.zeros(d, device="cuda"),
              "dg": torch.zeros(1, d, dtype=ty, device="cuda"),
              "dw": torch.zeros(o, d, device="cuda"), "r1": torch.zeros(t, device="cuda"),
              "r2": torch.zeros(t, device="cuda")}
        kept = [crc.checkpoint_empty(t, d) for _ in range(3)]
        ws = torch.empty(max(crc.block_norm_backward_workspace(t, d, 1),
                             crc.checkpoint_wgrad_workspace(t, o, d, ty)), dtype=torch.uint8,
                         device="cuda")
        return b, kept, ws

    def step(b, kept, ws, stream=None):
        n = dict(post_weight=w1, gate=gate, pre_weight=w2, branch_scale=0.5)
        crc.block_norm(parts, x, b["xo"], b["z"], post_rstd=b["r1"], pre_rstd=b["r2"],
                       h_kept=kept[0], x_kept=kept[1], z_kept=kept[2], stream=stream, **n)
        crc.block_norm_backward(dz, dxo, kept[1], b["r2"], b["dx"], b["dh"], h=kept[0],
                                post_rstd=b["r1"], dpost_weight=b["dw1"], dgate=b["dg"],
                                dpre_weight=b["dw2"], workspace=ws, stream=stream, **n)
        crc.checkpoint_wgrad(dy, kept[2], b["dw"], workspace=ws, stream=stream)

    eager = room()
    step(*eager)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        other = room()
        side.wait_stream(torch.cuda.current_stream())
        step(other[0], other[1], None, stream=stream)
        side.synchronize()
        for n, v in eager[0].items():
            assert torch.equal(v, other[0][n]), n
    cap = room()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*cap)
    for _ in range(4):
        for v in cap[0].values():
            v.zero_()
        graph.replay()
        step(*eager)
        torch.cuda.synchronize()
        for n, v in eager[0].items():
            assert torch.equal(v, cap[0][n]), n


def test_tensor_checks():
    x = torch.zeros(8, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda")
    bad = [
        lambda: crc.block_norm([x[:4]], x, x.clone()),
        lambda: crc.block_norm([x.float()], x, x.clone()),
        lambda: crc.block_norm([x.t().contiguous().t()], x, x.clone()),
        lambda: crc.block_norm([x, torch.zeros(8, 72, device="cuda", dtype=x.dtype)[:, :64]], x),
        lambda: crc.block_norm([x], x, x.clone(), z=x.clone(), pre_weight=w[:63]),
        lambda: crc.block_norm([x], x, gate=torch.ones(3, 64, device="cuda", dtype=x.dtype)),
        lambda: crc.block_norm([x], x, gate=x[:1].expand(8, 64)),
        lambda: crc.block_norm([x], x, x_kept=(x, x)),
        lambda: crc.block_norm([x], x, post_weight=w, pre_weight=w.bfloat16()),
        lambda: crc.block_norm_backward(x, x.clone(), (x, x), w, h=x.clone()),
        lambda: crc.checkpoint_wgrad(x, crc.checkpoint_empty(7, 64), torch.zeros(64, 64, device="cuda")),
        lambda: crc.checkpoint_wgrad(x, crc.checkpoint_empty(8, 64), torch.zeros(63, 64, device="cuda")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was taken")
    with pytest.raises(TypeError):
        crc.block_norm([x], x, post_weight=w.half())
    with pytest.raises(crc.PtoredError):  # outputs over each other
        o = x.clone()
        crc.block_norm([x], x, o, o, pre_weight=w)


def test_offsets_past_32_bits():
    """Rows whose byte offsets pass 2^32, in every operator that has them: a
    few rows far apart."""
    rows, cols, pitch = 3, 4096, 1 << 31
    buf = torch.empty((rows - 1) * pitch + cols, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((rows, cols), (pitch, 1))
    gen = torch.Generator().manual_seed(12)
    v, y = draw(gen, rows, cols).bfloat16(), draw(gen, rows, cols).bfloat16()
    far.copy_(v)
    w = torch.ones(cols, device="cuda")
    z, z2 = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda"), None
    crc.block_norm([y.cuda()], far, far, z, pre_weight=w)
    want = R.forward([y], v, None, None, w.cpu(), eps=EPS, offset=0.0, alpha=1.0, beta=1.0)
    R.close(far, *want["x_out"], "x_out")
    R.close(z, *want["z"], "z")
    k = crc.checkpoint_empty(rows, cols)
    crc.checkpoint_pack(far, k)
    near = torch.empty_like(z)
    crc.checkpoint_unpack(k, near)
    crc.checkpoint_unpack(k, far)
    assert torch.equal(far, near)
    dw = torch.empty(64, cols, device="cuda")
    dw2 = torch.empty(cols, cols, device="cuda")
    crc.checkpoint_wgrad(far, k, dw2)
    far2 = near.contiguous()
    dw3 = torch.empty(cols, cols, device="cuda")
    crc.checkpoint_wgrad(far2, k, dw3)
    assert torch.equal(dw2, dw3)
    del dw
