"""Block-boundary calls on the GPU as callers make them: the C ABI's own
conventions, buffers reused in place or far apart, values at the ends of the
types' ranges.  References and bounds as in tests/test_block_gpu.py."""

import ctypes

import pytest
import torch

import cross_rank_collective_amd as crc
from cross_rank_collective_amd import block as K
from tests import block_reference as R
from tests.test_block_gpu import (EPS, TYPES, Room, check_rest, draw, grad_case, make, norms,
                                  run_backward, say)

pytestmark = pytest.mark.gpu


def raw_backward(params, **kw):
    """The C call: tensors, or what the structure takes, by field."""
    v = {n: None if t is ctypes.c_void_p else t() for n, t in K.ptored_block_grad_io._fields_}
    for n, a in kw.items():
        if not isinstance(a, torch.Tensor):
            v[n] = a
        elif a.dim() == 2:
            v[n] = K.ptored_rows(a.data_ptr(), a.stride(0))
        else:
            v[n] = a.data_ptr()
    io = K.ptored_block_grad_io(*[v[n] for n, _ in K.ptored_block_grad_io._fields_])
    status = crc.ptored_block_norm_backward(params, io, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return status


def test_gate_rows_are_not_read_without_a_gate():
    rows, cols = 64, 264
    say("no gate", rows, cols)
    gen = torch.Generator().manual_seed(7)
    dz, dxo, x, h = (draw(gen, rows, cols).bfloat16().cuda() for _ in range(4))
    w1, w2 = (draw(gen, cols).float().cuda() for _ in range(2))
    r1, r2 = (0.5 + torch.rand(rows, generator=gen).cuda() for _ in range(2))
    ws = torch.empty(crc.block_norm_backward_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    outs = []
    for left in (0, 1, 4, 3, -1):
        p = K.ptored_block_params(rows, cols, w1.data_ptr(), w2.data_ptr(), K.ptored_rows(), left, 0.0,
                                  0.7, 1.0, 1e-6, 1, 0)
        out = {"dx": torch.empty_like(dz), "dh": torch.empty_like(dz),
               "dpost_weight": torch.empty_like(w1), "dpre_weight": torch.empty_like(w1)}
        assert raw_backward(p, dz=dz, dx_out=dxo, x_out=x, h=h, post_rstd=r1, pre_rstd=r2,
                            workspace=ws, workspace_bytes=ws.numel(), **out) == 0
        outs.append(out)
    for other in outs[1:]:
        for name, v in outs[0].items():
            assert torch.equal(v, other[name]), name


# Sums of squares that pass binary32's range with a mean that does not, in both
# norms; columns and rows of every kernel.
LARGE = [("bf16", 5, 8192, False), ("bf16", 300, 4100, True), ("f32", 4, 7, True), ("f32", 300, 1003, False),
         ("f32", 257, 16384, True), ("bf16", 3, 16383, False), ("f32", 3, 4096, True)]


@pytest.mark.parametrize("dtype,rows,cols,keep", LARGE)
def test_squares_whose_sum_passes_the_range_but_not_their_mean(dtype, rows, cols, keep):
    say("large", dtype, rows, cols, keep)
    ty = TYPES[dtype]
    c, g = make(dtype, rows, cols, 2, True, 1, True, True, 17)
    # magnitudes 0.5 to 1 times the scale, so that the mean square is known to hold
    flat = lambda v: (v.double().sign() * (0.5 + 0.5 * torch.rand(v.shape)) + 0).to(v.dtype)  # noqa: E731
    torch.manual_seed(4)
    c["parts"] = [flat(v) for v in c["parts"]]
    c["x"] = flat(c["x"])
    c["parts"][0][0] *= 1.6e19  # the fold's row: mean square near 1e38
    c["parts"][1][0] *= 1e10
    c["x"][1] *= 1.6e19         # the stream's row
    c["parts"][0][rows - 1] *= 3e17
    c["x"][rows - 1] *= 3e17
    g["parts"], g["x"] = [v.cuda() for v in c["parts"]], c["x"].cuda()
    out = {n: torch.empty(rows, cols, dtype=ty, device="cuda") for n in ("x_out", "z", "h")}
    vec = {n: torch.empty(rows, device="cuda") for n in ("post_rstd", "pre_rstd")}
    kept = {n: crc.checkpoint_empty(rows, cols) for n in ("x_kept", "z_kept")} if keep else {}
    crc.block_norm(g["parts"], g["x"], **out, **vec, **kept, eps=EPS, **norms(g))
    want = R.forward(c["parts"], c["x"], c["w1"], c["gate"], c["w2"], eps=EPS, offset=0.0, alpha=1.0,
                     beta=1.0)
    assert float(want["r1"][0].min()) > 0 and float(want["r2"][0].min()) > 0
    for name, key in (("h", "h"), ("post_rstd", "r1"), ("x_out", "x_out"), ("pre_rstd", "r2"), ("z", "z")):
        R.close({**out, **vec}[name], *want[key], name)
    for name, k in kept.items():
        q, s = R.pack(out[{"x_kept": "x_out", "z_kept": "z"}[name]].cpu())
        assert torch.equal(k.q.cpu(), q) and torch.equal(k.scales.cpu(), s), name


@pytest.mark.parametrize("native", [True, False])
def test_one_row_of_buffers_with_different_pitches(native, monkeypatch):
    """A decoded token's partial outputs, each a row of a buffer of its own width."""
    say("one row", native)
    if not native:
        monkeypatch.setattr(K, "_native_call", lambda *a: False)
    cols = 520
    c, g = make("bf16", 1, cols, 3, False, 0, True, True, 3)
    wide = [torch.zeros(4, cols + 8 * r, dtype=torch.bfloat16, device="cuda") for r in range(3)]
    parts = [w[r:r + 1, :cols] for r, w in enumerate(wide)]
    for p, v in zip(parts, c["parts"]):
        p.copy_(v)
    assert len({p.stride(0) for p in parts}) == 3
    x, z = torch.empty(1, 2 * cols, dtype=torch.bfloat16, device="cuda")[:, :cols], torch.empty(
        1, cols, dtype=torch.bfloat16, device="cuda")
    x.copy_(c["x"])
    # x' over the same row seen with another pitch
    crc.block_norm(parts, x, x.as_strided((1, cols), (cols, 1)), z, pre_weight=g["w2"], eps=EPS)
    want = R.forward(c["parts"], c["x"], None, None, c["w2"], eps=EPS, offset=0.0, alpha=1.0, beta=1.0)
    R.close(x, *want["x_out"], "x_out")
    R.close(z, *want["z"], "z")


@pytest.mark.parametrize("native", [True, False])
def test_outputs_count_as_changed_in_place(native, monkeypatch):
    """Every output's version moves on and no input's; a tensor that autograd
    saved before a call wrote it is refused by the backward pass."""
    say("versions", native)
    if not native:
        monkeypatch.setattr(K, "_native_call", lambda *a: False)
    t, d, o = 6, 40, 16
    rand = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    ins = {n: rand(t, d) for n in ("y", "x", "dz", "dxo")} | {
        "w1": rand(d), "w2": rand(d), "gate": rand(2, d), "dy": rand(t, o)}
    outs = {n: rand(t, d) for n in ("xo", "z", "h", "dx", "dh", "back")} | {
        "r1": rand(t), "r2": rand(t), "dw1": rand(d), "dw2": rand(d), "dg": rand(2, d), "dw": rand(o, d)}
    kept = {n: crc.checkpoint_empty(t, d) for n in "hxzp"}
    flat = lambda: list(ins.values()), lambda: [*outs.values(), *(v for k in kept.values() for v in k)]
    before = [[v._version for v in f()] for f in flat]
    n = {"post_weight": ins["w1"], "gate": ins["gate"], "pre_weight": ins["w2"]}
    crc.block_norm([ins["y"]], ins["x"], outs["xo"], outs["z"], h=outs["h"], post_rstd=outs["r1"],
                   pre_rstd=outs["r2"], h_kept=kept["h"], x_kept=kept["x"], z_kept=kept["z"], **n)
    crc.block_norm_backward(ins["dz"], ins["dxo"], kept["x"], outs["r2"], outs["dx"], outs["dh"],
                            h=kept["h"], post_rstd=outs["r1"], dpost_weight=outs["dw1"],
                            dgate=outs["dg"], dpre_weight=outs["dw2"], **n)
    crc.checkpoint_pack(ins["x"], kept["p"])
    crc.checkpoint_unpack(kept["p"], outs["back"])
    crc.checkpoint_wgrad(ins["dy"], kept["z"], outs["dw"])
    after = [[v._version for v in f()] for f in flat]
    assert after[0] == before[0]
    assert after[1] == [v + 1 for v in before[1]]

    proj = rand(d, o).requires_grad_()
    loss = (outs["z"] @ proj).sum()  # saves z
    crc.block_norm([ins["y"]], ins["x"], z=outs["z"], pre_weight=ins["w2"])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        z = rand(t, d)
        crc.block_norm([ins["y"]], ins["x"], z=z, pre_weight=ins["w2"])
    crc.block_norm([ins["y"]], ins["x"], z=z, pre_weight=ins["w2"])  # its tensors have no versions


# As in test_block_gpu.BACKWARD, activations whole: rows of several waves, several
# rows a workgroup, ends inside a slot, with and without the norms.
IN_PLACE = [
    ("bf16", 601, 4099, True, 601, True, False, False, 1, 1, 1.0, True),
    ("bf16", 521, 8192, True, 0, True, False, False, 0, 0, 0.0, True),
    ("bf16", 280, 9000, False, 1, True, True, False, 0, 0, 0.0, True),
    ("bf16", 1540, 4104, True, 220, True, True, False, 0, 0, 0.0, True),
    ("f32", 300, 8196, True, 1, True, True, False, 0, 0, 0.0, False),
    ("f32", 1400, 1003, True, 20, True, True, False, 0, 1, 0.0, True),
    ("f32", 300, 12001, True, 0, False, True, False, 1, 0, 0.0, True),
    ("f16", 6600, 39, False, 600, True, False, False, 0, 0, 1.0, True),
    ("f16", 3000, 3, True, 3, True, True, False, 1, 1, 0.0, True),
    ("f16", 900, 1025, False, 4, False, True, False, 0, 0, 0.0, True),
]


@pytest.mark.parametrize("case", IN_PLACE, ids=lambda c: "-".join(map(str, c)))
def test_gradients_over_the_activations(case):
    say("in place", *case)
    _, g, acts, ins, vec = grad_case(case)
    full = run_backward(case, g, acts, ins, vec)
    have = [n for n, v in (("x_out", acts["x_out"]), ("h", acts["h"]), ("dz", ins["dz"]),
                           ("dxo", ins["dxo"])) if v is not None]
    for dx, dh in [(have[0], have[1]), (have[1], have[0]), (have[-1], have[0])]:
        _, g, acts, ins, vec = grad_case(case)
        bufs = {**acts, **ins}
        out = run_backward(case, g, acts, ins, vec, dx=bufs[dx], dh=bufs[dh])
        assert torch.equal(bufs[dx], full["dx"].t), (dx, dh)
        assert torch.equal(bufs[dh], full["dh"].t), (dx, dh)
        for name in ("dw1", "dw2", "dgate"):
            if name in out:
                assert torch.equal(out[name].t, full[name].t), (name, dx, dh)


def far(rows, cols, dtype, value=None):
    """Rows further apart than 2^31 bytes: the third one's offset passes 2^32."""
    pitch = (1 << 31) // torch.empty(0, dtype=dtype).element_size() + 8
    buf = torch.empty((rows - 1) * pitch + cols, dtype=dtype, device="cuda")
    t = buf.as_strided((rows, cols), (pitch, 1))
    if value is not None:
        t.copy_(value)
    return t


@pytest.mark.parametrize("packed,groups", [(False, 3), (True, 1)])
def test_gradients_of_rows_past_32_bits(packed, groups):
    """All matrices far apart, the packed ones and the gate among them."""
    say("far gradients", packed, groups)
    rows, cols = 3, 4100
    case = ("bf16", rows, cols, True, groups, True, True, packed, 0, 0, 0.0, True)
    _, g, acts, ins, vec = grad_case(case)
    near = run_backward(case, g, acts, ins, vec)
    move = lambda v: far(*v.shape, v.dtype, v)  # noqa: E731
    acts = {n: tuple(move(t) for t in v) if packed else move(v) for n, v in acts.items()}
    ins = {n: move(v) for n, v in ins.items()}
    g["gate"] = move(g["gate"])
    dx, dh = (far(rows, cols, torch.bfloat16) for _ in range(2))
    dgate = far(groups, cols, torch.bfloat16)
    out = run_backward(case, g, acts, ins, vec, dx=dx, dh=dh, dgate=dgate)
    for name, v in (("dx", dx), ("dh", dh), ("dgate", dgate), ("dw1", out["dw1"].t), ("dw2", out["dw2"].t)):
        assert torch.equal(v, near[name].t), name
    del acts, ins, dx, dh, dgate, g
    torch.cuda.empty_cache()


def test_forward_and_weight_gradient_of_rows_past_32_bits():
    """Partials, stream, gate and every output of the forward pass; the packed
    input and the weight gradient."""
    say("far forward")
    rows, cols, outs = 3, 2052, 8
    c, g = make("bf16", rows, cols, 2, True, 3, True, True, 13)
    like = lambda n, d: torch.empty(rows, n, dtype=d, device="cuda")  # noqa: E731
    nb = (cols + 31) // 32
    out = {n: like(cols, torch.bfloat16) for n in ("x_out", "z", "h")}
    kept = {n: (like(cols, torch.int8), like(nb, torch.uint8)) for n in ("x_kept", "z_kept", "h_kept")}
    crc.block_norm(g["parts"], g["x"], **out, **kept, **norms(g))
    dy = draw(torch.Generator().manual_seed(1), rows, outs).bfloat16().cuda()
    dw = torch.empty(outs, cols, device="cuda")
    crc.checkpoint_wgrad(dy, kept["z_kept"], dw)

    moved = {n: far(rows, cols, torch.bfloat16) for n in out}
    packs = {n: (far(rows, cols, torch.int8), far(rows, nb, torch.uint8)) for n in kept}
    parts = [far(rows, cols, torch.bfloat16, v) for v in g["parts"]]
    n = {**norms(g), "gate": far(3, cols, torch.bfloat16, g["gate"])}
    crc.block_norm(parts, far(rows, cols, torch.bfloat16, g["x"]), **moved, **packs, **n)
    for name, v in out.items():
        assert torch.equal(moved[name], v), name
    for name, pair in kept.items():
        for a, b in zip(packs[name], pair):
            assert torch.equal(a, b), name
    del moved, parts, n
    torch.cuda.empty_cache()
    wide = far(outs, cols, torch.float32)
    crc.checkpoint_wgrad(dy, packs["z_kept"], wide)
    assert torch.equal(wide, dw)
    del wide, packs
    torch.cuda.empty_cache()


# f16, where a workgroup that meets a block of x outside f16's exponents starts
# again: tiles of 256 x 256 and of 128 x 128, tokens split, rows shorter than a chunk.
RESTART = [(200, 2997, 4008), (200, 2048, 4096), (300, 136, 160), (4096, 130, 131), (129, 200, 15),
           (700, 3, 300), (2001, 7, 9)]


@pytest.mark.parametrize("rows,outs,cols", RESTART)
def test_wgrad_of_f16_starts_again(rows, outs, cols):
    gen = torch.Generator().manual_seed(38)
    dy = torch.randn(rows, outs, generator=gen).half()
    x = torch.randn(rows, cols, generator=gen)
    spots = {"first": (0, 0), "middle": (rows // 2, cols // 2), "last": (rows - 1, cols - 1)}
    for name, (t, i) in spots.items():
        for scale in (2.0 ** 40, 2.0 ** -60, float("nan")):
            say("f16 restart", rows, outs, cols, name, scale)
            v = x.clone()
            block = slice(i // 32 * 32, i // 32 * 32 + 32)
            v[t, block] *= scale
            q, s = R.pack(v)
            want, bound = R.wgrad(dy, q, s)
            dw = Room(outs, cols, torch.float32, 1, 1)
            crc.checkpoint_wgrad(dy.cuda(), (q.cuda(), s.cuda()), dw.t)
            R.close(dw.t, want, bound, f"{name} {scale}")
            check_rest({"dw": dw})


@pytest.mark.parametrize("rows,outs,cols", [(300, 136, 160), (33, 5, 40), (2500, 300, 520)])
def test_wgrad_of_f32s_smallest_values(rows, outs, cols):
    """dy below 2^-110 enters as a multiple of 2^-133 (of bfloat16's smallest
    step), off by less than one; the products' sums are binary32's, whose
    smallest step is 2^-149."""
    for low, high in ((2.0 ** -119, 2.0 ** 3), (2.0 ** -130, 2.0 ** 70), (2.0 ** -140, 2.0 ** 100)):
        say("f32 smallest", rows, outs, cols, low)
        gen = torch.Generator().manual_seed(48)
        dy = (draw(gen, rows, outs) * low).float()
        q, s = R.pack((draw(gen, rows, cols) * high).float())
        want, bound = R.wgrad(dy, q, s)
        bound = bound + 2.0 ** -133 * R.unpack(q, s).abs().sum(0) + rows * 2.0 ** -149
        dw = torch.empty(outs, cols, device="cuda")
        crc.checkpoint_wgrad(dy.cuda(), (q.cuda(), s.cuda()), dw)
        R.close(dw, want, bound, f"dy of {low}")
