"""Block-boundary calls on the GPU as callers make them: the C ABI's own
conventions, buffers reused in place or far apart, values at the ends of the
types' ranges.  References and bounds as in tests/test_block_gpu.py."""

import ctypes

import pytest
import torch

import cross_rank_collective_amd as crc
from cross_rank_collective_amd import block as K
from tests import block_reference as R
from tests.test_block_gpu import EPS, TYPES, draw, make, norms, say

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
