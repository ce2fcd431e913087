"""Block-boundary operators on the GPU at the sizes where their kernels change:
many rows and few, rows that end inside a slot or a vector, chunks that
interleave rows, tiles of every shape, tokens split and not, f16's range; and
the two ways a call takes from Python.  References and bounds as in
tests/test_block_gpu.py."""

import pytest
import torch

import cross_rank_collective_amd as crc
from cross_rank_collective_amd import block as K
from tests import block_reference as R
from tests.test_block_gpu import (EPS, TYPES, Room, check_rest, draw, grad_case, make, norms,
                                  run_backward, say)

pytestmark = pytest.mark.gpu


# More than 256 rows take 16 elements a thread (bf16, f16: 2 slots; f32: 4),
# fewer when the row is short: columns around every change, and around the
# workgroups of 64 threads.
MANY_ROWS = [("bf16", c) for c in (1, 7, 9, 510, 512, 520, 1016, 1025, 1032, 2049, 8191, 16383, 16384)]
MANY_ROWS += [("f32", c) for c in (3, 5, 256, 260, 516, 767, 772, 1021, 3077, 4097, 16381)]
MANY_ROWS += [("f16", c) for c in (15, 1000, 4095)]


@pytest.mark.parametrize("dtype,cols", MANY_ROWS)
def test_forward_of_many_rows(dtype, cols):
    rows, ranks = 258, 5
    say("many rows", dtype, cols)
    ty = TYPES[dtype]
    c, g = make(dtype, rows, cols, ranks, True, 3, True, dtype != "f16", 31, 1, 3, 1.0)
    kw = dict(branch_scale=0.6, residual_scale=1.2, weight_offset=1.0, eps=EPS)
    nb = (cols + 31) // 32
    out = {n: Room(rows, cols, ty, 1, i) for i, n in enumerate(("x_out", "z", "h"))}
    kept = {n: (Room(rows, cols, torch.int8, 1, i), Room(rows, nb, torch.uint8, 1, i))
            for i, n in enumerate(("x_kept", "z_kept", "h_kept"))}
    vec = {n: Room(1, rows, torch.float32) for n in ("post_rstd", "pre_rstd")}
    crc.block_norm(g["parts"], g["x"], **norms(g), **{k: r.t for k, r in out.items()},
                   **{k: (q.t, s.t) for k, (q, s) in kept.items()},
                   **{k: r.t[0] for k, r in vec.items()}, **kw)
    torch.cuda.synchronize()
    want = R.forward(c["parts"], c["x"], c["w1"], c["gate"], c["w2"], eps=EPS, offset=1.0,
                     alpha=0.6, beta=1.2)
    for name, room in out.items():
        R.close(room.t, *want[name], name)
    for name, key in (("post_rstd", "r1"), ("pre_rstd", "r2")):
        R.close(vec[name].t[0], *want[key], name)
    for name, (q, s) in kept.items():
        wq, ws = R.pack(out[{"x_kept": "x_out", "h_kept": "h", "z_kept": "z"}[name]].t.cpu())
        assert torch.equal(q.t.cpu(), wq) and torch.equal(s.t.cpu(), ws), name
    check_rest({**out, **vec, **{k + str(i): r for k, p in kept.items() for i, r in enumerate(p)}})
    # the same without what is kept, which another kernel does
    z = torch.empty(rows, cols, dtype=ty, device="cuda")
    crc.block_norm(g["parts"], g["x"], z=z, **norms(g), **kw)
    assert torch.equal(z, out["z"].t)


def test_forward_of_more_rows_than_a_launch_has():
    """2^25 workgroups of one wave are a launch's limit; the rows past them are
    the same workgroups' second."""
    rows, cols = (1 << 25) + 77, 8
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    y = torch.empty_like(x).normal_()
    w = torch.full((cols,), 1.5, device="cuda")
    z = torch.empty_like(x)
    crc.block_norm([y], x, z=z, post_weight=w, pre_weight=w)
    for at in (slice(0, 100), slice((1 << 25) - 50, rows)):
        want = R.forward([y[at].cpu()], x[at].cpu(), w.cpu(), None, w.cpu(), eps=EPS, offset=0.0,
                         alpha=1.0, beta=1.0)
        R.close(z[at], *want["z"], str(at))


# As in test_block_gpu.BACKWARD; rows past the number of workgroups, so that
# each takes several, interleaved.
CHUNKS = [
    ("bf16", 700, 4104, True, 1, True, True, True, 0, 0, 0.0, True),
    ("bf16", 521, 8192, True, 0, True, False, False, 0, 0, 0.0, True),
    ("f16", 600, 4100, True, 600, True, True, True, 4, 0, 0.0, True),   # a gate row each
    ("bf16", 601, 4099, True, 601, True, False, False, 1, 1, 1.0, True),
    ("bf16", 1536, 4104, True, 512, True, True, True, 0, 0, 0.0, True),  # three rows a gate row
    ("f32", 800, 2052, True, 2, True, True, False, 0, 0, 0.0, True),
    ("f32", 700, 4100, True, 700, True, True, True, 1, 0, 0.0, True),
    ("f32", 300, 8196, True, 1, True, True, False, 0, 0, 0.0, False),
    ("bf16", 300, 16376, True, 300, True, True, True, 0, 0, 0.0, True),
    ("bf16", 280, 9000, False, 1, True, True, False, 0, 0, 0.0, True),
    # few columns and many chunks, joined by narrower workgroups
    ("bf16", 3000, 747, True, 2, True, True, True, 0, 0, 0.0, True),
    ("f16", 5000, 36, True, 5, True, False, True, 1, 1, 1.0, True),
    ("f32", 2100, 1003, True, 1, True, True, False, 0, 0, 0.0, True),
    # many gate rows of a few chunks each, few of them, and some of many chunks
    ("bf16", 1040, 520, True, 65, True, True, True, 1, 0, 0.0, True),
    ("f32", 1400, 1003, True, 40, True, True, False, 0, 1, 0.0, True),
    ("f16", 6600, 39, False, 600, True, False, False, 0, 0, 1.0, True),
    ("f32", 1400, 1003, True, 20, True, True, False, 0, 1, 0.0, True),
    ("bf16", 4000, 259, True, 5, False, True, True, 0, 0, 0.0, True),
]


@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: "-".join(map(str, c)))
def test_backward_of_several_rows_a_workgroup(case):
    say("chunks", *case)
    offset = case[10]
    c, g, acts, ins, vec = grad_case(case)
    out = run_backward(case, g, acts, ins, vec)
    want = R.backward(c["dz"], c["dxo"], c["xo"], c["h"], c["r1"], c["r2"], c["w1"], c["gate"],
                      c["w2"], offset=offset, alpha=0.6, beta=1.2)
    for name, room in out.items():
        v, b = want[name]
        R.close(room.t, v.view(room.t.shape), b.view(room.t.shape), name)
    check_rest(out)
    if case[4] > 1:  # without the gate's gradient the rows are cut otherwise
        some = run_backward(case, g, acts, ins, vec, dgate=None)
        for name in ("dx", "dh"):
            assert torch.equal(some[name].t, out[name].t), name
        for name in ("dw1", "dw2"):
            if name in some:
                R.close(some[name].t[0], *want[name], name)


@pytest.mark.parametrize("case", [c for c in CHUNKS if c[4] > 1],
                         ids=lambda c: "-".join(map(str, c)))
def test_a_gates_gradient_alone_keeps_its_bits(case):
    say("gate alone", *case)
    _, g, acts, ins, vec = grad_case(case)
    full = run_backward(case, g, acts, ins, vec)
    alone = run_backward(case, g, acts, ins, vec, dx=None, dh=None, dpost_weight=None,
                         dpre_weight=None)
    assert torch.equal(alone["dgate"].t, full["dgate"].t)
    check_rest(alone)


def test_backward_without_a_norm_after_the_block_passes_an_infinite_fold():
    """Without the norm dh does not depend on h: its infinities reach the
    gate's gradient alone."""
    rows, cols = 6, 40
    gen = torch.Generator().manual_seed(5)
    h = draw(gen, rows, cols).bfloat16()
    h[2, 3] = float("inf")
    dxo = draw(gen, rows, cols).bfloat16()
    gate = draw(gen, 1, cols).bfloat16()
    dx, dh = (torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dg = torch.empty(1, cols, dtype=torch.bfloat16, device="cuda")
    crc.block_norm_backward(None, dxo.cuda(), None, None, dx, dh, h=h.cuda(), gate=gate.cuda(),
                            dgate=dg)
    assert torch.equal(dx.cpu(), dxo)
    assert torch.equal(dh.cpu(), (dxo.float() * gate.float()).bfloat16())
    finite = torch.isfinite(dg.cpu()[0])
    assert not finite[3] and int(finite.sum()) == cols - 1


# Four slots a thread from 2^20 slots on; rows narrower than a workgroup.
@pytest.mark.parametrize("dtype,rows,cols", [("bf16", 4100, 2050), ("f32", 3000, 1403),
                                             ("f16", 150000, 40), ("bf16", 300000, 5),
                                             ("f32", 5, 900000)])
def test_pack_of_many_slots(dtype, rows, cols):
    say("pack", dtype, rows, cols)
    ty = TYPES[dtype]
    gen = torch.Generator().manual_seed(9)
    v = torch.randn(rows, cols, generator=gen).to(ty)
    x = Room(rows, cols, ty, 1, 2, v).t
    q = Room(rows, cols, torch.int8, 3, 1)
    s = Room(rows, (cols + 31) // 32, torch.uint8, 1, 1)
    crc.checkpoint_pack(x, (q.t, s.t))
    wq, ws = R.pack(v.float())
    assert torch.equal(s.t.cpu(), ws)
    assert torch.equal(q.t.cpu(), wq)
    out = Room(rows, cols, torch.float32, 1, 1)
    crc.checkpoint_unpack((q.t, s.t), out.t)
    assert torch.equal(out.t.cpu().double(), R.unpack(wq, ws))
    check_rest({"q": q, "scales": s, "out": out})


WGRAD_TILES = [
    # dtype, rows, outs, cols, pad: 256 x 256 tiles, their edges
    ("bf16", 200, 3000, 4000, 0), ("bf16", 131, 3001, 3999, 1), ("f16", 200, 2997, 4008, 0),
    ("f32", 97, 2050, 2049, 1),
    # tokens split, with and without whole steps
    ("bf16", 3333, 640, 512, 0), ("f16", 4096, 130, 131, 1), ("f32", 2500, 300, 520, 0),
    ("bf16", 9001, 64, 64, 0), ("f16", 1001, 777, 130, 1),
    # rows shorter than a chunk
    ("bf16", 700, 3, 300, 1), ("f16", 129, 200, 15, 0), ("f32", 300, 7, 5, 2), ("bf16", 65, 8, 16, 0),
    ("f32", 64, 9, 17, 0), ("bf16", 1, 300, 300, 0), ("f16", 2, 129, 257, 1),
]


@pytest.mark.parametrize("case", WGRAD_TILES, ids=lambda c: "-".join(map(str, c)))
def test_wgrad_tiles(case):
    dtype, rows, outs, cols, pad = case
    say("wgrad tiles", *case)
    ty = TYPES[dtype]
    gen = torch.Generator().manual_seed(18)
    dy = torch.randn(rows, outs, generator=gen).to(ty)
    q, s = R.pack((torch.randn(rows, cols, generator=gen) * torch.exp(torch.randn(cols, generator=gen))))
    dw = Room(outs, cols, torch.float32, pad, 1)
    args = (Room(rows, outs, ty, pad, 1, dy).t,
            (Room(rows, cols, torch.int8, pad, 3, q).t, Room(rows, s.shape[1], torch.uint8, 1, 0, s).t))
    crc.checkpoint_wgrad(*args, dw.t)
    want, bound = R.wgrad(dy, q, s)
    R.close(dw.t, want, bound, "dw")
    check_rest({"dw": dw})
    low = Room(outs, cols, ty, pad, 0, torch.ones(outs, cols))
    crc.checkpoint_wgrad(*args, low.t, accumulate=True)
    R.close(low.t, want + 1, bound + R.U * (want.abs() + 1), "dw of dy's type, added")
    check_rest({"dw": low})


def test_wgrad_of_f16_at_the_ends_of_its_range():
    """Blocks of x that f16 does not hold (too large, too small, NaN) next to
    ones that it does, blocks of zeros, subnormal and infinite dy."""
    rows, outs, cols = 300, 136, 160
    gen = torch.Generator().manual_seed(28)
    dy = torch.randn(rows, outs, generator=gen).half()
    dy[:, 5] *= 2.0 ** -18  # subnormal in f16
    dy[3, 7] = torch.tensor(6e-8).half()
    x = torch.randn(rows, cols, generator=gen)
    x[:, 64:96] = 0
    near = x.clone()
    near[10, 32:64] *= 2.0 ** 13   # the largest blocks that f16 holds, or nearly
    near[11, 32:64] *= 2.0 ** -18  # and the smallest
    far = x.clone()
    far[40, 96:128] *= 2.0 ** 40
    far[200, :32] *= 2.0 ** -60
    nan = x.clone()
    nan[77, 130] = float("nan")
    for name, v in (("plain", x), ("near", near), ("far", far), ("nan", nan)):
        say("f16 range", name)
        q, s = R.pack(v)
        want, bound = R.wgrad(dy, q, s)
        dw = torch.empty(outs, cols, device="cuda")
        crc.checkpoint_wgrad(dy.cuda(), (q.cuda(), s.cuda()), dw)
        R.close(dw, want, bound, name)
    inf = dy.clone()
    inf[50, 20], inf[51, 21] = float("inf"), float("nan")
    q, s = R.pack(x)
    want, bound = R.wgrad(inf, q, s)
    dw = torch.empty(outs, cols, device="cuda")
    crc.checkpoint_wgrad(inf.cuda(), (q.cuda(), s.cuda()), dw)
    finite = torch.isfinite(want)
    assert torch.equal(torch.isnan(dw.cpu()), torch.isnan(want))
    assert torch.equal(torch.isinf(dw.cpu()), torch.isinf(want))
    R.close(dw.cpu()[finite], want[finite], bound[finite], "infinite dy")


def test_both_ways_from_python_make_the_same_calls(monkeypatch):
    t, d, o = 70, 520, 96
    gen = torch.Generator().manual_seed(3)
    ty = torch.float16
    parts = [draw(gen, t, d).to(ty).cuda() for _ in range(3)]
    x = draw(gen, t, d).to(ty).cuda()
    dz, dxo, dy = (draw(gen, t, n).to(ty).cuda() for n in (d, d, o))
    w1, w2 = ((1 + draw(gen, d, scale=0.2)).float().cuda() for _ in range(2))
    gate = draw(gen, 7, d).to(ty).cuda()
    n = dict(post_weight=w1, gate=gate, pre_weight=w2, branch_scale=0.5, weight_offset=0.25)

    def step(stream=None):
        b = {k: torch.zeros(t, d, dtype=ty, device="cuda") for k in ("xo", "z", "h", "dx", "dh")}
        b |= {"dw1": torch.zeros_like(w1), "dw2": torch.zeros_like(w1), "dg": torch.zeros_like(gate),
              "dw": torch.zeros(o, d, device="cuda"), "r1": torch.zeros(t, device="cuda"),
              "r2": torch.zeros(t, device="cuda"), "back": torch.zeros(t, d, device="cuda")}
        k = [crc.checkpoint_empty(t, d) for _ in range(4)]
        crc.block_norm(tuple(parts), x, b["xo"], b["z"], h=b["h"], post_rstd=b["r1"],
                       pre_rstd=b["r2"], h_kept=k[0], x_kept=k[1], z_kept=k[2], stream=stream, **n)
        crc.block_norm_backward(dz, dxo, k[1], b["r2"], b["dx"], b["dh"], h=k[0],
                                post_rstd=b["r1"], dpost_weight=b["dw1"], dgate=b["dg"],
                                dpre_weight=b["dw2"], stream=stream, **n)
        crc.checkpoint_pack(x, k[3], stream=stream)
        crc.checkpoint_unpack(k[3], b["back"], stream=stream)
        crc.checkpoint_wgrad(dy, k[2], b["dw"], stream=stream)
        return b

    calls = []
    native = K._native_call

    def counted(name, stream, *args):
        calls.append((name, native(name, stream, *args)))
        return calls[-1][1]

    monkeypatch.setattr(K, "_native_call", counted)
    first = step()
    assert len(calls) == 5 and all(done for _, done in calls)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step(side)
    side.synchronize()
    monkeypatch.setattr(K, "_native_call", lambda *a: False)
    for b in (step(), other):
        for name, v in first.items():
            assert torch.equal(v, b[name]), name


def test_what_the_extension_leaves_to_the_checks():
    """A single row with any pitch, a column-strided view, a tensor from
    another place: the extension makes no call, the Python code decides."""
    x = torch.zeros(8, 64, device="cuda", dtype=torch.bfloat16)
    K._Group(x, "x")
    none = [None] * 7
    args = lambda p, x: (p, x, None, None, None, None, None, 1e-6, 0.0, 1.0, 1.0, *none)  # noqa: E731
    assert K._native.block_norm(*args([x], x)) == 0
    for bad in (args([x.cpu()], x), args([x], x.cpu()), args([x.t().contiguous().t()], x),
                args([x.float()], x), args([x[:7]], x), args(["x"], x), args([x], None),
                args([x], x[:0]), args(iter([x]), x)):
        assert K._native.block_norm(*bad) is None
    assert K._native.block_norm(x) is None
    one = torch.randn(1, 64, device="cuda").expand(1, 64)
    z = torch.empty(1, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    crc.block_norm([one.as_strided((1, 64), (1, 1))], one, z=z, pre_weight=w)  # a row has no pitch
    want = R.forward([one.cpu()], one.cpu(), None, None, w.cpu(), eps=EPS, offset=0.0, alpha=1.0,
                     beta=1.0)
    R.close(z, *want["z"], "one row")
    crc.block_norm(iter([one]), one, z=z, pre_weight=w)
    R.close(z, *want["z"], "parts from an iterator")
