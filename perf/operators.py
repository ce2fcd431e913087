"""Cases of the block-boundary operators and of the 8-bit activation checkpoints.

A tensor-parallel block ends with N ranks' partial outputs.  The operators
timed here fold them, normalise, gate and scale the fold, add it to the
residual stream and normalise the result for the next block (``norm``), take
the gradients of that (``grad``), keep activations in 8 bits and read them
back (``ckpt``), take a projection's weight gradient from what was kept
(``wgrad``), and run a boundary's forward and backward pass together
(``step``).

With T rows, D columns, partials y_0..y_{N-1}, residual x, norm weights w1
(after the block) and w2 (before the next), gate g, scales a and b:

    h  = y_0 + ... + y_{N-1}
    p  = h r1 (w1 + off),          r1 = 1 / sqrt(mean(h^2) + eps)
    x' = b x + a g p
    z  = x' r2 (w2 + off),         r2 = 1 / sqrt(mean(x'^2) + eps)

The gate has G rows, each for T / G consecutive rows of the stream (1: one
value per channel; T: one per element; in between: one row per sequence).

8 bits: 32 consecutive elements of a row share a power of two 2^E, the
smallest for which rint(amax 2^(6-E)) <= 127; q = rint(v 2^(6-E)) and the
value kept is q 2^(E-6), which bfloat16 holds exactly.
"""

import torch

own = False

EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decoded token of eight ranks' partial sums; only the next block's norm
        _norm("norm_token", "bf16", 1, 8192, 8, post=False, gate_rows=0),
        # a decode batch: norms on both sides, a gate per channel, weights kept as offsets from 1
        _norm("norm_decode", "f16", 48, 5120, 4, offset=1.0),
        # a prompt: the plain fold, residual and norm
        _norm("norm_prompt", "bf16", 4096, 8192, 8, post=False, gate_rows=0),
        # odd sizes and strides in 32 bits, a gate row per sequence, the fold kept for training
        _norm("norm_odd", "f32", 1001, 2501, 3, gate_rows=7, pad=3, train=True),
        # training batch: both norms' gradients from packed activations
        _grad("grad_packed", "bf16", 16384, 4096, packed=True),
        # gradients in 32 bits from activations kept whole, a gate row per sequence
        _grad("grad_sequences", "f32", 4096, 1536, gate_rows=8),
        # forward and backward of one boundary, activations kept in 8 bits between them
        _step("step_packed", "bf16", 4096, 4096, 2),
        # keep a batch's activations and read them back
        _ckpt("ckpt_batch", "bf16", 8192, 8192),
        # odd columns, a row ends inside a block of 32
        _ckpt("ckpt_odd", "f32", 777, 1003, pad=5),
        # a projection's weight gradient over a batch of tokens
        _wgrad("wgrad_batch", "bf16", 8192, 4096, 4096),
        # few outputs, many tokens: the sum is the long axis
        _wgrad("wgrad_long", "bf16", 32768, 640, 512),
        # odd sizes in 16-bit floats
        _wgrad("wgrad_odd", "f16", 1001, 1501, 777, pad=1),
    ]


def _norm(name, dtype, rows, cols, ranks, post=True, gate_rows=1, offset=0.0, pad=0, train=False):
    return {"name": name, "op": "norm", "dtype": dtype, "rows": rows, "cols": cols,
            "ranks": ranks, "post": post, "gate_rows": gate_rows, "offset": offset, "pad": pad,
            "train": train}


def _grad(name, dtype, rows, cols, packed=False, gate_rows=1, pad=0, post=True):
    return {"name": name, "op": "grad", "dtype": dtype, "rows": rows, "cols": cols,
            "packed": packed, "gate_rows": gate_rows, "pad": pad, "post": post, "offset": 0.0}


def _step(name, dtype, rows, cols, ranks, gate_rows=1):
    return {"name": name, "op": "step", "dtype": dtype, "rows": rows, "cols": cols,
            "ranks": ranks, "gate_rows": gate_rows, "post": True, "offset": 0.0, "pad": 0}


def _ckpt(name, dtype, rows, cols, pad=0):
    return {"name": name, "op": "ckpt", "dtype": dtype, "rows": rows, "cols": cols, "pad": pad}


def _wgrad(name, dtype, rows, outs, cols, pad=0):
    return {"name": name, "op": "wgrad", "dtype": dtype, "rows": rows, "outs": outs,
            "cols": cols, "pad": pad}


def _size(rng, low, high):
    """A size between low and high, even over the logarithm; odd half the time."""
    n = round(low * (high / low) ** rng.random())
    return max(low, min(high, n | 1 if rng.random() < 0.5 else n))


def draw(rng):
    op = rng.choice(("norm", "norm", "grad", "step", "ckpt", "wgrad"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    pad = rng.choice((0, 0, 1, 8))
    if op == "wgrad":
        outs, cols = _size(rng, 64, 4096), _size(rng, 64, 4096)
        rows = _size(rng, 16, max(17, min(32768, (8192 << 22) // (outs * cols))))
        return {k: v for k, v in _wgrad("", dtype, rows, outs, cols, pad).items() if k != "name"}
    cols = _size(rng, 128, 8192)
    if op == "norm":
        ranks = rng.randint(1, 8)
        rows, gate_rows = _grouped(rng, min(8192, (1 << 27) // (ranks * cols)))
        case = _norm("", dtype, rows, cols, ranks, post=rng.random() < 0.7, gate_rows=gate_rows,
                     offset=rng.choice((0.0, 1.0)), pad=pad, train=rng.random() < 0.5)
    elif op == "ckpt":
        case = _ckpt("", dtype, _size(rng, 1, 8192), cols, pad)
    elif op == "grad":
        rows, gate_rows = _grouped(rng, min(16384, (1 << 25) // cols))
        case = _grad("", dtype, rows, cols, packed=rng.random() < 0.5, gate_rows=gate_rows,
                     pad=pad, post=rng.random() < 0.7)
    else:
        rows, gate_rows = _grouped(rng, min(4096, (1 << 24) // cols))
        case = _step("", rng.choice(("bf16", "f16")), rows, cols, rng.randint(1, 4), gate_rows)
    return {k: v for k, v in case.items() if k != "name"}


def _grouped(rng, most):
    """(rows, gate rows): no gate, one row, a row per sequence, or one per row."""
    kind = rng.choice(("none", "one", "sequences", "full"))
    if kind == "sequences":
        groups = rng.randint(2, 8)
        return groups * _size(rng, 1, max(2, most // groups)), groups
    rows = _size(rng, 1, max(2, most))
    return rows, {"none": 0, "one": 1, "full": rows}[kind]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ty, rows, cols, pad = TYPES[case["dtype"]], case["rows"], case["cols"], case["pad"]
    st = dict(case)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * scale

    def strided(value, dtype=ty):
        """The values in rows `pad` elements further apart than they are wide."""
        room = torch.zeros(*value.shape[:-1], value.shape[-1] + pad, dtype=dtype, device="cuda")
        out = room[..., :value.shape[-1]]
        out.copy_(value)
        return out

    def stream(n):
        """A residual stream: a few channels far larger than the others."""
        return normal(rows, n) * torch.exp(normal(n) * 0.8)

    if case["op"] == "ckpt":
        st["x"] = strided(stream(cols))
        st["kept"] = _room(rows, cols)
        st["back"] = strided(torch.zeros(rows, cols, device="cuda"), torch.bfloat16)
        return st
    if case["op"] == "wgrad":
        st["dy"] = strided(normal(rows, case["outs"]))
        st["kept"] = _pack(stream(cols).to(ty).float())
        st["dw"] = torch.zeros(case["outs"], cols, dtype=torch.float32, device="cuda")
        return st

    # alpha and beta as a deep model scales them
    st["alpha"], st["beta"] = 0.5, 1.25
    # whole gradients in the type of the weights: 32 bits unless activations pass through 8 bits inside the pass
    wt = ty if case["op"] == "step" else torch.float32
    mid = 1.0 - case["offset"]
    st["w1"] = (mid + normal(cols, scale=0.2)).to(wt) if case["post"] else None
    st["w2"] = (mid + normal(cols, scale=0.2)).to(wt)
    st["gate"] = strided(0.5 + normal(case["gate_rows"], cols, scale=0.3)) if case["gate_rows"] else None
    x = stream(cols)
    if case["op"] in ("norm", "step"):
        st["parts"] = strided(normal(case["ranks"], rows, cols)).unbind(0)
        st["stack"] = torch.stack(st["parts"])
        st["x"] = strided(x)
        st["x_out"], st["z"] = strided(torch.zeros_like(x)), strided(torch.zeros_like(x))
    if case["op"] == "norm" and case["train"]:
        st["h"] = strided(torch.zeros_like(x))
    if case["op"] in ("grad", "step"):
        st["dz"], st["dx_out"] = strided(normal(rows, cols)), strided(normal(rows, cols, scale=0.3))
        st["dx"], st["dh"] = strided(torch.zeros_like(x)), strided(torch.zeros_like(x))
        st["dw1"] = torch.zeros(cols, dtype=wt, device="cuda") if case["post"] else None
        st["dw2"] = torch.zeros(cols, dtype=wt, device="cuda")
        st["dgate"] = strided(torch.zeros(case["gate_rows"], cols, device="cuda")) if case["gate_rows"] else None
    if case["op"] != "grad":
        st["r1"], st["r2"] = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
        if case["op"] == "step":
            st["h_kept"], st["x_kept"] = _room(rows, cols), _room(rows, cols)
        return st
    # what the forward pass left
    h = normal(rows, cols, scale=1.4)
    st["r1"], st["r2"] = _rstd(h), _rstd(x)
    if case["packed"]:
        st["h"], st["x_out"] = _pack(h.to(ty).float()), _pack(x.to(ty).float())
    else:
        st["h"], st["x_out"] = strided(h), strided(x)
    return st


def _room(rows, cols):
    """Uninitialised room for a packed activation: (values, one scale byte per 32)."""
    return (torch.zeros(rows, cols, dtype=torch.int8, device="cuda"),
            torch.zeros(rows, (cols + 31) // 32, dtype=torch.uint8, device="cuda"))


# ---------------------------------------------------------------- plain forms

def _power(e):
    """2^e in float32, exactly, for whole e in [-126, 127]."""
    return ((e + 127) << 23).view(torch.float32)


def _blocks(x):
    rows, cols = x.shape
    room = torch.zeros(rows, (cols + 31) // 32 * 32, dtype=x.dtype, device=x.device)
    room[:, :cols] = x
    return room.view(rows, -1, 32)


def _pack(x):
    """(q int8, scales uint8) of finite 32-bit values."""
    v = _blocks(x)
    bits = v.abs().amax(-1).contiguous().view(torch.int32)
    e = (bits >> 23) - 127 + ((bits & 0x7FFFFF) >= 0x7F0000).int()
    e = e.clamp(-120, 127)
    q = torch.round(v * _power(6 - e)[..., None]).clamp(-127, 127)
    return (q.to(torch.int8).view(x.shape[0], -1)[:, :x.shape[1]].contiguous(),
            (e + 127).to(torch.uint8))


def _unpack(kept):
    q, scales = kept
    f = _power(scales.int() - 127 - 6)
    return (_blocks(q.float()) * f[..., None]).view(q.shape[0], -1)[:, :q.shape[1]]


def _rstd(v):
    return torch.rsqrt(v.square().mean(-1) + EPS)


def _gated(v, gate):
    """v times its gate rows."""
    if gate is None:
        return v
    g = gate.float()
    return (v.view(g.shape[0], -1, v.shape[1]) * g[:, None]).view(v.shape)


def _forward(st):
    h = st["stack"].float().sum(0)
    p = h
    r1 = _rstd(h)
    if st["w1"] is not None:
        p = h * r1[:, None] * (st["w1"].float() + st["offset"])
    x_out = st["beta"] * st["x"].float() + st["alpha"] * _gated(p, st["gate"])
    r2 = _rstd(x_out)
    return h, r1, x_out, r2, x_out * r2[:, None] * (st["w2"].float() + st["offset"])


def _backward(st, h, r1, x_out, r2):
    ty = TYPES[st["dtype"]]
    xh = x_out * r2[:, None]
    dz = st["dz"].float()
    u = dz * (st["w2"].float() + st["offset"])
    dx_out = st["dx_out"].float() + r2[:, None] * (u - xh * (u * xh).mean(-1, keepdim=True))
    out = {"dx": (st["beta"] * dx_out).to(ty), "dw2": (dz * xh).sum(0).to(st["w2"].dtype)}
    dp = st["alpha"] * _gated(dx_out, st["gate"])
    p = h
    if st["w1"] is None:
        out["dh"] = dp.to(ty)
    else:
        w1, hh = st["w1"].float() + st["offset"], h * r1[:, None]
        p = hh * w1
        v = dp * w1
        out["dh"] = (r1[:, None] * (v - hh * (v * hh).mean(-1, keepdim=True))).to(ty)
        out["dw1"] = (dp * hh).sum(0).to(st["w1"].dtype)
    if st["gate"] is not None:
        dg = st["alpha"] * p * dx_out
        out["dgate"] = dg.view(st["gate"].shape[0], -1, dg.shape[1]).sum(1).to(ty)
    return out


def _plain(st):
    ty, op = TYPES[st["dtype"]], st["op"]
    if op == "ckpt":
        return _unpack(_pack(st["x"].float())).to(torch.bfloat16)
    if op == "wgrad":
        return st["dy"].float().t() @ _unpack(st["kept"])
    if op == "grad":
        whole = _unpack if st["packed"] else torch.Tensor.float
        return _backward(st, whole(st["h"]), st["r1"], whole(st["x_out"]), st["r2"])
    h, r1, x_out, r2, z = _forward(st)
    out = {"x_out": x_out.to(ty), "z": z.to(ty)}
    if op == "step":
        h, x_out = (_unpack(_pack(v.to(ty).float())) for v in (h, x_out))
        return {**out, **_backward(st, h, r1, x_out, r2)}
    if st["train"]:
        out |= {"h": h.to(ty), "r2": r2}
        if st["post"]:
            out["r1"] = r1
    return out


# ---------------------------------------------------------------- the calls

def run(state):
    if not own:
        return _plain(state)
    import cross_rank_collective_amd as crc

    st, op = state, state["op"]
    if op == "ckpt":
        crc.checkpoint_pack(st["x"], st["kept"])
        crc.checkpoint_unpack(st["kept"], st["back"])
        return st["back"]
    if op == "wgrad":
        crc.checkpoint_wgrad(st["dy"], st["kept"], st["dw"])
        return st["dw"]
    out = {}
    norms = {"post_weight": st["w1"], "gate": st["gate"], "pre_weight": st["w2"],
             "weight_offset": st["offset"], "branch_scale": st["alpha"], "residual_scale": st["beta"]}
    if op in ("norm", "step"):
        keep = {}
        if op == "step":
            keep = {"h_kept": st["h_kept"], "x_kept": st["x_kept"]}
        elif st["train"]:
            keep = {"h": st["h"]}
            out |= {"h": st["h"], "r2": st["r2"]}
        if keep:
            keep["pre_rstd"] = st["r2"]
            if st["post"]:
                keep["post_rstd"] = st["r1"]
                if op == "norm":
                    out["r1"] = st["r1"]
        crc.block_norm(st["parts"], st["x"], st["x_out"], st["z"], eps=EPS, **norms, **keep)
        out |= {"x_out": st["x_out"], "z": st["z"]}
    if op in ("grad", "step"):
        h, x_out = (st["h_kept"], st["x_kept"]) if op == "step" else (st["h"], st["x_out"])
        crc.block_norm_backward(st["dz"], st["dx_out"], x_out, st["r2"], st["dx"], st["dh"], h=h,
                                post_rstd=st["r1"] if st["post"] else None,
                                dpost_weight=st["dw1"], dgate=st["dgate"], dpre_weight=st["dw2"],
                                **norms)
        out |= {"dx": st["dx"], "dh": st["dh"], "dw2": st["dw2"]}
        if st["post"]:
            out["dw1"] = st["dw1"]
        if st["gate"] is not None:
            out["dgate"] = st["dgate"]
    return out


# ---------------------------------------------------------------- 64 bits

def _exact_pack(v):
    """The values kept of v (64 bits, already of the activations' type)."""
    rows, cols = v.shape
    padded = torch.nn.functional.pad(v, (0, -cols % 32)).view(rows, -1, 32)
    top = padded.abs().amax(-1, keepdim=True)
    _, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1)
    e = torch.where(torch.round(torch.ldexp(top, 7 - e)) > 127, e, e - 1)
    e = e.clamp(-120, 127)
    q = torch.round(torch.ldexp(padded, 6 - e)).clamp(-127, 127)
    return torch.ldexp(q, e - 6).view(rows, -1)[:, :cols]


def _exact_kept(kept):
    q, scales = kept
    each = scales.double().repeat_interleave(32, 1)[:, :q.shape[1]]
    return q.double() * torch.exp2(each - 133)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "ckpt":
        return _exact_pack(st["x"].double())
    if case["op"] == "wgrad":
        return torch.matmul(st["dy"].double().t(), _exact_kept(st["kept"]))
    rows, cols = case["rows"], case["cols"]
    ones = torch.ones(cols, dtype=torch.float64, device="cuda")
    w1 = ones if st["w1"] is None else st["w1"].double() + case["offset"]
    w2 = st["w2"].double() + case["offset"]
    g = torch.ones(1, cols, dtype=torch.float64, device="cuda") if st["gate"] is None else st["gate"].double()
    g = st["alpha"] * g.repeat_interleave(rows // g.shape[0], 0)
    out, ty = {}, TYPES[case["dtype"]]
    if case["op"] in ("norm", "step"):
        h = st["parts"][0].double().clone()
        for y in st["parts"][1:]:
            h += y.double()
        r1 = (torch.linalg.vector_norm(h, dim=1) ** 2 / cols + EPS) ** -0.5
        branch = g * w1 * h
        if st["w1"] is not None:
            branch *= r1[:, None]
        x_out = branch + st["beta"] * st["x"].double()
        r2 = (torch.linalg.vector_norm(x_out, dim=1) ** 2 / cols + EPS) ** -0.5
        out = {"x_out": x_out, "z": w2 * (r2[:, None] * x_out)}
        if case["op"] == "norm":
            if case["train"]:
                out |= {"h": h, "r2": r2}
                if st["w1"] is not None:
                    out["r1"] = r1
            return out
        h, x_out = _exact_pack(h.to(ty).double()), _exact_pack(x_out.to(ty).double())
    else:
        r1, r2 = st["r1"].double(), st["r2"].double()
        h, x_out = (_exact_kept(st[k]) if case["packed"] else st[k].double() for k in ("h", "x_out"))
    # dz reaches x' through z = w2 x' r2, r2 a function of x': the Jacobian's
    # symmetric form, r2 (1 - r2^2 x' x'^T / D), applied to dz w2
    dz = st["dz"].double()
    a = dz * w2
    along = (a * x_out).sum(1) * r2 ** 3 / cols
    stream = st["dx_out"].double() + r2[:, None] * a - along[:, None] * x_out
    out["dx"] = st["beta"] * stream
    out["dw2"] = r2 @ (dz * x_out)
    b = g * w1 * stream
    if st["w1"] is None:
        out["dh"] = b
        scaled = h
    else:
        along = (b * h).sum(1) * r1 ** 3 / cols
        out["dh"] = r1[:, None] * b - along[:, None] * h
        scaled = r1[:, None] * h
        out["dw1"] = r1 @ (g * stream * h)
    if st["gate"] is not None:
        each = st["alpha"] * w1 * scaled * stream
        out["dgate"] = torch.stack([e.sum(0) for e in each.chunk(st["gate"].shape[0])])
    return out


# ---------------------------------------------------------------- work

def work(case):
    s = 4 if case["dtype"] == "f32" else 2
    rows, cols = case["rows"], case["cols"]
    n, kept = rows * cols, rows * (cols + (cols + 31) // 32)
    if case["op"] == "ckpt":  # x read, 8 bits written; 8 bits read, bfloat16 written
        return {"bytes": n * s + 2 * kept + 2 * n, "flops": 4 * n}
    if case["op"] == "wgrad":
        outs = case["outs"]
        return {"bytes": rows * outs * s + kept + 4 * outs * cols, "flops": 2 * rows * outs * cols}
    small = cols * (2 if case["op"] == "step" else 4) * (1 + case["post"]) + case["gate_rows"] * cols * s
    total = {"bytes": 0, "flops": 0}
    if case["op"] in ("norm", "step"):  # partials and residual read, x' and z written
        total["bytes"] += (case["ranks"] + 3) * n * s + small
        total["flops"] += (case["ranks"] + 9) * n
        if case["op"] == "step":  # both activations kept
            total["bytes"] += 2 * kept
        elif case["train"]:
            total["bytes"] += n * s
    if case["op"] in ("grad", "step"):  # two gradients and two activations read, two gradients written
        whole = case["op"] == "grad" and not case["packed"]
        total["bytes"] += 4 * n * s + (2 * n * s if whole else 2 * kept) + 2 * small
        total["flops"] += 30 * n
    return total
