"""Cases of the layer-norm boundary, the gated feed-forward block and the
clipping of gradients by their global norm.

What a tensor-parallel training step runs next to the reduction and the
RMS-norm boundary: a block's end and the next one's start where the model uses
layer norm (``ln``) and its gradients (``lngrad``); the column-parallel half of
a gated feed-forward block (``ffn``), whose products need a token's row at
decoding and a batch's in training, and its gradients (``ffngrad``); and after
the gradients' reduction the norm over all of them and the clipping (``clip``).

With T rows, D columns, partials y_0..y_{N-1} and residual x:

    x' = x + y_0 + ... + y_{N-1}
    z  = (x' - m) r w + b,     m = mean(x'), r = 1 / sqrt(mean((x' - m)^2) + eps)

With weights Wg, Wu of F x D and an activation f (silu, or gelu in its exact or
its tanh form):

    g = x Wg^T,  u = x Wu^T,  y = f(g) u
    dg = dy u f'(g),  du = dy f(g),  dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x

With gradients of any number and shape, n the root of the sum of all their
squares:

    out = grad min(1, most / n)
"""

import math
import random

import torch

own = False

EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decoded token of eight ranks' partial sums
        _ln("ln_token", "bf16", 1, 8192, 8),
        # a training batch's boundary, statistics kept for the backward pass
        _ln("ln_batch", "bf16", 8192, 4096, 4, train=True),
        # odd sizes and strides in 32 bits, no partials: the norm alone
        _ln("ln_odd", "f32", 1001, 2501, 0, pad=3, train=True),
        # gradients of a training batch
        _lngrad("lngrad_batch", "bf16", 16384, 4096),
        # odd sizes in 16-bit floats
        _lngrad("lngrad_odd", "f16", 1777, 1003, pad=5),
        # one decoded token: the weights are read once
        _ffn("ffn_token", "bf16", 1, 4096, 8192),
        # a prompt of a wide block
        _ffn("ffn_prompt", "bf16", 4096, 4096, 12288),
        # odd sizes, the projections kept for the backward pass, exact gelu
        _ffn("ffn_odd", "f16", 501, 1003, 2501, act="gelu", pad=1, train=True),
        # gradients of a training batch
        _ffngrad("ffngrad_batch", "bf16", 8192, 4096, 8192),
        # gradients in 32 bits, the tanh form
        _ffngrad("ffngrad_f32", "f32", 1024, 1536, 4096, act="gelu_tanh"),
        # a small model's few gradients: latency
        _clip("clip_few", "f32", 8, 100_000),
        # a bucket of a large model: matrices of 16 bits, vectors of 32, some with gaps between rows
        _clip("clip_many", "bf16", 300, 200_000_000, mixed=True, pad=8),
    ]


def _ln(name, dtype, rows, cols, ranks, pad=0, train=False):
    return {"name": name, "op": "ln", "dtype": dtype, "rows": rows, "cols": cols, "ranks": ranks,
            "pad": pad, "train": train}


def _lngrad(name, dtype, rows, cols, pad=0):
    return {"name": name, "op": "lngrad", "dtype": dtype, "rows": rows, "cols": cols, "pad": pad}


def _ffn(name, dtype, rows, cols, wide, act="silu", pad=0, train=False):
    return {"name": name, "op": "ffn", "dtype": dtype, "rows": rows, "cols": cols, "wide": wide,
            "act": act, "pad": pad, "train": train}


def _ffngrad(name, dtype, rows, cols, wide, act="silu", pad=0):
    return {"name": name, "op": "ffngrad", "dtype": dtype, "rows": rows, "cols": cols, "wide": wide,
            "act": act, "pad": pad}


def _clip(name, dtype, count, elems, mixed=False, pad=0, known=False):
    return {"name": name, "op": "clip", "dtype": dtype, "count": count, "elems": elems,
            "mixed": mixed, "pad": pad, "known": known}


def _size(rng, low, high):
    """A size between low and high, even over the logarithm; odd half the time."""
    n = round(low * (high / low) ** rng.random())
    return max(low, min(high, n | 1 if rng.random() < 0.5 else n))


def _width(rng, low, high):
    """As sizes are, but a multiple of 64 half the time, as widths of models are."""
    n = _size(rng, low, high)
    return max(low, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(("ln", "lngrad", "ffn", "ffn", "ffngrad", "clip"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    pad = rng.choice((0, 0, 1, 8))
    if op == "clip":
        elems = _size(rng, 1000, 1 << 27)
        case = _clip("", dtype, _size(rng, 1, min(400, elems // 100)), elems,
                     mixed=rng.random() < 0.5, pad=pad, known=rng.random() < 0.3)
    elif op == "ln":
        cols, ranks = _width(rng, 128, 8192), rng.randint(0, 8)
        case = _ln("", dtype, _size(rng, 1, min(16384, (1 << 27) // ((ranks + 1) * cols))), cols,
                   ranks, pad, train=rng.random() < 0.5)
    elif op == "lngrad":
        cols = _width(rng, 128, 8192)
        case = _lngrad("", dtype, _size(rng, 1, min(16384, (1 << 26) // cols)), cols, pad)
    else:
        cols, wide = _width(rng, 256, 8192), _width(rng, 256, 12288)
        most = (1 << 34) if dtype == "f32" else (1 << 37)  # tokens x columns x features
        rows = _size(rng, 1, max(2, min(8192, most // (cols * wide))))
        act = rng.choice(("silu", "silu", "gelu", "gelu_tanh"))
        if op == "ffn":
            case = _ffn("", dtype, rows, cols, wide, act, pad, train=rng.random() < 0.5)
        else:
            case = _ffngrad("", dtype, rows, cols, wide, act, pad)
    return {k: v for k, v in case.items() if k != "name"}


# ---------------------------------------------------------------- inputs

def _shapes(case):
    """(shape, 32 bits, gap behind each row) of the gradients: a few matrices hold most elements."""
    rng = random.Random(case["count"] * 1_000_003 + case["elems"])
    shares = [math.exp(2.0 * rng.gauss(0.0, 1.0)) for _ in range(case["count"])]
    each = case["elems"] / sum(shares)
    out = []
    for i, share in enumerate(shares):
        n = max(1, round(share * each))
        if i % 3 == 2 or n < 64:  # biases, norms' weights
            out.append(((n if n < 20000 else n // 64,), case["mixed"], 0))
        else:
            rows = max(1, round(math.sqrt(n) * rng.choice((0.25, 0.5, 1.0))))
            out.append(((rows, max(1, n // rows)), False, case["pad"] if i % 4 == 1 else 0))
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ty, st = TYPES[case["dtype"]], dict(case)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * scale

    if case["op"] == "clip":
        # gradients of a norm around 3, scaled as 16-bit floats are in training
        up = 1024.0 if case["dtype"] == "f16" else 1.0
        scale = up * 3.0 / math.sqrt(case["elems"])
        st["most"] = up
        st["grads"], outs = [], []
        for shape, wide, gap in _shapes(case):
            room = normal(*shape[:-1], shape[-1] + gap, scale=scale).to(torch.float32 if wide else ty)
            st["grads"].append(room[..., :shape[-1]])
            outs.append((shape, wide))
        # the clipped gradients lie one behind the other, as an optimizer's bucket holds them
        for key, want in (("flat", False), ("flat32", True)):
            st[key] = torch.zeros(sum(math.prod(s) for s, w in outs if w == want),
                                  dtype=torch.float32 if want else ty, device="cuda")
        at = {False: 0, True: 0}
        st["outs"] = []
        for shape, wide in outs:
            n = math.prod(shape)
            st["outs"].append(st["flat32" if wide else "flat"][at[wide]:at[wide] + n].view(shape))
            at[wide] += n
        st["norm"] = torch.zeros(1, device="cuda")
        return st

    rows, cols, pad = case["rows"], case["cols"], case["pad"]

    def strided(value, dtype=ty):
        """The values in rows `pad` elements further apart than they are wide."""
        room = torch.zeros(*value.shape[:-1], value.shape[-1] + pad, dtype=dtype, device="cuda")
        out = room[..., :value.shape[-1]]
        out.copy_(value)
        return out

    if case["op"] in ("ln", "lngrad"):
        # a residual stream: a mean, and a few channels far larger than the others
        x = normal(rows, cols) * torch.exp(normal(cols) * 0.8) + normal(rows, 1)
        st["w"], st["b"] = 1.0 + normal(cols, scale=0.2), normal(cols, scale=0.1)
        st["x"] = strided(x)
        if case["op"] == "ln":
            st["parts"] = [strided(normal(rows, cols)) for _ in range(case["ranks"])]
            st["x_out"], st["z"] = strided(torch.zeros_like(x)), strided(torch.zeros_like(x))
        else:
            st["dz"], st["dx_out"] = strided(normal(rows, cols)), strided(normal(rows, cols, scale=0.3))
            st["dx"] = strided(torch.zeros_like(x))
            st["dw"], st["db"] = torch.zeros_like(st["w"]), torch.zeros_like(st["b"])
        # what the forward pass leaves
        st["mean"], st["rstd"] = (v.contiguous() for v in _statistics(st["x"].float()))
        return st

    wide = case["wide"]
    st["x"] = strided(normal(rows, cols))
    st["wg"], st["wu"] = (strided(normal(wide, cols, scale=cols ** -0.5)) for _ in range(2))
    new = lambda *shape: strided(torch.zeros(*shape, device="cuda"))  # noqa: E731
    if case["op"] == "ffn":
        st["y"] = new(rows, wide)
        if case["train"]:
            st["g"], st["u"] = new(rows, wide), new(rows, wide)
        return st
    # what the forward pass kept
    st["g"], st["u"] = (strided(st["x"].float() @ st[w].float().t()) for w in ("wg", "wu"))
    st["dy"] = strided(normal(rows, wide))
    st["dg"], st["du"], st["dx"] = new(rows, wide), new(rows, wide), new(rows, cols)
    st["dwg"], st["dwu"] = new(wide, cols), new(wide, cols)
    return st


# ---------------------------------------------------------------- plain forms

def _statistics(x):
    mean = x.mean(-1)
    return mean, torch.rsqrt((x - mean[:, None]).square().mean(-1) + EPS)


def _normal_cdf(g):
    return 0.5 * torch.erfc(g * -math.sqrt(0.5))


def _activation(act, g):
    """f(g) and f'(g)."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        s = _normal_cdf(g)
        return g * s, s + g * torch.exp(-0.5 * g * g) * (2.0 * math.pi) ** -0.5
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 0.134145 * g * g)


def _plain(st):
    ty, op = TYPES[st["dtype"]], st["op"]
    if op == "clip":
        every = torch.cat([g.reshape(-1).float() for g in st["grads"]])
        norm = every.double().square().sum().sqrt()
        by = torch.clamp(st["most"] / norm, max=1.0).float()
        small, wide = ([(g.reshape(-1).float() * by).to(g.dtype) for g, (_, w, _) in
                        zip(st["grads"], _shapes(st)) if w == want] for want in (False, True))
        return {"norm": norm.float().view(1), "flat": torch.cat(small) if small else st["flat"],
                "flat32": torch.cat(wide) if wide else st["flat32"]}
    if op == "ln":
        x_out = st["x"].float()
        if st["parts"]:
            x_out = x_out + torch.stack(st["parts"]).float().sum(0)
        mean, rstd = _statistics(x_out)
        z = (x_out - mean[:, None]) * rstd[:, None] * st["w"] + st["b"]
        out = {"x_out": x_out.to(ty), "z": z.to(ty)}
        return {**out, "mean": mean, "rstd": rstd} if st["train"] else out
    if op == "lngrad":
        rstd = st["rstd"][:, None]
        xh, dz = (st["x"].float() - st["mean"][:, None]) * rstd, st["dz"].float()
        u = dz * st["w"]
        dx = st["dx_out"].float() + rstd * (u - u.mean(-1, keepdim=True)
                                            - xh * (u * xh).mean(-1, keepdim=True))
        return {"dx": dx.to(ty), "dw": (dz * xh).sum(0), "db": dz.sum(0)}
    x, wg, wu = (st[k].float() for k in ("x", "wg", "wu"))
    if op == "ffn":
        g, u = x @ wg.t(), x @ wu.t()
        out = {"y": (_activation(st["act"], g)[0] * u).to(ty)}
        return {**out, "g": g.to(ty), "u": u.to(ty)} if st["train"] else out
    dy = st["dy"].float()
    f, slope = _activation(st["act"], st["g"].float())
    dg, du = dy * st["u"].float() * slope, dy * f
    return {"dg": dg.to(ty), "du": du.to(ty), "dx": (dg @ wg + du @ wu).to(ty),
            "dwg": (dg.t() @ x).to(ty), "dwu": (du.t() @ x).to(ty)}


# ---------------------------------------------------------------- the calls

def run(state):
    if not own:
        return _plain(state)
    import cross_rank_collective_amd as crc

    st, op = state, state["op"]
    if op == "clip":
        if st["known"]:
            crc.grad_norm(st["grads"], st["norm"])
            crc.grad_scale(st["grads"], st["norm"], st["most"], outs=st["outs"])
        else:
            crc.grad_clip(st["grads"], st["most"], st["norm"], outs=st["outs"])
        return {k: st[k] for k in ("norm", "flat", "flat32")}
    if op == "ln":
        kept = {"mean": st["mean"], "rstd": st["rstd"]} if st["train"] else {}
        crc.layer_norm(st["parts"], st["x"], st["x_out"], st["z"], weight=st["w"], bias=st["b"],
                       eps=EPS, **kept)
        return {"x_out": st["x_out"], "z": st["z"], **kept}
    if op == "lngrad":
        crc.layer_norm_backward(st["dz"], st["dx_out"], st["x"], st["mean"], st["rstd"], st["dx"],
                                weight=st["w"], dweight=st["dw"], dbias=st["db"])
        return {k: st[k] for k in ("dx", "dw", "db")}
    if op == "ffn":
        kept = {"gate": st["g"], "up": st["u"]} if st["train"] else {}
        crc.gated_ffn(st["x"], st["wg"], st["wu"], st["y"], activation=st["act"], **kept)
        return {"y": st["y"], **({"g": st["g"], "u": st["u"]} if kept else {})}
    crc.gated_ffn_backward(st["dy"], st["g"], st["u"], st["dg"], st["du"], activation=st["act"],
                           x=st["x"], w_gate=st["wg"], w_up=st["wu"], dx=st["dx"],
                           dw_gate=st["dwg"], dw_up=st["dwu"])
    return {k: st[k] for k in ("dg", "du", "dx", "dwg", "dwu")}


# ---------------------------------------------------------------- 64 bits

def _exact_activation(act, g):
    """f(g) and f'(g), the slope by differentiation of the definition."""
    with torch.enable_grad():
        v = g.detach().clone().requires_grad_()
        if act == "silu":
            f = v * torch.sigmoid(v)
        elif act == "gelu":
            f = v * torch.special.ndtr(v)
        else:
            f = v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
        slope, = torch.autograd.grad(f.sum(), v)
    return f.detach(), slope


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g.double())
                                                     for g in st["grads"]]))
        by = st["most"] / norm if norm > st["most"] else torch.ones_like(norm)
        flat = {False: [], True: []}
        for g, (_, wide, _) in zip(st["grads"], _shapes(case)):
            flat[wide].append((g.double() * by).flatten())
        none = torch.zeros(0, dtype=torch.float64, device="cuda")
        return {"norm": norm.view(1), "flat": torch.cat(flat[False] or [none]),
                "flat32": torch.cat(flat[True] or [none])}
    if op == "ln":
        x_out = st["x"].double()
        for y in st["parts"]:
            x_out = x_out + y.double()
        var, mean = torch.var_mean(x_out, dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        z = torch.addcmul(st["b"].double(), (x_out - mean[:, None]) * rstd[:, None], st["w"].double())
        out = {"x_out": x_out, "z": z}
        return {**out, "mean": mean, "rstd": rstd} if case["train"] else out
    if op == "lngrad":
        # the Jacobian's symmetric form: the part of u along the constant row
        # and along the normalised one is taken out
        rstd, dz = st["rstd"].double()[:, None], st["dz"].double()
        xh = (st["x"].double() - st["mean"].double()[:, None]) * rstd
        u, n = dz * st["w"].double(), case["cols"]
        along = (u * xh).sum(1, keepdim=True) / n
        dx = rstd * (u - u.sum(1, keepdim=True) / n - along * xh) + st["dx_out"].double()
        return {"dx": dx, "dw": torch.einsum("td,td->d", dz, xh), "db": dz.sum(0)}
    x, wg, wu = (st[k].double() for k in ("x", "wg", "wu"))
    if op == "ffn":
        g = torch.mm(x, wg.t())
        u = torch.mm(x, wu.t())
        out = {"y": _exact_activation(case["act"], g)[0] * u}
        return {**out, "g": g, "u": u} if case["train"] else out
    f, slope = _exact_activation(case["act"], st["g"].double())
    du = f * st["dy"].double()
    dg = slope * st["u"].double() * st["dy"].double()
    dx = torch.mm(torch.cat([dg, du], 1), torch.cat([wg, wu]))
    return {"dg": dg, "du": du, "dx": dx, "dwg": torch.mm(x.t(), dg).t(), "dwu": torch.mm(x.t(), du).t()}


# ---------------------------------------------------------------- work

def work(case):
    s = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "clip":  # read for the norm, read and written for the scaling
        sizes = [math.prod(shape) * (4 if wide else s) for shape, wide, _ in _shapes(case)]
        return {"bytes": 3 * sum(sizes), "flops": 3 * case["elems"]}
    rows, cols = case["rows"], case["cols"]
    n = rows * cols
    if case["op"] == "ln":  # partials and residual read, x' and z written
        return {"bytes": (case["ranks"] + 3) * n * s + 8 * cols + (8 * rows if case["train"] else 0),
                "flops": (case["ranks"] + 8) * n}
    if case["op"] == "lngrad":  # two gradients and the stream read, one gradient written
        return {"bytes": 4 * n * s + 12 * cols + 8 * rows, "flops": 16 * n}
    wide = case["wide"]
    if case["op"] == "ffn":
        outs = 3 if case["train"] else 1
        return {"bytes": (n + 2 * cols * wide + outs * rows * wide) * s, "flops": 4 * n * wide}
    # dy and the projections read, their gradients written; x and the weights read, their gradients written
    return {"bytes": (5 * rows * wide + 2 * n + 4 * cols * wide) * s, "flops": 8 * n * wide}
