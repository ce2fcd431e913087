"""The block-boundary operators in 64 bits on the CPU, with bounds on what
32-bit arithmetic may differ by.

Written from the formulas; shares no code with the library.  Every function
returns (value, bound) pairs: the bound is for a computation in binary32 that
follows the formula with sums of any order over at most `terms` serial
additions, before the one rounding to the output's type, which ``close`` adds.
U is half a step of binary32.
"""

from __future__ import annotations

import torch

U = 2.0 ** -24
# A row's sum: at most 16 serial terms a lane, 6 steps in a wave, 16 waves, and
# the roundings of the squares, the mean, eps, the root and the quotient.
ROW = 64


def close(got: torch.Tensor, want: torch.Tensor, bound: torch.Tensor, what: str):
    """|got - want| within the bound and half a step of got's type; NaN for NaN."""
    t = got.dtype
    g = got.detach().cpu().double()
    tiny = torch.finfo(t).tiny * torch.finfo(t).eps / 2  # half a subnormal step
    tol = bound + torch.finfo(t).eps / 2 * (want.abs() + bound) + tiny
    over = want.abs() > torch.finfo(t).max
    w = torch.where(over, want.sign() * float("inf"), want)
    nan_w = torch.isnan(w)
    assert torch.equal(torch.isnan(g), nan_w), f"{what}: NaN where none is due, or none where one is"
    inf = torch.isinf(w)
    assert torch.equal(g[inf], w[inf]), f"{what}: infinities"
    ok = nan_w | inf | ((g - w).abs() <= tol)
    if not bool(ok.all()):
        bad = (~ok).nonzero()[0].tolist()
        i = tuple(bad)
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} off; at {i} got "
                             f"{g[i].item()!r}, want {w[i].item()!r} +- {tol[i].item():.3g}")


def rows_of_gate(gate, rows):
    return gate.double().repeat_interleave(rows // gate.shape[0], 0)


def rnorm(v):
    return v.square().sum(-1, keepdim=True).sqrt()


def forward(parts, x, w1, gate, w2, *, eps, offset, alpha, beta):
    """{name: (value, bound)} of h, r1, x_out, r2, z."""
    rows, cols = x.shape
    x = x.double()
    h = torch.zeros_like(x)
    mag = torch.zeros_like(x)
    for y in parts:
        h = h + y.double()
        mag = mag + y.double().abs()
    eh = U * max(0, len(parts) - 1) * mag
    out = {"h": (h, eh)}
    g = rows_of_gate(gate, rows) if gate is not None else torch.ones_like(x)
    b, eb = alpha * g * h, (alpha * g).abs() * (eh + 4 * U * h.abs())
    if w1 is not None:
        w = w1.double() + offset
        ew = U * (w1.double().abs() + abs(offset))
        r = 1 / (h.square().mean(-1, keepdim=True) + eps).sqrt()
        rho = ROW * U + rnorm(eh) / (rnorm(h) + (cols * eps) ** 0.5 + 1e-300)
        out["r1"] = (r[:, 0], (r * rho)[:, 0])
        b = b * r * w
        eb = (alpha * g * r).abs() * ((eh + h.abs() * (rho + 8 * U)) * w.abs() + h.abs() * ew)
    xo = beta * x + b
    ex = eb + 4 * U * ((beta * x).abs() + b.abs())
    out["x_out"] = (xo, ex)
    if w2 is not None:
        w = w2.double() + offset
        ew = U * (w2.double().abs() + abs(offset))
        r = 1 / (xo.square().mean(-1, keepdim=True) + eps).sqrt()
        rho = ROW * U + rnorm(ex) / (rnorm(xo) + (cols * eps) ** 0.5 + 1e-300)
        out["r2"] = (r[:, 0], (r * rho)[:, 0])
        out["z"] = (xo * r * w, r * ((ex + xo.abs() * (rho + 4 * U)) * w.abs() + xo.abs() * ew))
    return out


def backward(dz, dxo, xo, h, r1, r2, w1, gate, w2, *, offset, alpha, beta):
    """{name: (value, bound)} of dx, dh, dw1, dw2, dgate; xo and h are the
    activations as kept, r1 and r2 the forward pass's reciprocal norms."""
    ref = dz if dz is not None else dxo
    rows, cols = ref.shape
    zero = torch.zeros(rows, cols, dtype=torch.float64)
    d = dxo.double() if dxo is not None else zero
    k = ROW + 32  # a row sum's roundings and those of its terms and of its use
    out = {}
    s, ms = d, d.abs()
    direct, xh, xm = d.abs(), zero, 0.0
    if w2 is not None:
        w = w2.double() + offset
        wa = w2.double().abs() + abs(offset)
        xh = xo.double() * r2.double()[:, None]
        u = dz.double() * w
        ua = dz.double().abs() * wa
        r = r2.double()[:, None]
        mean_abs = (ua * xh.abs()).mean(-1, keepdim=True)
        s = d + r * (u - xh * (u * xh).mean(-1, keepdim=True))
        ms = d.abs() + r * (ua + xh.abs() * mean_abs)
        direct, xm = d.abs() + r * ua, r * mean_abs
        t = dz.double() * xh
        out["dw2"] = (t.sum(0), U * (rows + 64) * t.abs().sum(0))
    out["dx"] = (beta * s, abs(beta) * k * U * ms)
    g = rows_of_gate(gate, rows) if gate is not None else torch.ones(rows, cols, dtype=torch.float64)
    e, me = alpha * g * s, (alpha * g).abs() * ms
    p = h.double() if h is not None else zero
    pa = p.abs()
    if w1 is None:
        out["dh"] = (e, k * U * me)
    else:
        w = w1.double() + offset
        wa = w1.double().abs() + abs(offset)
        r = r1.double()[:, None]
        hh = p * r
        v = e * w
        ka = (alpha * g).abs() * wa * hh.abs()
        mean_abs = ((ka * direct).mean(-1, keepdim=True)
                    + xm * (ka * xh.abs()).mean(-1, keepdim=True))
        out["dh"] = (r * (v - hh * (v * hh).mean(-1, keepdim=True)),
                     2 * k * U * r * (me * wa + hh.abs() * mean_abs))
        t = e * hh
        out["dw1"] = (t.sum(0), U * ((rows + 64) * t.abs() + k * me * hh.abs()).sum(0))
        p, pa = hh * w, hh.abs() * wa
    if gate is not None:
        n = gate.shape[0]
        t = alpha * p * s
        b = U * ((rows // n + 64) * t.abs() + k * abs(alpha) * pa * ms)
        out["dgate"] = (t.view(n, -1, cols).sum(1) if rows else torch.zeros(n, cols).double(),
                        b.view(n, -1, cols).sum(1) if rows else torch.zeros(n, cols).double())
    return out


def pack(x):
    """(q int8, scales uint8) of x (exact in float32), by the definition."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -cols % 32)).view(rows, -1, 32)
    bad = ~torch.isfinite(v).all(-1)
    v = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    top = v.abs().amax(-1)
    e = torch.full_like(top, -120.0)
    while True:  # the smallest E that holds the block, by trying each
        big = (torch.round(top * torch.exp2(6 - e)) > 127) & (e < 127)
        if not bool(big.any()):
            break
        e = e + big
    w = torch.round(v * torch.exp2(6 - e)[..., None]).clamp(-127, 127)
    w = torch.where(bad[..., None], torch.zeros_like(w), w).view(rows, -1)[:, :cols]
    return (w.to(torch.int8).contiguous(),
            torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8))


def unpack(q, sc):
    each = sc.double().repeat_interleave(32, 1)[:, :q.shape[1]]
    f = torch.where(each == 255, torch.full_like(each, float("nan")), torch.exp2(each - 133))
    return q.double() * f


def wgrad(dy, q, sc):
    """(value, bound): each output is a sum of exact products; the bound holds
    for any order of binary32 additions."""
    x = unpack(q, sc)
    dy = dy.double()
    return dy.t() @ x, U * (dy.shape[0] + 64) * (dy.abs().t() @ x.abs())
