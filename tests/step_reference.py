"""The step's operators in 64 bits on the CPU, with bounds on what 32-bit
arithmetic may differ by.

Written from the formulas; shares no code with the library.  Functions return
(value, bound) pairs: the bound is for a computation in binary32 that follows
the formula, before the one rounding to the output's type, which
``block_reference.close`` adds.  U is half a step of binary32.
"""

from __future__ import annotations

import math

import torch

from tests.block_reference import ROW, U

# Second-order terms of the bounds below.
SLACK = 1.01


def layer_norm(parts, x, w, b, eps):
    """x_out, mean, rstd, z."""
    terms = [x.double(), *[p.double() for p in parts]]
    v = sum(terms)
    ev = U * len(parts) * sum(t.abs() for t in terms)  # each addition rounds a partial sum
    mean = v.mean(-1, keepdim=True)
    d = v - mean
    # the mean as first summed is off by at most first; its differences' own sum
    # puts that right to within the roundings of the differences and of their sum
    first = U * (ROW + 2) * v.abs().mean(-1, keepdim=True) + ev.mean(-1, keepdim=True)
    spread = (d.abs() + first).mean(-1, keepdim=True)
    em = ev.mean(-1, keepdim=True) + U * (ROW + 4) * spread
    var = d.square().mean(-1, keepdim=True)
    evar = U * (ROW + 12) * (var + first.square()) + 2 * (d.abs() * (ev + em)).mean(-1, keepdim=True)
    rstd = (var + eps) ** -0.5
    rel = 0.5 * evar / (var + eps) + 4 * U
    ed = ev + em + 3 * U * (d.abs() + first)
    w = torch.ones(v.shape[-1], dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(v.shape[-1], dtype=torch.float64) if b is None else b.double()
    z = d * rstd * w + b
    ez = w.abs() * rstd * (ed + d.abs() * (rel + 3 * U)) + 2 * U * z.abs()
    flat = lambda t: t.squeeze(-1)  # noqa: E731
    return {"x_out": (v, SLACK * ev), "mean": (flat(mean), SLACK * flat(em + U * mean.abs())),
            "rstd": (flat(rstd), SLACK * flat(rel * rstd)), "z": (z, SLACK * ez)}


def layer_norm_backward(dz, dxo, x, mean, rstd, w):
    """dx, dweight, dbias from the statistics as given."""
    dz, x = dz.double(), x.double()
    m, r = mean.double()[:, None], rstd.double()[:, None]
    w = torch.ones(x.shape[1], dtype=torch.float64) if w is None else w.double()
    dxo = torch.zeros_like(x) if dxo is None else dxo.double()
    xh, u = (x - m) * r, dz * w
    exh = 2 * U * xh.abs()
    avg = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    c0, c1 = avg(u), avg(u * xh)
    ec0 = U * (ROW + 3) * avg(u.abs())
    ec1 = U * (ROW + 6) * avg((u * xh).abs())
    dx = dxo + r * (u - c0 - xh * c1)
    parts = u.abs() + c0.abs() + (xh * c1).abs()
    edx = U * 6 * (dxo.abs() + r * parts) + r * (ec0 + xh.abs() * ec1 + exh * c1.abs())
    serial = min(x.shape[0], 256) + 80  # a chunk's rows, then the chunks' partial sums
    dw = (dz * xh).abs().sum(0)
    return {"dx": (dx, SLACK * edx), "dweight": ((dz * xh).sum(0), SLACK * U * (serial + 4) * dw),
            "dbias": (dz.sum(0), SLACK * U * serial * dz.abs().sum(0))}


def activation(name, g):
    """(f, its bound where g is exact), (f', its bound)."""
    if name == "silu":
        s = torch.sigmoid(g)
        q, rel = s * torch.sigmoid(-g), 10.0 * torch.ones_like(g)
    elif name == "gelu":
        s = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        q = torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
        rel = 20.0 + 4.0 * g * g  # the argument's rounding, by erfc's and exp's slopes
    else:
        c = 2.0 * math.sqrt(2.0 / math.pi)
        t = c * (g + 0.044715 * g ** 3)
        s = torch.sigmoid(t)
        q = s * torch.sigmoid(-t) * c * (1.0 + 0.134145 * g * g)
        rel = 20.0 + 8.0 * t.abs()
    f, slope = g * s, s + g * q
    tiny = 2.0 ** -126  # exp flushes or is subnormal below
    ef = U * (rel + 2) * f.abs() + tiny * (1 + g.abs())
    # 1 - s is off by s's own rounding, whatever is left of it
    flat = g.abs() * s * (0 if name == "gelu" else 1) * (1 if name == "silu" else
                                                         2 * (1 + 0.14 * g * g))
    es = U * (rel + 10) * (s + (g * q).abs()) + U * 12 * flat + tiny * (1 + g.abs())
    return (f, ef), (slope, es)


def product(a, b, exact: bool):
    """a b^T with sums in binary32 of any order; exact: products are not rounded."""
    a, b = a.double(), b.double()
    k = a.shape[1]
    return a @ b.t(), SLACK * U * (k + (0 if exact else 1)) * (a.abs() @ b.abs().t())


def gated_ffn(x, wg, wu, act):
    """y, gate, up."""
    exact = x.dtype != torch.float32
    (g, eg), (u, eu) = product(x, wg, exact), product(x, wu, exact)
    (f, ef), _ = activation(act, g)
    # |f'| and |f''| are below 1.2, so that an error of g moves f by 1.2 times it
    ef = ef + 1.2 * eg
    return {"gate": (g, eg), "up": (u, eu),
            "y": (f * u, SLACK * (ef * u.abs() + (f.abs() + ef) * eu + U * (f * u).abs()))}


def gated_slopes(dy, g, u, act):
    """dgate, dup from the projections as given."""
    dy, u = dy.double(), u.double()
    (f, ef), (slope, es) = activation(act, g.double())
    return {"dgate": (dy * u * slope, SLACK * ((dy * u).abs() * es + 3 * U * (dy * u * slope).abs())),
            "dup": (dy * f, SLACK * (dy.abs() * ef + 2 * U * (dy * f).abs()))}


def norm(grads):
    total = sum(float(g.double().square().sum()) for g in grads)
    return math.sqrt(total)


def factor(n, most):
    return most / n if n > most else (1.0 if n == n else math.nan)


def scaled(grad, n, most):
    """A gradient's scaled form: the norm, the quotient and the product rounded."""
    v = grad.double() * factor(n, most)
    return v, (4 * U * v.abs() if factor(n, most) != 1.0 else torch.zeros_like(v))
