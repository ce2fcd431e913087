"""One gated feed-forward block of a training step, on one GPU.

The block of a tensor-parallel model with layer norm: N ranks (here: N sets of
weights on one GPU) hold 1/N of the features each.  The step folds the last
block's partial outputs into the residual stream and normalises it; every rank
takes its gate and up projections, activation and product in one kernel and its
down projection, whose N partial outputs the next boundary folds.  Then the
gradients come back: of the boundaries, of every rank's projections, of the
input, whose N shares ``treduce`` sums; and all of them are clipped by their
norm.

    python examples/ffn_step.py [--tokens 4096] [--width 4096] [--wide 8192] [--ranks 2]

prints the time of each part and of the same step in elementary torch operations,
and how far the two are apart.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import cross_rank_collective_amd as crc  # noqa: E402

EPS = 1e-5


class Boundary:
    """Layer norm's weights, and what its backward pass needs."""

    def __init__(self, width, device="cuda"):
        self.weight, self.bias = torch.ones(width, device=device), torch.zeros(width, device=device)

    def forward(self, parts, x):
        x_out, z = torch.empty_like(x), torch.empty_like(x)
        mean, rstd = (torch.empty(x.shape[0], device=x.device) for _ in range(2))
        crc.layer_norm(parts, x, x_out, z, weight=self.weight, bias=self.bias, eps=EPS, mean=mean, rstd=rstd)
        return z, (x_out, mean, rstd)

    def backward(self, dz, dx_out, saved):
        """(gradient of the stream and of every partial, [dweight, dbias])"""
        dx, dw, db = torch.empty_like(dz), torch.empty_like(self.weight), torch.empty_like(self.bias)
        crc.layer_norm_backward(dz, dx_out, *saved, dx, weight=self.weight, dweight=dw, dbias=db)
        return dx, [dw, db]


class Rank:
    """One rank's features."""

    def __init__(self, width, wide, dtype, device="cuda"):
        new = lambda *s: torch.randn(*s, device=device, dtype=dtype) * s[1] ** -0.5  # noqa: E731
        self.gate, self.up, self.down = new(wide, width), new(wide, width), new(width, wide)

    def forward(self, z):
        y, g, u = (torch.empty(z.shape[0], self.gate.shape[0], dtype=z.dtype, device=z.device) for _ in range(3))
        crc.gated_ffn(z, self.gate, self.up, y, gate=g, up=u)
        return y @ self.down.t(), (y, g, u)

    def backward(self, dout, z, saved):
        """(this rank's share of z's gradient, [dgate, dup, ddown])"""
        y, g, u = saved
        dy = dout @ self.down
        dz, dwg, dwu = torch.empty_like(z), torch.empty_like(self.gate), torch.empty_like(self.up)
        # the projections' gradients take their place
        crc.gated_ffn_backward(dy, g, u, g, u, x=z, w_gate=self.gate, w_up=self.up, dx=dz,
                               dw_gate=dwg, dw_up=dwu)
        return dz, [dwg, dwu, dout.t() @ y]


class Block:
    def __init__(self, width, wide, ranks, dtype=torch.bfloat16):
        self.first, self.second = Boundary(width), Boundary(width)
        self.ranks = [Rank(width, wide // ranks, dtype) for _ in range(ranks)]

    def forward(self, parts, x):
        z, kept = self.first.forward(parts, x)
        outs, saved = zip(*(r.forward(z) for r in self.ranks))
        z2, kept2 = self.second.forward(list(outs), kept[0])
        return z2, (z, kept, saved, kept2)

    def backward(self, dz2, dstream, state, most):
        """(gradient of the stream and of every partial output that came in, clipped
        gradients of the weights, their norm before)"""
        z, kept, saved, kept2 = state
        dout, grads = self.second.backward(dz2, dstream, kept2)
        shares = []
        for r, s in zip(self.ranks, saved):
            share, more = r.backward(dout, z, s)
            shares.append(share)
            grads += more
        dz = torch.empty_like(z)
        crc.treduce(shares, dz)
        dx, more = self.first.backward(dz, dout, kept)
        grads += more
        norm = torch.empty(1, device=z.device)
        crc.grad_clip(grads, most, norm)
        return dx, grads, norm


def plain(b: Block, parts, x, dz2, dstream, most):
    """The same step by autograd over elementary operations in float32."""
    leaf = lambda t: t.detach().float().requires_grad_()  # noqa: E731
    weights = [leaf(t) for t in (b.second.weight, b.second.bias)]
    for r in b.ranks:
        weights += [leaf(r.gate), leaf(r.up), leaf(r.down)]
    weights += [leaf(b.first.weight), leaf(b.first.bias)]
    stream = leaf(torch.stack(parts).float().sum(0) + x.float()) if parts else leaf(x)

    def norm(v, w, bias):
        d = v - v.mean(-1, keepdim=True)
        return d * torch.rsqrt(d.square().mean(-1, keepdim=True) + EPS) * w + bias

    z = norm(stream, weights[-2], weights[-1])
    out = stream
    for i in range(len(b.ranks)):
        gate, up, down = weights[2 + 3 * i:5 + 3 * i]
        g = z @ gate.t()
        out = out + (g * torch.sigmoid(g) * (z @ up.t())) @ down.t()
    z2 = norm(out, weights[0], weights[1])
    torch.autograd.backward([z2, out], [dz2.float(), dstream.float()])
    grads = [w.grad for w in weights]
    n = torch.cat([g.reshape(-1) for g in grads]).square().sum().sqrt()
    by = torch.clamp(most / n, max=1.0)
    return z2.detach(), stream.grad, [g * by for g in grads], n


def milliseconds(call, runs: int = 10) -> float:
    call()
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(runs):
        call()
    stop.record()
    torch.cuda.synchronize()
    return start.elapsed_time(stop) / runs


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--wide", type=int, default=8192)
    ap.add_argument("--ranks", type=int, default=2)
    ap.add_argument("--dtype", choices=["bfloat16", "float16", "float32"], default="bfloat16")
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    dtype = getattr(torch, a.dtype)
    rand = lambda: torch.randn(a.tokens, a.width, device="cuda", dtype=dtype)  # noqa: E731
    parts, x, dz2, dstream = [rand() for _ in range(a.ranks)], rand(), rand(), rand()
    b, most = Block(a.width, a.wide, a.ranks, dtype), 1.0

    z2, state = b.forward(parts, x)
    kept = [[t.clone() for t in s] for s in state[2]]  # the backward pass writes over them
    dx, grads, norm = b.backward(dz2, dstream, state, most)
    want_z, want_dx, want, n = plain(b, parts, x, dz2, dstream, most)
    far = lambda got, ref: float((got.float() - ref).norm() / ref.norm())  # noqa: E731
    names = ["second.weight", "second.bias"]
    names += [f"rank{i}.{k}" for i in range(a.ranks) for k in ("gate", "up", "down")]
    names += ["first.weight", "first.bias"]
    apart = {"z": far(z2, want_z), "dx": far(dx, want_dx), "norm": far(norm, n.view(1)),
             **{k: far(g, w) for k, g, w in zip(names, grads, want)}}

    def backward():
        for s, k in zip(state[2], kept):
            for t, v in zip(s, k):
                t.copy_(v)
        b.backward(dz2, dstream, state, most)

    print(f"forward {milliseconds(lambda: b.forward(parts, x)):.3f} ms, "
          f"backward and clipping {milliseconds(backward):.3f} ms (with the projections put back), "
          f"plain step {milliseconds(lambda: plain(b, parts, x, dz2, dstream, most), 3):.3f} ms")
    print("relative distance from float32: " + ", ".join(f"{k} {v:.1e}" for k, v in apart.items()))
    return apart


if __name__ == "__main__":
    main()
