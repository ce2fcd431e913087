"""One tensor-parallel block boundary of a training step, on one GPU.

A block ends with N ranks' partial outputs (here: N buffers of one GPU, as for
``treduce``).  The step folds them, normalises, gates and scales the fold, adds
it to the residual stream and normalises the result for the next block, which
projects it.  What the backward pass needs of this is kept in 8 bits.  Then the
gradients come back: of the projection's weight, from its packed input; of the
boundary, from the packed fold and stream.

    python examples/block_step.py [--tokens 4096] [--width 4096] [--ranks 8]

prints what is kept, the time of each part and of the same step in elementary
torch operations, and how far the two are apart.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import cross_rank_collective_amd as crc  # noqa: E402

EPS = 1e-6


class Boundary:
    """A block's end and the next one's start: weights, a gate per channel."""

    def __init__(self, width: int, outs: int, device="cuda"):
        self.post = torch.ones(width, device=device)
        self.pre = torch.ones(width, device=device)
        self.gate = torch.full((width,), 0.5, device=device, dtype=torch.bfloat16)
        self.proj = torch.randn(outs, width, device=device, dtype=torch.bfloat16) * width ** -0.5

    def norms(self):
        return {"post_weight": self.post, "gate": self.gate, "pre_weight": self.pre}

    def forward(self, parts, x):
        """(new stream, projection's output, what the backward pass needs)."""
        rows, cols = x.shape
        x_out, z = torch.empty_like(x), torch.empty_like(x)
        kept = {n: crc.checkpoint_empty(rows, cols, x.device) for n in ("h", "x", "z")}
        post, pre = (torch.empty(rows, device=x.device) for _ in range(2))
        crc.block_norm(parts, x, x_out, z, post_rstd=post, pre_rstd=pre, h_kept=kept["h"],
                       x_kept=kept["x"], z_kept=kept["z"], eps=EPS, **self.norms())
        return x_out, z @ self.proj.t(), (kept, post, pre)

    def backward(self, dx_out, dy, saved):
        """Gradients of the stream, of every rank's partial output and of the
        weights, from those of the new stream and of the projection's output."""
        kept, post, pre = saved
        grads = {"proj": torch.empty_like(self.proj), "post": torch.empty_like(self.post),
                 "pre": torch.empty_like(self.pre), "gate": torch.empty_like(self.gate)}
        crc.checkpoint_wgrad(dy, kept["z"], grads["proj"])
        dz = dy @ self.proj
        dx, dpart = torch.empty_like(dx_out), torch.empty_like(dx_out)
        crc.block_norm_backward(dz, dx_out, kept["x"], pre, dx, dpart, h=kept["h"], post_rstd=post,
                                dpost_weight=grads["post"], dgate=grads["gate"],
                                dpre_weight=grads["pre"], **self.norms())
        return dx, dpart, grads


def plain(b: Boundary, parts, x, dx_out, dy):
    """The same step by autograd over elementary operations in float32."""
    leaves = [t.detach().float().requires_grad_() for t in (torch.stack(parts).float().sum(0), x,
                                                            b.post, b.pre, b.gate, b.proj)]
    h, xs, post, pre, gate, proj = leaves
    x_out = xs + gate * (h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * post)
    z = x_out * torch.rsqrt(x_out.square().mean(-1, keepdim=True) + EPS) * pre
    y = z @ proj.t()
    torch.autograd.backward([x_out, y], [dx_out.float(), dy.float()])
    return {"stream": x_out, "y": y, "dpart": h.grad, "dx": xs.grad, "post": post.grad,
            "pre": pre.grad, "gate": gate.grad, "proj": proj.grad}


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
    ap.add_argument("--outs", type=int, default=4096)
    ap.add_argument("--ranks", type=int, default=8)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    parts = [rand(a.tokens, a.width) for _ in range(a.ranks)]
    x, dx_out, dy = rand(a.tokens, a.width), rand(a.tokens, a.width), rand(a.tokens, a.outs)
    b = Boundary(a.width, a.outs)

    x_out, y, saved = b.forward(parts, x)
    dx, dpart, grads = b.backward(dx_out, dy, saved)
    want = {k: v.detach() for k, v in plain(b, parts, x, dx_out, dy).items()}
    got = {"stream": x_out, "y": y, "dx": dx, "dpart": dpart, **grads}
    apart = {k: float((got[k].float() - w).norm() / w.norm()) for k, w in want.items()}

    kept = sum(t.numel() * t.element_size() for k in saved[0].values() for t in k)
    print(f"kept for the backward pass: {kept / 2**20:.1f} MiB "
          f"({3 * x.numel() * x.element_size() / 2**20:.1f} in bfloat16)")
    print(f"forward {milliseconds(lambda: b.forward(parts, x)):.3f} ms, "
          f"backward {milliseconds(lambda: b.backward(dx_out, dy, saved)):.3f} ms, "
          f"plain step {milliseconds(lambda: plain(b, parts, x, dx_out, dy)):.3f} ms")
    print("relative distance from float32: " + ", ".join(f"{k} {v:.1e}" for k, v in apart.items()))
    return apart


if __name__ == "__main__":
    main()
