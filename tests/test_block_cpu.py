"""Block-boundary operators without a GPU: every refusal before any HIP call,
workspace sizes, the tensor wrappers' checks, and the 64-bit reference itself
(its gradients against differences and its packing against its definition)."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import cross_rank_collective_amd as crc
from cross_rank_collective_amd import binding as B
from cross_rank_collective_amd import block as K
from tests import block_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Fake device addresses: never dereferenced.
def at(i):
    return 0x10000000 + 0x4000000 * i


T, D = 8, 64


def rows(i, ld=D):
    return K.ptored_rows(at(i), ld)


def kept(i, q_ld=D, s_ld=2):
    return K.ptored_checkpoint(at(i), q_ld, at(i) + 0x200000, s_ld)


def params(**kw):
    v = dict(rows=T, cols=D, post_weight=at(20), pre_weight=at(21), gate=rows(22), gate_rows=1,
             weight_offset=0.0, branch_scale=1.0, residual_scale=1.0, eps=1e-6, dtype=1,
             weight_dtype=0)
    v.update(kw)
    return K.ptored_block_params(*[v[n] for n, _ in K.ptored_block_params._fields_])


def io(**kw):
    v = {n: None if t is ctypes.c_void_p else t() for n, t in K.ptored_block_io._fields_}
    v.update(x=rows(0), x_out=rows(1), z=rows(2))
    v.update(kw)
    return K.ptored_block_io(*[v[n] for n, _ in K.ptored_block_io._fields_])


def grad_io(**kw):
    v = {n: None if t is ctypes.c_void_p else t() for n, t in K.ptored_block_grad_io._fields_}
    v["workspace_bytes"] = 1 << 20
    v.update(dz=rows(0), dx_out=rows(1), x_out=rows(2), h=rows(3), post_rstd=at(4), pre_rstd=at(5),
             dx=rows(6), dh=rows(7), dgate=rows(8), dpost_weight=at(9), dpre_weight=at(10),
             workspace=at(11))
    v.update(kw)
    return K.ptored_block_grad_io(*[v[n] for n, _ in K.ptored_block_grad_io._fields_])


def norm(parts=2, part_ld=D, p=None, **kw):
    return crc.ptored_block_norm([at(30 + r) for r in range(parts)] if isinstance(parts, int)
                                 else parts, parts if isinstance(parts, int) else len(parts),
                                 part_ld, params() if p is None else p, io(**kw), 0)


INVALID, UNSUPPORTED, OVERLAP = -1, -2, -3


@pytest.mark.parametrize("kw,status", [
    (dict(parts=65), INVALID), (dict(parts=[at(30), 0]), INVALID),
    (dict(parts=0), INVALID),  # post_weight without a branch
    (dict(part_ld=D - 1), INVALID), (dict(x=K.ptored_rows()), INVALID),
    (dict(x=rows(0, D - 1)), INVALID), (dict(z=rows(2, 0)), INVALID),
    (dict(p=params(rows=-1)), INVALID), (dict(p=params(cols=-1)), INVALID),
    (dict(p=params(rows=1 << 50, cols=1 << 14)), INVALID),
    (dict(p=params(gate_rows=3)), INVALID), (dict(p=params(gate_rows=0)), INVALID),
    (dict(p=params(gate=rows(22, 5))), INVALID),
    (dict(p=params(eps=-1.0)), INVALID), (dict(p=params(eps=float("nan"))), INVALID),
    (dict(p=params(post_weight=None), post_rstd=at(4)), INVALID),
    (dict(p=params(pre_weight=None)), INVALID),  # z wanted
    (dict(p=params(pre_weight=None), z=K.ptored_rows(), pre_rstd=at(4)), INVALID),
    (dict(h_kept=kept(5, D - 1)), INVALID), (dict(x_kept=kept(5, D, 1)), INVALID),
    (dict(z_kept=K.ptored_checkpoint(at(5), D, None, 2)), INVALID),
    (dict(p=params(dtype=3)), UNSUPPORTED), (dict(p=params(dtype=-1)), UNSUPPORTED),
    (dict(p=params(weight_dtype=2)), UNSUPPORTED), (dict(p=params(weight_dtype=3)), UNSUPPORTED),
    (dict(p=params(cols=16385, gate=rows(22, 16385)), part_ld=16385, x=rows(0, 16385),
          x_out=rows(1, 16385), z=rows(2, 16385)), UNSUPPORTED),
    (dict(x=K.ptored_rows(at(0) + 1, D)), INVALID),
    (dict(p=params(post_weight=at(20) + 2)), INVALID), (dict(pre_rstd=at(4) + 2), INVALID),
    (dict(x_out=K.ptored_rows(at(0) + 2, D)), OVERLAP), (dict(x_out=rows(0, D + 8)), OVERLAP),
    (dict(z=rows(1)), OVERLAP), (dict(h=rows(1)), OVERLAP),
    (dict(z=rows(20, D)), OVERLAP), (dict(pre_rstd=at(1)), OVERLAP),
    (dict(x_kept=kept(0)), OVERLAP), (dict(x_kept=kept(5), h_kept=kept(5)), OVERLAP),
    (dict(x_out=rows(22)), OVERLAP),
])
def test_forward_refusals(kw, status):
    assert norm(**kw) == status


def test_forward_takes_null_structs_and_empty_shapes():
    assert crc.ptored_block_norm([], 0, 0, None, io(), 0) == INVALID
    assert crc.ptored_block_norm([], 0, 0, params(), None, 0) == INVALID
    assert norm(p=params(rows=0)) == 0
    assert norm(p=params(cols=0, gate=rows(22, 0))) == 0
    assert norm(p=params(rows=0), x_out=rows(0), h=rows(30)) == 0


def grad(p=None, **kw):
    return crc.ptored_block_norm_backward(params() if p is None else p, grad_io(**kw), 0)


NONE = K.ptored_rows()


@pytest.mark.parametrize("kw,status", [
    (dict(dz=NONE), INVALID), (dict(p=params(pre_weight=None)), INVALID),
    (dict(p=params(pre_weight=None), dz=NONE, dx_out=NONE, dpre_weight=None), INVALID),
    (dict(x_out=NONE), INVALID), (dict(h=NONE), INVALID), (dict(pre_rstd=None), INVALID),
    (dict(post_rstd=None), INVALID), (dict(x_kept=kept(12)), INVALID),
    (dict(x_out=NONE, h=NONE, x_kept=kept(12)), INVALID),
    (dict(p=params(post_weight=None)), INVALID),  # dpost_weight wanted
    (dict(p=params(gate=NONE)), INVALID),  # dgate wanted
    (dict(p=params(gate_rows=3)), INVALID), (dict(dh=rows(7, D - 1)), INVALID),
    (dict(workspace=None), INVALID), (dict(workspace_bytes=T * D * 12 - 1), INVALID),
    (dict(workspace=at(11) + 8), INVALID),
    (dict(p=params(dtype=3)), UNSUPPORTED), (dict(p=params(weight_dtype=2)), UNSUPPORTED),
    (dict(dx=rows(6), dh=rows(6)), OVERLAP), (dict(dx=rows(0, D + 2)), OVERLAP),
    (dict(dgate=rows(22)), OVERLAP), (dict(dpre_weight=at(21)), OVERLAP),
    (dict(workspace=at(6)), OVERLAP), (dict(dpost_weight=at(10)), OVERLAP),
])
def test_backward_refusals(kw, status):
    assert grad(**kw) == status


def test_checkpoint_refusals():
    pk, un = crc.ptored_checkpoint_pack, crc.ptored_checkpoint_unpack
    assert pk(K.ptored_rows(), T, D, 1, kept(1), 0) == INVALID
    assert pk(rows(0), T, D, 1, K.ptored_checkpoint(), 0) == INVALID
    assert pk(rows(0), -1, D, 1, kept(1), 0) == INVALID
    assert pk(rows(0, D - 1), T, D, 1, kept(1), 0) == INVALID
    assert pk(rows(0), T, D, 1, kept(1, D, 1), 0) == INVALID
    assert pk(rows(0), T, D, 3, kept(1), 0) == UNSUPPORTED
    assert pk(K.ptored_rows(at(0) + 1, D), T, D, 1, kept(1), 0) == INVALID
    assert pk(rows(0), T, D, 1, kept(0), 0) == OVERLAP
    assert un(kept(0), T, D, 1, rows(0), 0) == OVERLAP
    assert un(kept(1), T, D, 9, rows(0), 0) == UNSUPPORTED
    assert pk(rows(0), 0, D, 1, kept(1), 0) == 0
    assert un(kept(1), T, 0, 1, rows(0), 0) == 0


def test_wgrad_refusals():
    def call(dy=None, x=None, t=T, o=D, i=D, dt=1, dw=None, wt=0, acc=0, ws=at(11), n=1 << 30):
        return crc.ptored_checkpoint_wgrad(rows(0) if dy is None else dy,
                                           kept(1) if x is None else x, t, o, i, dt,
                                           rows(2) if dw is None else dw, wt, acc, ws, n, 0)

    assert call(dy=K.ptored_rows()) == INVALID
    assert call(x=K.ptored_checkpoint()) == INVALID
    assert call(dw=K.ptored_rows()) == INVALID
    assert call(t=-1) == INVALID
    assert call(dw=rows(2, D - 1)) == INVALID
    assert call(dt=3) == UNSUPPORTED
    assert call(wt=2) == UNSUPPORTED
    assert call(dw=K.ptored_rows(at(2) + 2, D)) == INVALID
    assert call(dw=rows(0), wt=1) == OVERLAP
    assert call(dw=rows(1)) == OVERLAP
    assert call(o=0) == 0 and call(i=0) == 0 and call(t=0, acc=1) == 0
    st, need = crc.ptored_checkpoint_wgrad_workspace(1 << 15, D, D, 1)
    assert st == 0 and need > 0  # few outputs, many tokens: split
    assert call(t=1 << 15, x=kept(1), n=need - 1) == INVALID
    assert call(t=1 << 15, ws=None) == INVALID
    assert call(t=1 << 15, ws=at(11) + 4) == INVALID
    assert call(t=1 << 15, ws=at(2)) == OVERLAP


def test_workspace_sizes():
    ws = crc.ptored_block_norm_backward_workspace
    assert ws(0, 100, 0) == (0, 0)
    assert ws(8, 64, 3)[0] == INVALID
    assert ws(-1, 64, 0)[0] == INVALID
    assert ws(8, 16385, 0)[0] == UNSUPPORTED
    assert ws(8, 64, 0) == (0, 8 * 64 * 8)
    assert ws(8, 64, 8) == (0, 8 * 64 * 8)  # a gate row per row needs no partial sums
    assert ws(8, 64, 1) == (0, 8 * 64 * 12)
    assert crc.block_norm_backward_workspace(1 << 20, 4096) <= 1 << 27  # does not grow with rows
    with pytest.raises(crc.PtoredError):
        crc.block_norm_backward_workspace(8, 16385)
    assert crc.ptored_checkpoint_wgrad_workspace(8, 1 << 14, 1 << 14, 1) == (0, 0)
    assert crc.ptored_checkpoint_wgrad_workspace(8, 64, 64, 3)[0] == UNSUPPORTED
    with pytest.raises(TypeError):
        crc.checkpoint_wgrad_workspace(8, 64, 64, torch.float64)


def test_tensor_wrappers_refuse_before_the_library():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):  # not on a GPU
        crc.block_norm([x], x, x)
    with pytest.raises(TypeError):
        crc.block_norm([], torch.zeros(4, 64, dtype=torch.float64))
    with pytest.raises(ValueError):
        crc.block_norm([], torch.zeros(64))
    with pytest.raises(ValueError):
        crc.block_norm_backward(None, None, None, None)
    with pytest.raises(ValueError):
        crc.checkpoint_pack(x, crc.checkpoint_empty(4, 64, "cpu"))
    k = crc.checkpoint_empty(3, 65, "cpu")
    assert k.q.shape == (3, 65) and k.scales.shape == (3, 3)


def test_constants_and_struct_sizes_match_the_header(tmp_path):
    """include/ptored_block.h as C11 against the binding's structures."""
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    names = ("ptored_rows", "ptored_checkpoint", "ptored_block_params", "ptored_block_io",
             "ptored_block_grad_io")
    src = tmp_path / "s.c"
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "ptored_block.h"', "int main(void) {",
             'printf("%d %d\\n", PTORED_BLOCK_MAX_COLS, PTORED_CHECKPOINT_BLOCK);']
    for n in names:
        for f, _ in getattr(K, n)._fields_:
            lines.append(f'printf("%zu ", offsetof({n}, {f}));')
        lines.append(f'printf("%zu\\n", sizeof({n}));')
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = str(tmp_path / "s")
    subprocess.run([gcc, "-std=c11", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__",
                    "-I" + os.path.join(ROOT, "include"), "-I/opt/rocm/include", str(src), "-o",
                    exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()
    assert out[0].split() == [str(K.PTORED_BLOCK_MAX_COLS), str(K.PTORED_CHECKPOINT_BLOCK)]
    for n, line in zip(names, out[1:]):
        s = getattr(K, n)
        want = [getattr(s, f).offset for f, _ in s._fields_] + [ctypes.sizeof(s)]
        assert [int(v) for v in line.split()] == want, n


# ------------------------------------------------------- the reference itself

@pytest.mark.parametrize("post,pre,groups,offset", [
    (True, True, 1, 0.0), (True, True, 3, 1.0), (True, True, 6, 0.0), (True, True, 0, 0.0),
    (False, True, 2, 0.0), (True, False, 1, 0.0), (False, True, 0, 1.0), (False, False, 6, 0.0)])
def test_reference_gradients_against_differences(post, pre, groups, offset):
    torch.manual_seed(3)
    t, d = 6, 10
    kw = dict(offset=offset, alpha=0.7, beta=1.3)
    v = {"x": torch.randn(t, d), "h": torch.randn(t, d)}
    if post:
        v["w1"] = 1 + 0.3 * torch.randn(d)
    if pre:
        v["w2"] = 1 + 0.3 * torch.randn(d)
    if groups:
        v["gate"] = torch.randn(groups, d)
    v = {k: t_.double() for k, t_ in v.items()}
    cz, cx = torch.randn(t, d).double(), torch.randn(t, d).double()

    def loss(v):
        f = R.forward([v["h"]], v["x"], v.get("w1"), v.get("gate"), v.get("w2"), eps=1e-5, **kw)
        total = (f["x_out"][0] * cx).sum()
        return total + (f["z"][0] * cz).sum() if pre else total

    f = R.forward([v["h"]], v["x"], v.get("w1"), v.get("gate"), v.get("w2"), eps=1e-5, **kw)
    g = R.backward(cz if pre else None, cx, f["x_out"][0], v["h"], f["r1"][0] if post else None,
                   f["r2"][0] if pre else None, v.get("w1"), v.get("gate"), v.get("w2"), **kw)
    for name, key in (("x", "dx"), ("h", "dh"), ("w1", "dw1"), ("w2", "dw2"), ("gate", "dgate")):
        if name not in v:
            assert key not in g
            continue
        got = g[key][0]
        assert got.shape == v[name].shape
        step = 1e-5
        for _ in range(3):
            way = torch.randn_like(v[name])
            up = loss({**v, name: v[name] + step * way})
            down = loss({**v, name: v[name] - step * way})
            # central differences in 64 bits: step^2 of the third derivative
            # and 1e-16 / step of the loss, both about 1e-10
            want = (up - down) / (2 * step)
            assert abs((got * way).sum() - want) < 1e-7 * (1 + abs(want)), (name, key)


def test_reference_packing_holds_its_definition():
    torch.manual_seed(1)
    x = (torch.randn(40, 70) * torch.exp(3 * torch.randn(70))).float()
    x[3, :32] = 0
    x[4, 5] = 2.0 ** 100
    q, s = R.pack(x)
    back = R.unpack(q, s)
    step = torch.exp2(s.double().repeat_interleave(32, 1)[:, :70] - 133)
    assert bool(((back - x.double()).abs() <= step / 2).all())
    top = torch.nn.functional.pad(q.abs().int(), (0, 26)).view(40, 3, 32).amax(-1)
    used = s > 7
    assert bool((top[used] >= 64).all())  # the smallest exponent that holds the block
    assert bool((back.to(torch.bfloat16).double() == back).all())
    v = torch.tensor([[127.5 / 64, 0.5], [127.49 / 64, 0.5], [float("inf"), 1.0]])
    q, s = R.pack(v)
    assert q.tolist() == [[64, 16], [127, 32], [0, 0]] and s.tolist() == [[128], [127], [255]]
