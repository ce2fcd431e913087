"""Block-boundary calls on the GPU as callers make them: the C ABI's own
conventions, buffers reused in place or far apart, values at the ends of the
types' ranges.  References and bounds as in tests/test_block_gpu.py."""

import ctypes

import pytest
import torch

import cross_rank_collective_amd as crc
from cross_rank_collective_amd import block as K
from tests.test_block_gpu import draw, say

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
