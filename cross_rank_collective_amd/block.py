"""The block boundary after a cross-rank reduction, and 8-bit activation
checkpoints: ctypes binding and tensor-level calls (``include/ptored_block.h``).

A tensor-parallel block ends with N ranks' partial outputs.  ``block_norm``
folds them, normalises, gates and scales the fold, adds it to the residual
stream and normalises the result for the next block, in one pass over the
data; ``block_norm_backward`` takes its gradients.  ``checkpoint_pack`` keeps
an activation in 8 bits (32 elements of a row share a power of two),
``checkpoint_unpack`` reads it back, and the backward pass and
``checkpoint_wgrad`` (a projection's weight gradient) take it as it is.

As in ``binding``, every step runs in the library's HIP kernels: these
functions check tensors, hand over pointers and raise on errors.  Calls whose
tensors fit as they are go through ``_torch_calls.so``, the rest (and every
error) through the Python code below; both make the same library call.  Outputs are
the caller's tensors; nothing is allocated but, where none is given, the
workspace of a backward pass (from torch's allocator, on the call's stream).
Calls are asynchronous on ``stream`` (default: torch's current stream).  A
caller that uses tensors on another stream than the one they were allocated on
keeps them alive until that stream is done, as with every torch call.

These are not differentiable functions of autograd: a call records nothing,
whatever requires a gradient, and its gradients are calls of their own
(``block_norm_backward``, ``checkpoint_wgrad``).  Outputs count as changed in
place, so autograd refuses to use a tensor that it saved before such a call
wrote it.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

from . import binding as B

PTORED_BLOCK_MAX_COLS = 16384
PTORED_CHECKPOINT_BLOCK = 32

_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class ptored_rows(ctypes.Structure):
    _fields_ = [("data", _vp), ("ld", _i64)]


class ptored_checkpoint(ctypes.Structure):
    _fields_ = [("q", _vp), ("q_ld", _i64), ("scales", _vp), ("scales_ld", _i64)]


class ptored_block_params(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i64), ("post_weight", _vp), ("pre_weight", _vp),
                ("gate", ptored_rows), ("gate_rows", _i64), ("weight_offset", _f32),
                ("branch_scale", _f32), ("residual_scale", _f32), ("eps", _f32),
                ("dtype", _i32), ("weight_dtype", _i32)]


class ptored_block_io(ctypes.Structure):
    _fields_ = [("x", ptored_rows), ("x_out", ptored_rows), ("z", ptored_rows),
                ("h", ptored_rows), ("post_rstd", _vp), ("pre_rstd", _vp),
                ("h_kept", ptored_checkpoint), ("x_kept", ptored_checkpoint),
                ("z_kept", ptored_checkpoint)]


class ptored_block_grad_io(ctypes.Structure):
    _fields_ = [("dz", ptored_rows), ("dx_out", ptored_rows), ("x_out", ptored_rows),
                ("h", ptored_rows), ("x_kept", ptored_checkpoint),
                ("h_kept", ptored_checkpoint), ("post_rstd", _vp), ("pre_rstd", _vp),
                ("dx", ptored_rows), ("dh", ptored_rows), ("dgate", ptored_rows),
                ("dpost_weight", _vp), ("dpre_weight", _vp), ("workspace", _vp),
                ("workspace_bytes", _i64)]


class Checkpoint(NamedTuple):
    """A T x D activation in 8 bits: ``q`` int8 [T, D] and ``scales`` uint8
    [T, ceil(D / 32)].  Any pair of such tensors serves as one."""

    q: "torch.Tensor"  # noqa: F821
    scales: "torch.Tensor"  # noqa: F821


_lib = None


def _load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = B.load()
        P = ctypes.POINTER
        lib.ptored_block_norm.argtypes = [P(_vp), ctypes.c_int, _i64, P(ptored_block_params),
                                          P(ptored_block_io), _vp]
        lib.ptored_block_norm_backward.argtypes = [P(ptored_block_params),
                                                   P(ptored_block_grad_io), _vp]
        lib.ptored_block_norm_backward_workspace.argtypes = [_i64, _i64, _i64, P(_i64)]
        lib.ptored_checkpoint_pack.argtypes = [ptored_rows, _i64, _i64, ctypes.c_int,
                                               ptored_checkpoint, _vp]
        lib.ptored_checkpoint_unpack.argtypes = [ptored_checkpoint, _i64, _i64, ctypes.c_int,
                                                 ptored_rows, _vp]
        lib.ptored_checkpoint_wgrad.argtypes = [ptored_rows, ptored_checkpoint, _i64, _i64, _i64,
                                                ctypes.c_int, ptored_rows, ctypes.c_int,
                                                ctypes.c_int, _vp, _i64, _vp]
        lib.ptored_checkpoint_wgrad_workspace.argtypes = [_i64, _i64, _i64, ctypes.c_int, P(_i64)]
        for name in ("ptored_block_norm", "ptored_block_norm_backward",
                     "ptored_block_norm_backward_workspace", "ptored_checkpoint_pack",
                     "ptored_checkpoint_unpack", "ptored_checkpoint_wgrad",
                     "ptored_checkpoint_wgrad_workspace"):
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


# ---------------------------------------------------------------- raw calls

def ptored_block_norm(parts, nranks: int, part_ld: int, params: ptored_block_params,
                      io: ptored_block_io, stream: int) -> int:
    """Raw call: ``parts`` are device pointers as ints; returns the status code."""
    return _load().ptored_block_norm(B._ptrs(parts), nranks, part_ld, params, io, stream)


def ptored_block_norm_backward(params: ptored_block_params, io: ptored_block_grad_io,
                               stream: int) -> int:
    return _load().ptored_block_norm_backward(params, io, stream)


def ptored_block_norm_backward_workspace(rows: int, cols: int, gate_rows: int):
    out = _i64()
    st = _load().ptored_block_norm_backward_workspace(rows, cols, gate_rows, out)
    return st, out.value


def ptored_checkpoint_pack(x: ptored_rows, rows: int, cols: int, dtype: int,
                           kept: ptored_checkpoint, stream: int) -> int:
    return _load().ptored_checkpoint_pack(x, rows, cols, dtype, kept, stream)


def ptored_checkpoint_unpack(kept: ptored_checkpoint, rows: int, cols: int, dtype: int,
                             out: ptored_rows, stream: int) -> int:
    return _load().ptored_checkpoint_unpack(kept, rows, cols, dtype, out, stream)


def ptored_checkpoint_wgrad(dy: ptored_rows, x: ptored_checkpoint, rows: int, outs: int, cols: int,
                            dtype: int, dw: ptored_rows, dw_dtype: int, accumulate: int,
                            workspace: int, workspace_bytes: int, stream: int) -> int:
    return _load().ptored_checkpoint_wgrad(dy, x, rows, outs, cols, dtype, dw, dw_dtype,
                                           accumulate, workspace, workspace_bytes, stream)


def ptored_checkpoint_wgrad_workspace(rows: int, outs: int, cols: int, dtype: int):
    out = _i64()
    st = _load().ptored_checkpoint_wgrad_workspace(rows, outs, cols, dtype, out)
    return st, out.value


# ---------------------------------------------------------------- tensors

def _is_kept(v) -> bool:
    return isinstance(v, (tuple, list))


_NO_ROWS = ptored_rows()
_NO_KEPT = ptored_checkpoint()
_torch = None
_native = None  # the extension module of the tensor calls
_FLOATS = {}  # torch dtype -> C ABI code, with the next three filled on first use
_FLOAT32 = _INT8 = _UINT8 = None


def _init() -> None:
    global _torch, _native, _FLOAT32, _INT8, _UINT8
    import torch

    _load()
    try:
        from . import _torch_calls
    except ImportError as e:
        raise RuntimeError("the extension of the tensor calls is missing or was built for another "
                           "torch: build it with `python -m cross_rank_collective_amd.build`") from e
    _native = _torch_calls

    _FLOAT32, _INT8, _UINT8 = torch.float32, torch.int8, torch.uint8
    _FLOATS.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
    _torch = torch


def _float_code(dtype, what: str) -> int:
    code = _FLOATS.get(dtype)
    if code is None:
        raise TypeError(f"{what} must be float32, bfloat16 or float16, not {dtype}")
    return code


def _pitch(t, rows: int, cols: int, what: str) -> int:
    """Row pitch of a 2-D row-major tensor with unit column stride."""
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{what} must be row-major with unit column stride")
    if rows <= 1:
        return s0 if s0 > cols else cols  # a single row has no pitch of its own
    if s0 < cols:
        raise ValueError(f"{what}: rows overlap (a broadcast tensor? pass it unexpanded)")
    return s0


class _Group:
    """The shape, type and device that a call's tensors have to share.

    A tensor that fits passes with plain comparisons, and only one that does
    not is looked at again for the error to raise.
    """

    __slots__ = ("rows", "cols", "shape", "dtype", "index", "code")

    def __init__(self, t, what: str):
        if _torch is None:
            _init()
        if t.dim() != 2:
            raise ValueError(f"{what} must be 2-D (rows x columns)")
        self.shape = t.shape
        self.rows, self.cols = t.shape
        self.dtype = t.dtype
        self.code = _float_code(t.dtype, what)
        self.index = t.get_device()
        if self.index < 0 or not t.is_cuda:
            raise ValueError(f"{what} must be on a GPU")

    def _misfit(self, t, dtype, shape, what):
        if t.dtype != dtype or tuple(t.shape) != tuple(shape):
            raise ValueError(f"{what} must be {dtype} of shape {tuple(shape)}, not {t.dtype} of "
                             f"{tuple(t.shape)}")
        raise ValueError(f"{what} must be on cuda:{self.index}")

    def mat(self, t, what: str) -> ptored_rows:
        """A [T, D] tensor of the group's type, or None."""
        if t is None:
            return _NO_ROWS
        if t.dtype is not self.dtype or t.shape != self.shape or t.get_device() != self.index:
            self._misfit(t, self.dtype, self.shape, what)
        s0, s1 = t.stride()
        if s1 != 1 or s0 < self.cols:
            s0 = _pitch(t, self.rows, self.cols, what)
        return ptored_rows(t.data_ptr(), s0)

    def other(self, t, what: str, rows: int, cols: int, dtype) -> ptored_rows:
        """A tensor of another shape or type on the group's device."""
        if t.dtype is not dtype or t.shape != (rows, cols) or t.get_device() != self.index:
            self._misfit(t, dtype, (rows, cols), what)
        return ptored_rows(t.data_ptr(), _pitch(t, rows, cols, what))

    def kept(self, k, what: str, cols: Optional[int] = None) -> ptored_checkpoint:
        if k is None:
            return _NO_KEPT
        q, s = k
        cols = self.cols if cols is None else cols
        blocks = (cols + PTORED_CHECKPOINT_BLOCK - 1) // PTORED_CHECKPOINT_BLOCK
        qr = self.other(q, what + "'s values", self.rows, cols, _INT8)
        sr = self.other(s, what + "'s scales", self.rows, blocks, _UINT8)
        return ptored_checkpoint(qr.data, qr.ld, sr.data, sr.ld)

    def vec(self, t, n: int, dtype, what: str) -> Optional[int]:
        if t is None:
            return None
        if t.dtype is not dtype or t.shape != (n,) or t.get_device() != self.index:
            self._misfit(t, dtype, (n,), what)
        if n > 1 and t.stride(0) != 1:
            raise ValueError(f"{what} must be contiguous")
        return t.data_ptr()

    def params(self, post_weight, pre_weight, gate, eps, weight_offset, branch_scale,
               residual_scale) -> ptored_block_params:
        w = pre_weight if post_weight is None else post_weight
        wt = self.dtype if w is None else w.dtype
        code = self.code if wt is self.dtype else _float_code(wt, "weights")
        if code not in (0, self.code):
            raise TypeError("weights must be float32 or of the activations' type")
        gate_rows, g = 0, _NO_ROWS
        if gate is not None:
            if gate.dim() == 1:
                gate = gate.unsqueeze(0)
            gate_rows = gate.shape[0]
            if gate.dim() != 2 or gate_rows == 0 or self.rows % gate_rows:
                raise ValueError("gate must be [D] or [G, D] with G a divisor of the rows")
            g = self.other(gate, "gate", gate_rows, self.cols, self.dtype)
        return ptored_block_params(
            self.rows, self.cols, self.vec(post_weight, self.cols, wt, "post_weight"),
            self.vec(pre_weight, self.cols, wt, "pre_weight"), g, gate_rows, weight_offset,
            branch_scale, residual_scale, eps, self.code, code)

    def run(self, stream, call, *args) -> None:
        """``call(*args, stream handle)`` with the group's GPU current, raising on errors."""
        handle = B._stream_handle(stream, self.index)
        if _torch.cuda.current_device() == self.index:
            status = call(*args, handle)
        else:
            with _torch.cuda.device(self.index):
                status = call(*args, handle)
        if status:
            B._raise_on(status)


def _wrote(*outputs) -> None:
    """Outputs of a call that was made: tensors, kept pairs or None."""
    for t in outputs:
        if _is_kept(t):
            _wrote(*t)
        elif t is not None:
            _torch.autograd.graph.increment_version(t)


def _native_call(name: str, stream, *args) -> bool:
    """The call on tensors that fit as they are, made natively: False where the
    code that follows has to look again (and make the call, or say what does
    not fit)."""
    if _native is None:
        _init()
    handle = stream if stream is None else B._stream_handle(stream, None)
    status = getattr(_native, name)(*args, handle)
    if status:
        B._raise_on(status)
    return status is not None


def _torch_stream(stream, index):
    """torch's object for the stream of a call."""
    if stream is None:
        return _torch.cuda.current_stream(index)
    if hasattr(stream, "cuda_stream"):
        return stream
    return _torch.cuda.ExternalStream(int(stream), device=index)


def _zero(tensors, index, stream) -> None:
    """Sums over no rows, on the call's stream."""
    with _torch.cuda.stream(_torch_stream(stream, index)):
        for t in tensors:
            if t is not None:
                t.zero_()


def _workspace(nbytes: int, given, index, stream):
    """(tensor to keep until the call is made, pointer, bytes)."""
    if given is not None:
        if given.get_device() != index or not given.is_contiguous():
            raise ValueError("workspace must be contiguous and on the call's GPU")
        return given, given.data_ptr(), given.numel() * given.element_size()
    if nbytes == 0:
        return None, None, 0
    if stream is None:
        t = _torch.empty(nbytes, dtype=_UINT8, device=index)
    else:  # belongs to the stream that uses it, so that it is not reused too early
        with _torch.cuda.stream(_torch_stream(stream, index)):
            t = _torch.empty(nbytes, dtype=_UINT8, device=index)
    return t, t.data_ptr(), nbytes


def block_norm(parts, x, x_out=None, z=None, *, post_weight=None, gate=None, pre_weight=None,
               eps: float = 1e-6, weight_offset: float = 0.0, branch_scale: float = 1.0,
               residual_scale: float = 1.0, h=None, post_rstd=None, pre_rstd=None, h_kept=None,
               x_kept=None, z_kept=None, stream=None) -> None:
    """The block boundary, forward, into the outputs that are given:

        h     = parts[0] + ... + parts[N-1]
        p     = h r1 (post_weight + weight_offset), r1 = 1/sqrt(mean(h^2) + eps)
        x_out = residual_scale x + branch_scale gate p
        z     = x_out r2 (pre_weight + weight_offset), r2 = 1/sqrt(mean(x_out^2) + eps)

    ``parts`` (0 to 64 ranks' partial outputs), ``x``, ``x_out``, ``z`` and
    ``h`` are [T, D] of one floating type; without ``post_weight`` p = h,
    without ``pre_weight`` there is no z.  ``gate`` is [D] or [G, D], each row
    for T / G consecutive rows.  Weights are float32 or of the activations'
    type.  For the backward pass: ``h`` (with one rank, parts[0] is h),
    ``post_rstd`` and ``pre_rstd`` (float32 [T]), and ``h_kept``, ``x_kept``,
    ``z_kept``, the 8-bit forms of h, x_out and z.  ``x_out`` may be ``x``.
    """
    if _native_call("block_norm", stream, parts, x, x_out, z, post_weight, gate, pre_weight, eps,
                    weight_offset, branch_scale, residual_scale, h, post_rstd, pre_rstd, h_kept,
                    x_kept, z_kept):
        return
    g = _Group(x, "x")
    ptrs, part_ld = [], g.cols
    for t in parts:
        part = g.mat(t, "every part" if ptrs else "parts[0]")
        if not ptrs:
            part_ld = part.ld
        elif part.ld != part_ld and g.rows > 1:  # a single row has no pitch
            raise ValueError("every part must have the same strides")
        ptrs.append(part.data)
    params = g.params(post_weight, pre_weight, gate, eps, weight_offset, branch_scale,
                      residual_scale)
    io = ptored_block_io(g.mat(x, "x"), g.mat(x_out, "x_out"), g.mat(z, "z"), g.mat(h, "h"),
                         g.vec(post_rstd, g.rows, _FLOAT32, "post_rstd"),
                         g.vec(pre_rstd, g.rows, _FLOAT32, "pre_rstd"),
                         g.kept(h_kept, "h_kept"), g.kept(x_kept, "x_kept"),
                         g.kept(z_kept, "z_kept"))
    if g.rows == 0 or g.cols == 0:
        return  # empty tensors have no storage
    g.run(stream, ptored_block_norm, ptrs, len(ptrs), part_ld, params, io)
    _wrote(x_out, z, h, post_rstd, pre_rstd, h_kept, x_kept, z_kept)


def block_norm_backward_workspace(rows: int, cols: int, gate_rows: int = 0) -> int:
    """Bytes of workspace of ``block_norm_backward``; ``gate_rows`` 0 where no
    gate gradient is asked for."""
    st, n = ptored_block_norm_backward_workspace(rows, cols, gate_rows)
    B._raise_on(st)
    return n


def block_norm_backward(dz, dx_out, x_out, pre_rstd, dx=None, dh=None, *, h=None, post_rstd=None,
                        post_weight=None, gate=None, pre_weight=None, dpost_weight=None,
                        dgate=None, dpre_weight=None, weight_offset: float = 0.0,
                        branch_scale: float = 1.0, residual_scale: float = 1.0, workspace=None,
                        stream=None) -> None:
    """Gradients of ``block_norm``, into the outputs that are given.

    ``dz`` is z's gradient (None without ``pre_weight``), ``dx_out`` the one
    that reaches x_out from further on (or None).  ``x_out`` and ``h`` are the
    forward pass's activations, both as tensors or both as 8-bit checkpoints;
    ``post_rstd`` and ``pre_rstd`` are its reciprocal norms.  ``dx`` is the
    residual stream's gradient, ``dh`` that of the fold and so of every rank's
    partial output; ``dgate``, ``dpost_weight`` and ``dpre_weight`` have the
    shapes and types of what they are gradients of.  ``dx`` and ``dh`` may be
    any of the [T, D] inputs.
    """
    if _native_call("block_norm_backward", stream, dz, dx_out, x_out, pre_rstd, dx, dh, h,
                    post_rstd, post_weight, gate, pre_weight, 0.0, weight_offset, branch_scale,
                    residual_scale, dpost_weight, dgate, dpre_weight, workspace):
        return
    ref = dz if dz is not None else dx_out
    if ref is None:
        raise ValueError("block_norm_backward needs dz, dx_out or both")
    g = _Group(ref, "dz" if dz is not None else "dx_out")
    params = g.params(post_weight, pre_weight, gate, 0.0, weight_offset, branch_scale,
                      residual_scale)
    packed = _is_kept(x_out) or _is_kept(h)
    if packed and not all(v is None or _is_kept(v) for v in (x_out, h)):
        raise ValueError("x_out and h must both be tensors or both be checkpoints")
    wt = _FLOAT32 if params.weight_dtype == 0 else g.dtype
    gate_rows, dgate_rows = _NO_ROWS, 0
    if dgate is not None:
        if dgate.dim() == 1:
            dgate = dgate.unsqueeze(0)
        dgate_rows = params.gate_rows
        gate_rows = g.other(dgate, "dgate", dgate_rows, g.cols, g.dtype)
    io = ptored_block_grad_io(
        g.mat(dz, "dz"), g.mat(dx_out, "dx_out"),
        _NO_ROWS if packed else g.mat(x_out, "x_out"), _NO_ROWS if packed else g.mat(h, "h"),
        g.kept(x_out, "x_out") if packed else _NO_KEPT,
        g.kept(h, "h") if packed else _NO_KEPT,
        g.vec(post_rstd, g.rows, _FLOAT32, "post_rstd"),
        g.vec(pre_rstd, g.rows, _FLOAT32, "pre_rstd"), g.mat(dx, "dx"), g.mat(dh, "dh"),
        gate_rows, g.vec(dpost_weight, g.cols, wt, "dpost_weight"),
        g.vec(dpre_weight, g.cols, wt, "dpre_weight"), None, 0)
    if g.cols == 0:
        return
    if g.rows == 0:  # nothing to read; the sums over no rows are zero
        _zero((dgate, dpost_weight, dpre_weight), g.index, stream)
        return
    nbytes = 0
    if g.cols <= PTORED_BLOCK_MAX_COLS and not (
            dgate is None and dpost_weight is None and dpre_weight is None):
        nbytes = block_norm_backward_workspace(g.rows, g.cols, dgate_rows)
    keep, io.workspace, io.workspace_bytes = _workspace(nbytes, workspace, g.index, stream)
    g.run(stream, ptored_block_norm_backward, params, io)
    _wrote(dx, dh, dpost_weight, dgate, dpre_weight)


def checkpoint_empty(rows: int, cols: int, device="cuda") -> Checkpoint:
    """Room for a rows x cols activation in 8 bits."""
    import torch

    blocks = (cols + PTORED_CHECKPOINT_BLOCK - 1) // PTORED_CHECKPOINT_BLOCK
    return Checkpoint(torch.empty(rows, cols, dtype=torch.int8, device=device),
                      torch.empty(rows, blocks, dtype=torch.uint8, device=device))


def checkpoint_pack(x, kept, stream=None) -> None:
    """``kept`` = the 8-bit form of ``x`` ([T, D] of a floating type): each
    value to within half a step, a step being 1/64 of the power of two below
    the largest magnitude of its block of 32 (or 1/32 where that magnitude
    comes within 1/256 of the next power).  A block with an infinity or a NaN
    stands for NaN."""
    if _native_call("checkpoint_pack", stream, x, kept):
        return
    g = _Group(x, "x")
    xm, k = g.mat(x, "x"), g.kept(kept, "kept")
    if g.rows and g.cols:
        g.run(stream, ptored_checkpoint_pack, xm, g.rows, g.cols, g.code, k)
        _wrote(kept)


def checkpoint_unpack(kept, out, stream=None) -> None:
    """``out`` = the values kept (exact in float32 and bfloat16)."""
    if _native_call("checkpoint_unpack", stream, kept, out):
        return
    g = _Group(out, "out")
    om, k = g.mat(out, "out"), g.kept(kept, "kept")
    if g.rows and g.cols:
        g.run(stream, _unpack_into, om, k, g.rows, g.cols, g.code)
        _wrote(out)


def _unpack_into(om, k, rows, cols, code, stream):
    return ptored_checkpoint_unpack(k, rows, cols, code, om, stream)


def checkpoint_wgrad_workspace(rows: int, outs: int, cols: int, dtype) -> int:
    """Bytes of workspace of ``checkpoint_wgrad``; ``dtype`` is dy's."""
    st, n = ptored_checkpoint_wgrad_workspace(rows, outs, cols, B._dtype_code(dtype))
    B._raise_on(st)
    return n


def checkpoint_wgrad(dy, kept, dw, accumulate: bool = False, workspace=None, stream=None) -> None:
    """dw = dy^T x (or dw += dy^T x): the weight gradient of y = x W^T from
    ``dy`` [T, O] and the kept input x [T, I], into ``dw`` [O, I], float32 or
    of dy's type.  Products are exact and sums in float32."""
    if _native_call("checkpoint_wgrad", stream, dy, kept, dw, accumulate, workspace):
        return
    g = _Group(dy, "dy")
    if dw.dim() != 2 or dw.shape[0] != g.cols:
        raise ValueError("dw must be [dy's columns, x's columns]")
    if kept[0].dim() != 2 or kept[0].shape[0] != g.rows:
        raise ValueError("dy and the kept input must have the same rows")
    code = _float_code(dw.dtype, "dw")
    if code not in (0, g.code):
        raise TypeError("dw must be float32 or of dy's type")
    dym = g.mat(dy, "dy")
    outs, cols = dw.shape
    dwm = g.other(dw, "dw", outs, cols, dw.dtype)
    k = g.kept(kept, "kept", cols)
    if outs == 0 or cols == 0 or (g.rows == 0 and accumulate):
        return
    if g.rows == 0:  # the sum over no rows
        _zero((dw,), g.index, stream)
        return
    st, nbytes = ptored_checkpoint_wgrad_workspace(g.rows, outs, cols, g.code)
    B._raise_on(st)
    keep, ptr, given = _workspace(nbytes, workspace, g.index, stream)
    g.run(stream, ptored_checkpoint_wgrad, dym, k, g.rows, outs, cols, g.code, dwm, code,
          1 if accumulate else 0, ptr, given)
    _wrote(dw)
