"""What a tensor-parallel step runs next to the reduction and the block
boundary: ctypes binding and tensor-level calls (``include/ptored_step.h``).

``layer_norm`` is the boundary of a model with layer norm: it folds the ranks'
partial outputs into the residual stream and normalises the result, in one pass;
``layer_norm_backward`` takes its gradients.  ``gated_ffn`` is the column-parallel
half of a gated feed-forward block, both projections, the activation and the
product in one kernel; ``gated_ffn_backward`` takes its gradients.
``grad_norm``, ``grad_scale`` and ``grad_clip`` take the norm over many gradients
and clip them by it, without the host waiting for the norm.

Conventions are those of ``block``: outputs are the caller's tensors, calls are
asynchronous on ``stream`` (default: torch's current stream), allocate nothing
but a workspace where none is given, record nothing for autograd, and count as
changes in place of their outputs.
"""

from __future__ import annotations

import ctypes

from . import binding as B
from . import block as K
from .block import _f32, _i32, _i64, _vp, ptored_rows

PTORED_FFN_MAX_PITCH = 1 << 22
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


class ptored_layer_norm_params(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i64), ("weight", _vp), ("bias", _vp), ("eps", _f32),
                ("dtype", _i32), ("weight_dtype", _i32)]


class ptored_ffn_params(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i64), ("wide", _i64), ("dtype", _i32),
                ("activation", _i32)]


class ptored_ffn_grad_io(ctypes.Structure):
    _fields_ = [("dy", ptored_rows), ("gate", ptored_rows), ("up", ptored_rows),
                ("dgate", ptored_rows), ("dup", ptored_rows), ("x", ptored_rows),
                ("w_gate", ptored_rows), ("w_up", ptored_rows), ("dx", ptored_rows),
                ("dw_gate", ptored_rows), ("dw_up", ptored_rows), ("dw_dtype", _i32),
                ("accumulate", _i32), ("workspace", _vp), ("workspace_bytes", _i64)]


class ptored_grad(ctypes.Structure):
    _fields_ = [("data", _vp), ("out", _vp), ("rows", _i64), ("cols", _i64), ("ld", _i64),
                ("out_ld", _i64), ("dtype", _i32), ("out_dtype", _i32)]


_lib = None


def _load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = B.load()
        P = ctypes.POINTER
        lib.ptored_layer_norm.argtypes = [P(_vp), ctypes.c_int, _i64, P(ptored_layer_norm_params),
                                          ptored_rows, ptored_rows, ptored_rows, _vp, _vp, _vp]
        lib.ptored_layer_norm_backward.argtypes = [P(ptored_layer_norm_params), ptored_rows,
                                                   ptored_rows, ptored_rows, _vp, _vp, ptored_rows,
                                                   _vp, _vp, _vp, _i64, _vp]
        lib.ptored_layer_norm_backward_workspace.argtypes = [_i64, _i64, P(_i64)]
        lib.ptored_gated_ffn.argtypes = [P(ptored_ffn_params), *[ptored_rows] * 6, _vp, _i64, _vp]
        lib.ptored_gated_ffn_workspace.argtypes = [_i64, _i64, _i64, ctypes.c_int, P(_i64)]
        lib.ptored_gated_ffn_backward.argtypes = [P(ptored_ffn_params), P(ptored_ffn_grad_io), _vp]
        lib.ptored_gated_ffn_backward_workspace.argtypes = [_i64, _i64, _i64, ctypes.c_int, P(_i64)]
        lib.ptored_grad_norm.argtypes = [P(ptored_grad), _i64, _vp, _vp, _i64, _vp]
        lib.ptored_grad_scale.argtypes = [P(ptored_grad), _i64, _vp, _f32, _vp, _i64, _vp]
        lib.ptored_grad_clip.argtypes = [P(ptored_grad), _i64, _f32, _vp, _vp, _i64, _vp]
        lib.ptored_grad_norm_workspace.argtypes = [P(ptored_grad), _i64, P(_i64)]
        for name in ("ptored_layer_norm", "ptored_layer_norm_backward",
                     "ptored_layer_norm_backward_workspace", "ptored_gated_ffn",
                     "ptored_gated_ffn_workspace", "ptored_gated_ffn_backward", "ptored_gated_ffn_backward_workspace",
                     "ptored_grad_norm", "ptored_grad_scale", "ptored_grad_clip",
                     "ptored_grad_norm_workspace"):
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


# ---------------------------------------------------------------- raw calls

def ptored_layer_norm(parts, nranks: int, part_ld: int, params: ptored_layer_norm_params,
                      x: ptored_rows, x_out: ptored_rows, z: ptored_rows, mean, rstd,
                      stream: int) -> int:
    """Raw call: ``parts`` are device pointers as ints; returns the status code."""
    return _load().ptored_layer_norm(B._ptrs(parts), nranks, part_ld, params, x, x_out, z, mean,
                                     rstd, stream)


def ptored_layer_norm_backward(params, dz, dx_out, x_out, mean, rstd, dx, dweight, dbias, workspace,
                               workspace_bytes: int, stream: int) -> int:
    return _load().ptored_layer_norm_backward(params, dz, dx_out, x_out, mean, rstd, dx, dweight,
                                              dbias, workspace, workspace_bytes, stream)


def ptored_layer_norm_backward_workspace(rows: int, cols: int):
    out = _i64()
    st = _load().ptored_layer_norm_backward_workspace(rows, cols, out)
    return st, out.value


def ptored_gated_ffn(params: ptored_ffn_params, x, w_gate, w_up, y, gate, up, workspace,
                     workspace_bytes: int, stream: int) -> int:
    return _load().ptored_gated_ffn(params, x, w_gate, w_up, y, gate, up, workspace,
                                    workspace_bytes, stream)


def ptored_gated_ffn_workspace(rows: int, cols: int, wide: int, dtype: int):
    out = _i64()
    st = _load().ptored_gated_ffn_workspace(rows, cols, wide, dtype, out)
    return st, out.value


def ptored_gated_ffn_backward(params: ptored_ffn_params, io: ptored_ffn_grad_io, stream: int) -> int:
    return _load().ptored_gated_ffn_backward(params, io, stream)


def ptored_gated_ffn_backward_workspace(rows: int, cols: int, wide: int, dtype: int):
    out = _i64()
    st = _load().ptored_gated_ffn_backward_workspace(rows, cols, wide, dtype, out)
    return st, out.value


def ptored_grad_norm(grads, count: int, norm, workspace, workspace_bytes: int, stream: int) -> int:
    """Raw call: ``grads`` is an array of ``ptored_grad``."""
    return _load().ptored_grad_norm(grads, count, norm, workspace, workspace_bytes, stream)


def ptored_grad_scale(grads, count: int, norm, max_norm: float, workspace, workspace_bytes: int,
                      stream: int) -> int:
    return _load().ptored_grad_scale(grads, count, norm, max_norm, workspace, workspace_bytes, stream)


def ptored_grad_clip(grads, count: int, max_norm: float, norm, workspace, workspace_bytes: int,
                     stream: int) -> int:
    return _load().ptored_grad_clip(grads, count, max_norm, norm, workspace, workspace_bytes, stream)


def ptored_grad_norm_workspace(grads, count: int):
    out = _i64()
    st = _load().ptored_grad_norm_workspace(grads, count, out)
    return st, out.value


# ---------------------------------------------------------------- layer norm

_NO_ROWS = K._NO_ROWS


def _weight_code(g, *weights):
    """(torch type, code) that the weights share."""
    given = [w for w in weights if w is not None]
    wt = given[0].dtype if given else K._FLOAT32
    code = g.code if wt is g.dtype else K._float_code(wt, "weights")
    if code not in (0, g.code):
        raise TypeError("weights must be float32 or of the activations' type")
    return wt, code


def layer_norm(parts, x, x_out=None, z=None, *, weight=None, bias=None, eps: float = 1e-5,
               mean=None, rstd=None, stream=None) -> None:
    """The boundary of a block with layer norm, into the outputs that are given:

        x_out = x + parts[0] + ... + parts[N-1]
        mean  = mean_d(x_out),  rstd = 1/sqrt(mean_d((x_out - mean)^2) + eps)
        z     = (x_out - mean) rstd weight + bias

    ``parts`` (0 to 64 ranks' partial outputs; with none, layer norm alone),
    ``x``, ``x_out`` and ``z`` are [T, D] of one floating type; ``weight`` and
    ``bias`` [D], float32 or of that type, or None: ones and zeros.  ``mean`` and
    ``rstd`` (float32 [T]) are for the backward pass.  ``x_out`` and ``z`` may be
    ``x`` or a part itself.
    """
    if K._native_call("layer_norm", stream, parts, x, x_out, z, weight, bias, eps, mean, rstd):
        return
    g = K._Group(x, "x")
    ptrs, part_ld = [], g.cols
    for t in parts:
        part = g.mat(t, "every part" if ptrs else "parts[0]")
        if not ptrs:
            part_ld = part.ld
        elif part.ld != part_ld and g.rows > 1:  # a single row has no pitch
            raise ValueError("every part must have the same strides")
        ptrs.append(part.data)
    wt, code = _weight_code(g, weight, bias)
    params = ptored_layer_norm_params(g.rows, g.cols, g.vec(weight, g.cols, wt, "weight"),
                                      g.vec(bias, g.cols, wt, "bias"), eps, g.code, code)
    args = (g.mat(x, "x"), g.mat(x_out, "x_out"), g.mat(z, "z"),
            g.vec(mean, g.rows, K._FLOAT32, "mean"), g.vec(rstd, g.rows, K._FLOAT32, "rstd"))
    if g.rows == 0 or g.cols == 0:
        return  # empty tensors have no storage
    g.run(stream, ptored_layer_norm, ptrs, len(ptrs), part_ld, params, *args)
    K._wrote(x_out, z, mean, rstd)


def layer_norm_backward_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace of ``layer_norm_backward`` with weights' gradients."""
    st, n = ptored_layer_norm_backward_workspace(rows, cols)
    B._raise_on(st)
    return n


def layer_norm_backward(dz, dx_out, x_out, mean, rstd, dx=None, *, weight=None, dweight=None,
                        dbias=None, workspace=None, stream=None) -> None:
    """Gradients of ``layer_norm``, into the outputs that are given.

    ``dz`` is z's gradient, ``dx_out`` the one that reaches x_out past z (or
    None); ``x_out``, ``mean`` and ``rstd`` are what the forward pass left.
    ``dx`` is the gradient of x and of every rank's partial output; ``dweight``
    and ``dbias`` have the weight's type (without a weight, float32 or the
    activations').  ``dx`` may be any of the [T, D] inputs.
    """
    if K._native_call("layer_norm_backward", stream, dz, dx_out, x_out, mean, rstd, dx, weight,
                      dweight, dbias, workspace):
        return
    g = K._Group(dz, "dz")
    for t, what in ((x_out, "x_out"), (mean, "mean"), (rstd, "rstd")):
        if t is None:
            raise ValueError(f"layer_norm_backward needs {what}")
    wt, code = _weight_code(g, weight, dweight, dbias)
    params = ptored_layer_norm_params(g.rows, g.cols, g.vec(weight, g.cols, wt, "weight"), None, 0.0,
                                      g.code, code)
    args = [g.mat(dz, "dz"), g.mat(dx_out, "dx_out"), g.mat(x_out, "x_out"),
            g.vec(mean, g.rows, K._FLOAT32, "mean"), g.vec(rstd, g.rows, K._FLOAT32, "rstd"),
            g.mat(dx, "dx"), g.vec(dweight, g.cols, wt, "dweight"),
            g.vec(dbias, g.cols, wt, "dbias")]
    if g.cols == 0:
        return
    if g.rows == 0:  # nothing to read; the sums over no rows are zero
        K._zero((dweight, dbias), g.index, stream)
        return
    nbytes = 0
    if g.cols <= K.PTORED_BLOCK_MAX_COLS and not (dweight is None and dbias is None):
        nbytes = layer_norm_backward_workspace(g.rows, g.cols)
    keep, ptr, given = K._workspace(nbytes, workspace, g.index, stream)
    g.run(stream, ptored_layer_norm_backward, params, *args, ptr, given)
    K._wrote(dx, dweight, dbias)


# ---------------------------------------------------------------- feed-forward

def _activation_code(name) -> int:
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, not {name!r}")
    return code


def gated_ffn_workspace(rows: int, cols: int, wide: int, dtype) -> int:
    """Bytes of workspace of ``gated_ffn`` for x [rows, cols] and weights
    [wide, cols]."""
    st, n = ptored_gated_ffn_workspace(rows, cols, wide, B._dtype_code(dtype))
    B._raise_on(st)
    return n


def gated_ffn(x, w_gate, w_up, y, *, activation: str = "silu", gate=None, up=None, workspace=None,
              stream=None) -> None:
    """y = f(x w_gate^T) (x w_up^T): the column-parallel half of a gated
    feed-forward block.

    ``x`` is [T, D], ``w_gate`` and ``w_up`` [F, D] and ``y`` [T, F], of one
    floating type; f is "silu", "gelu" (by the error function) or "gelu_tanh".
    ``gate`` and ``up`` ([T, F], of that type; the halves of one [T, 2F] tensor, if
    wanted) are given the two projections, for the backward pass.  Sums are in
    float32 and f takes them unrounded.
    """
    code = _activation_code(activation)
    if K._native_call("gated_ffn", stream, x, w_gate, w_up, y, code, gate, up, workspace):
        return
    g = K._Group(x, "x")
    if y.dim() != 2:
        raise ValueError("y must be 2-D (rows x features)")
    wide = y.shape[1]
    mat = lambda t, rows, cols, what: (_NO_ROWS if t is None  # noqa: E731
                                       else g.other(t, what, rows, cols, g.dtype))
    params = ptored_ffn_params(g.rows, g.cols, wide, g.code, code)
    args = (g.mat(x, "x"), mat(w_gate, wide, g.cols, "w_gate"), mat(w_up, wide, g.cols, "w_up"),
            mat(y, g.rows, wide, "y"), mat(gate, g.rows, wide, "gate"), mat(up, g.rows, wide, "up"))
    if g.rows == 0 or wide == 0:
        return
    if g.cols == 0:  # sums over no columns
        K._zero((y, gate, up), g.index, stream)
        return
    st, nbytes = ptored_gated_ffn_workspace(g.rows, g.cols, wide, g.code)
    B._raise_on(st)
    keep, ptr, given = K._workspace(nbytes, workspace, g.index, stream)
    g.run(stream, ptored_gated_ffn, params, *args, ptr, given)
    K._wrote(y, gate, up)


def gated_ffn_backward_workspace(rows: int, cols: int, wide: int, dtype) -> int:
    """Bytes of workspace of ``gated_ffn_backward`` for x [rows, cols] and
    weights [wide, cols]."""
    st, n = ptored_gated_ffn_backward_workspace(rows, cols, wide, B._dtype_code(dtype))
    B._raise_on(st)
    return n


def gated_ffn_backward(dy, gate, up, dgate, dup, *, activation: str = "silu", x=None, w_gate=None,
                       w_up=None, dx=None, dw_gate=None, dw_up=None, accumulate: bool = False,
                       workspace=None, stream=None) -> None:
    """Gradients of ``gated_ffn``:

        dgate = dy up f'(gate),  dup = dy f(gate)
        dx = dgate w_gate + dup w_up,  dw_gate = dgate^T x,  dw_up = dup^T x

    ``gate`` and ``up`` are the projections that the forward pass kept; ``dgate``
    and ``dup`` their gradients, always written, and each may be ``dy``, ``gate``
    or ``up`` itself.  The products take them as rounded to their type.  ``dx``
    (needs ``w_gate`` and ``w_up``) is the input's gradient: this rank's share, as
    the weights are this rank's.  ``dw_gate`` and ``dw_up`` (need ``x``) are [F, D],
    float32 or of the activations' type; with ``accumulate`` they are added to.
    Where x was kept in 8 bits, ``checkpoint_wgrad`` takes ``dgate`` and ``dup``.
    """
    code = _activation_code(activation)
    if K._native_call("gated_ffn_backward", stream, dy, gate, up, dgate, dup, code, x, w_gate, w_up,
                      dx, dw_gate, dw_up, accumulate, workspace):
        return
    g = K._Group(dy, "dy")
    for t, what in ((gate, "gate"), (up, "up"), (dgate, "dgate"), (dup, "dup")):
        if t is None:
            raise ValueError(f"gated_ffn_backward needs {what}")
    if dx is not None and (w_gate is None or w_up is None):
        raise ValueError("dx needs w_gate and w_up")
    if (dw_gate is not None or dw_up is not None) and x is None:
        raise ValueError("dw_gate and dw_up need x")
    rows, wide = g.rows, g.cols
    known = next((t for t in (x, dx, w_gate, w_up) if t is not None), None)
    cols = 0
    if known is not None:
        if known.dim() != 2:
            raise ValueError("x, dx and the weights must be 2-D")
        cols = known.shape[1]
    mat = lambda t, r, c, what: (_NO_ROWS if t is None  # noqa: E731
                                 else g.other(t, what, r, c, g.dtype))
    dw = [t for t in (dw_gate, dw_up) if t is not None]
    dw_type = dw[0].dtype if dw else g.dtype
    dw_code = K._float_code(dw_type, "dw_gate" if dw_gate is not None else "dw_up") if dw else g.code
    if dw_code not in (0, g.code):
        raise TypeError("dw_gate and dw_up must be float32 or of dy's type")
    weight = lambda t, what: (_NO_ROWS if t is None  # noqa: E731
                              else g.other(t, what, wide, cols, dw_type))
    params = ptored_ffn_params(rows, cols, wide, g.code, code)
    io = ptored_ffn_grad_io(
        g.mat(dy, "dy"), g.mat(gate, "gate"), g.mat(up, "up"), g.mat(dgate, "dgate"),
        g.mat(dup, "dup"), mat(x, rows, cols, "x"), mat(w_gate, wide, cols, "w_gate"),
        mat(w_up, wide, cols, "w_up"), mat(dx, rows, cols, "dx"), weight(dw_gate, "dw_gate"),
        weight(dw_up, "dw_up"), dw_code, 1 if accumulate else 0, None, 0)
    if rows == 0 or wide == 0 or (known is not None and cols == 0):
        # empty tensors have no storage; sums over nothing are zero
        sums = [] if rows == 0 and accumulate else list(dw)
        if wide == 0 and dx is not None:
            sums.append(dx)
        K._zero([t for t in sums if t.numel()], g.index, stream)
        if rows == 0 or wide == 0:
            return
        for field in ("x", "w_gate", "w_up", "dx", "dw_gate", "dw_up"):
            setattr(io, field, _NO_ROWS)
    nbytes = 0
    if io.dx.data or io.dw_gate.data or io.dw_up.data:
        nbytes = gated_ffn_backward_workspace(rows, cols, wide, g.dtype)
    keep, io.workspace, io.workspace_bytes = K._workspace(nbytes, workspace, g.index, stream)
    g.run(stream, ptored_gated_ffn_backward, params, io)
    K._wrote(dgate, dup, dx, dw_gate, dw_up)


# ---------------------------------------------------------------- gradient clipping

def _runs(t):
    """(rows, cols, pitch) of a tensor whose elements lie in rows of one pitch,
    in the order of its indices."""
    dims = [(n, s) for n, s in zip(t.shape, t.stride()) if n != 1]
    if not dims:
        return 1, 1, 1
    merged = [dims[0]]
    for n, s in dims[1:]:
        m, before = merged[-1]
        if before == s * n:
            merged[-1] = (m * n, s)
        else:
            merged.append((n, s))
    if merged[-1][1] == 1 and len(merged) <= 2:
        cols = merged[-1][0]
        if len(merged) == 1:
            return 1, cols, cols
        if merged[0][1] >= cols:
            return merged[0][0], cols, merged[0][1]
    if len(merged) == 1 and merged[0][1] > 1:  # single elements, evenly spaced
        return merged[0][0], 1, merged[0][1]
    return None


def _dense(t) -> bool:
    """Whether the elements fill a range of memory, in whatever order."""
    size = 1
    for s, n in sorted((s, n) for n, s in zip(t.shape, t.stride()) if n != 1):
        if s != size:
            return False
        size *= n
    return True


class _Grads:
    """The gradients of a call as the C ABI takes them."""

    def __init__(self, grads, norm, outs):
        if K._torch is None:
            K._init()
        torch = K._torch
        if norm.dtype is not torch.float32 or norm.numel() != 1 or not norm.is_cuda:
            raise ValueError("norm must be one float32 element on a GPU")
        self.index = norm.get_device()
        grads = list(grads)
        self.outs = grads if outs is None else list(outs)
        if len(self.outs) != len(grads):
            raise ValueError("outs must have one tensor for each gradient")
        self.count = len(grads)
        self.table = (ptored_grad * max(1, self.count))()
        for i, (t, out) in enumerate(zip(grads, self.outs)):
            self._entry(self.table[i], t, out, i)

    def _entry(self, e, t, out, i):
        for v, what in ((t, f"gradient {i}"), (out, f"outs[{i}]")):
            if not isinstance(v, K._torch.Tensor):
                raise TypeError(f"{what} must be a tensor, not {type(v).__name__}")
            if v.layout is not K._torch.strided:
                raise TypeError(f"{what} must be dense")
            if v.get_device() != self.index or not v.is_cuda:
                raise ValueError(f"{what} must be on cuda:{self.index}")
        e.dtype = K._float_code(t.dtype, f"gradient {i}")
        e.out_dtype = K._float_code(out.dtype, f"outs[{i}]")
        if out.shape != t.shape or e.out_dtype not in (0, e.dtype):
            raise ValueError(f"outs[{i}] must have gradient {i}'s shape, and its type or float32")
        n = t.numel()
        e.rows, e.cols, e.ld, e.out_ld = (1, n, n, n)
        if n == 0:
            e.rows = 0
            return
        e.data, e.out = t.data_ptr(), out.data_ptr()
        # out has t's strides where it is t, or where both fill memory alike
        if t.stride() == out.stride() and _dense(t):
            return
        a, b = _runs(t), _runs(out)
        if a is None or b is None:
            raise ValueError(f"gradient {i} must lie in rows with unit stride")
        if a[:2] != b[:2]:
            # one of them in a single run takes the other's rows
            if a[0] == 1:
                a = (*b[:2], b[1])
            elif b[0] == 1:
                b = (*a[:2], a[1])
            else:
                raise ValueError(f"outs[{i}] must lie in gradient {i}'s rows")
        e.rows, e.cols, e.ld, e.out_ld = a[0], a[1], a[2], b[2]

    def workspace(self, given, stream):
        st, n = ptored_grad_norm_workspace(self.table, self.count)
        B._raise_on(st)
        return K._workspace(n, given, self.index, stream)

    def run(self, stream, call, *args):
        handle = B._stream_handle(stream, self.index)
        with K._torch.cuda.device(self.index):
            status = call(*args, handle)
        if status:
            B._raise_on(status)


def grad_norm(grads, norm, workspace=None, stream=None) -> None:
    """``norm`` (one float32 element) = the root of the sum of all squares over
    ``grads``, a sequence of tensors of any floating types and shapes.  Summed in
    binary64; a NaN or an infinity passes through; no gradients give 0.

    A gradient's elements fill a range of memory in any order, or lie in rows
    of unit stride and one pitch."""
    if K._native_call("grad_norm", stream, grads, norm, workspace):
        return
    g = _Grads(grads, norm, None)
    keep, ptr, nbytes = g.workspace(workspace, stream)
    g.run(stream, ptored_grad_norm, g.table, g.count, norm.data_ptr(), ptr, nbytes)
    K._wrote(norm)


def grad_scale(grads, norm, max_norm: float, outs=None, workspace=None, stream=None) -> None:
    """Scales every gradient by c = max_norm / norm where norm > max_norm, 1
    where it is not and NaN where it is NaN, into ``outs`` (of the gradients'
    shapes, each of its gradient's type or float32; default: in place).

    ``norm`` is read on the GPU when the kernels run: the gradients' norm, or
    that of all shards after an all-reduce."""
    if K._native_call("grad_scale", stream, grads, norm, max_norm, outs, workspace):
        return
    g = _Grads(grads, norm, outs)
    keep, ptr, nbytes = g.workspace(workspace, stream)
    g.run(stream, ptored_grad_scale, g.table, g.count, norm.data_ptr(), max_norm, ptr, nbytes)
    K._wrote(*g.outs)


def grad_clip(grads, max_norm: float, norm, outs=None, workspace=None, stream=None) -> None:
    """``grad_norm`` into ``norm`` and ``grad_scale`` by it, without the host
    waiting for it."""
    if K._native_call("grad_clip", stream, grads, max_norm, norm, outs, workspace):
        return
    g = _Grads(grads, norm, outs)
    keep, ptr, nbytes = g.workspace(workspace, stream)
    g.run(stream, ptored_grad_clip, g.table, g.count, max_norm, norm.data_ptr(), ptr, nbytes)
    K._wrote(norm, *g.outs)
