"""The operators around the selection: the dense product with its epilogue,
the sparse decode, their gradients, and the clipping of a global norm
(include/topk.h, "Operators around the selection").

Argument checks and marshalling only; every step runs in the HIP library.
Scratch memory comes from torch's allocator for each call, so calls on
different streams, and captured graphs, never share any.
"""
from __future__ import annotations

import ctypes
import struct
from array import array
from contextlib import nullcontext
from operator import attrgetter

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _lib

_CODES = {torch.float32: 1, torch.bfloat16: 2}
_byref = ctypes.byref
_T = torch.Tensor
_pack_linear = struct.Struct(_lib.LINEAR_FORMAT).pack
_pack_selection = struct.Struct(_lib.SELECTION_FORMAT).pack
_dtype_of = attrgetter("dtype")


def _code(t: torch.Tensor, what: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: unsupported dtype {t.dtype}; use float32 or bfloat16")
    return code


def _check(t, what: str, like: torch.Tensor, shape=None, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: need a tensor")
    dtype = dtype or like.dtype
    if t.dtype != dtype or t.get_device() != like.get_device() or (shape is not None and t.shape != shape):
        raise ValueError(f"{what}: need a {dtype} tensor of shape {shape} on {like.device}, "
                         f"not {t.dtype} {tuple(t.shape)} on {t.device}")


def _gpu(t, what: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a GPU tensor")


_here = nullcontext()


def _on(index: int):
    """The library launches on the current device: switch when the tensors live elsewhere."""
    return _here if index == torch._C._cuda_getDevice() else torch.cuda.device(index)


# the current stream's handle on a device
_stream = torch._C._cuda_getCurrentRawStream


def _scratch(nbytes: int, like):
    return like.new_empty(nbytes, dtype=torch.uint8) if nbytes else None


def _ptr(t):
    return t.data_ptr() if t is not None else 0


_WIDTH_MAX = 1 << 22    # lines that a product reads in place are shorter
_STRIDE_MAX = 1 << 31


def _matrix(t: torch.Tensor, either: bool = False):
    """(tensor, row stride, stored transposed) of a 2-D tensor: rows with unit
    stride as they are; columns with unit stride too where the call takes
    ``either`` order; any other layout (expanded, stepped, lines that are too
    long or too far apart for the library) as a copy."""
    r, c = t.shape
    if t.is_contiguous():
        return t, c or 1, 0
    sr, sc = t.stride()
    if (sc == 1 or c <= 1) and (c <= sr < _STRIDE_MAX or r <= 1):
        return t, max(sr if r > 1 else c, c, 1), 0
    if either and (sr == 1 or r <= 1) and (r <= sc < _STRIDE_MAX or c <= 1) and r < _WIDTH_MAX:
        return t, max(sc if c > 1 else r, r, 1), 1
    return t.contiguous(), max(c, 1), 0


def _empty(*outs) -> bool:
    """Whether no wanted output has an element (the library takes an empty output, a null address, for not wanted)."""
    return not any(t is not None and t.numel() for t in outs)


def _act_code(activation: str) -> int:
    code = _lib.ACTIVATIONS.get(activation)
    if code is None:
        raise ValueError(f"activation: one of {', '.join(_lib.ACTIVATIONS)}, not {activation!r}")
    return code


def _no_tangents(*tensors):
    """Forward-mode derivatives do not pass through the library: a result without
    a tangent would be read as one of zero."""
    if forward_ad._current_level >= 0 and torch._C._is_fwd_grad_enabled():
        for t in tensors:
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                raise RuntimeError("forward-mode derivatives are not supported: take the tangent off "
                                   "(torch.autograd.forward_ad.unpack_dual) or use backward derivatives")


def _wants_grad(*tensors) -> bool:
    """Whether autograd records the call.  Not under graph capture: a captured
    backward meets the gradient accumulators of whatever eager graph of the
    same leaves is alive, on streams that are not captured, and that ends the
    process; the *_grad functions take no part in autograd and can be captured.
    Refuses tensors that carry a tangent."""
    _no_tangents(*tensors)
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("autograd cannot record this call under graph capture: call it with "
                                       "gradients off (torch.no_grad) and its *_grad function")
                return True
    return False


# ---------------------------------------------------------------- linear
def _linear_run(x, w, bias, act, residual, want_pre):
    m, k = x.shape
    n = w.shape[0]
    dev = x.get_device()
    x, ldx, xt = _matrix(x, True)
    w, ldw, wt = _matrix(w, True)
    ldr = 0
    if residual is not None:
        residual, ldr, _ = _matrix(residual)
    if bias is not None:
        bias = bias.contiguous()
    with _on(dev):
        y = x.new_empty((m, n))
        pre = x.new_empty((m, n)) if want_pre else None
        a = _pack_linear(x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(residual), y.data_ptr(), _ptr(pre),
                         m, n, k, ldx, ldw, ldr, n, n, _CODES[x.dtype], act, xt, wt)
        stream = _stream(dev)
        # few rows need no scratch: ask only when the call says so
        if m > 32 or _lib.lib.topk_linear(a, None, 0, stream) != _lib.TOPK_OK:
            size = ctypes.c_size_t()
            _lib.check(_lib.lib.topk_linear_workspace_size(a, _byref(size)), "linear")
            ws = _scratch(size.value, x)
            _lib.check(_lib.lib.topk_linear(a, _ptr(ws), size.value, stream), "linear")
    return y, pre


def _linear_grad_run(dy, x, w, act, pre, need):
    _no_tangents(dy, x, w, pre)
    m, n = dy.shape
    k = w.shape[1]
    dev = dy.get_device()
    dy, ldd, _ = _matrix(dy)
    x, ldx, xt = _matrix(x, True)
    w, ldw, wt = _matrix(w, True)
    ldp = 0
    if pre is not None:
        pre, ldp, _ = _matrix(pre)
    with _on(dev):
        dx = dy.new_empty((m, k)) if need[0] else None
        dw = dy.new_empty((n, k)) if need[1] else None
        db = dy.new_empty((n,)) if need[2] else None
        if _empty(dx, dw, db):
            return dx, dw, db
        a = _lib.LinearGradArgs(dy.data_ptr(), _ptr(pre), x.data_ptr(), w.data_ptr(), _ptr(dx), _ptr(dw),
                                _ptr(db), m, n, k, ldd, ldp, ldx, ldw, k, k, _CODES[dy.dtype], act, xt, wt)
        size = ctypes.c_size_t()
        _lib.check(_lib.lib.topk_linear_grad_workspace_size(_byref(a), _byref(size)), "linear_grad")
        ws = _scratch(size.value, dy)
        _lib.check(_lib.lib.topk_linear_grad(_byref(a), _ptr(ws), size.value, _stream(dev)),
                   "linear_grad")
    return dx, dw, db


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, residual, act):
        # relu's slope is read from y, unless the residual hides it; gelu and
        # silu need the pre-activation
        keep = act > 1 or (act == 1 and residual is not None)
        y, pre = _linear_run(x, w, bias, act, residual, keep)
        ctx.act, ctx.bias, ctx.residual = act, bias is not None, residual is not None
        ctx.save_for_backward(x, w, pre if keep else y if act else None)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, pre = ctx.saved_tensors
        nx, nw, nb, nr, _ = ctx.needs_input_grad
        dx = dw = db = None
        if nx or nw or nb:
            dx, dw, db = _linear_grad_run(dy, x, w, ctx.act, pre, (nx, nw, nb))
        return dx, dw, db, dy if nr else None, None


def linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
           activation: str = "none", residual: torch.Tensor | None = None) -> torch.Tensor:
    """``act(x @ weight.T + bias) + residual`` in one pass.

    ``x`` [..., k], ``weight`` [n, k] (as torch.nn.Linear keeps it; the
    transpose of a [k, n] tensor is read in place), ``bias`` [n], ``residual``
    [..., n]; float32 or bfloat16, all alike.  ``activation``: "none", "relu",
    "gelu" (z * Phi(z)) or "silu".  Sums and the epilogue are held in 32 bits.
    Differentiable (once, backward; tensors with a forward-mode tangent are
    refused).  Under HIP graph capture autograd is refused: call ``linear`` with
    gradients off, and ``linear_grad``."""
    _gpu(x, "x")
    _code(x, "x")
    act = _act_code(activation)
    if x.dim() < 1 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("x: [..., k]; weight: [n, k]")
    n, k = weight.shape
    lead = x.shape[:-1]
    _check(weight, "weight", x)
    if x.shape[-1] != k:
        raise ValueError(f"x has {x.shape[-1]} columns, weight {k}")
    if bias is not None:
        _check(bias, "bias", x, (n,))
    if residual is not None:
        _check(residual, "residual", x, (*lead, n))
    flat = x.dim() == 2
    x2 = x if flat else x.reshape(lead.numel(), k)
    r2 = residual if flat or residual is None else residual.reshape(lead.numel(), n)
    if _wants_grad(x, weight, bias, residual):
        y = _Linear.apply(x2, weight, bias, r2, act)
    else:
        y = _linear_run(x2, weight, bias, act, r2, False)[0]
    return y if flat else y.reshape(*lead, n)


def linear_grad(grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, activation: str = "none",
                pre: torch.Tensor | None = None, need: tuple = (True, True, True)) -> tuple:
    """Gradients (dx, dweight, dbias) of ``linear`` from ``grad`` = dL/dy.

    ``grad`` [m, n], ``x`` [m, k], ``weight`` [n, k]; ``pre`` [m, n]: the
    pre-activation ``linear(x, weight, bias)``, or for relu without a residual
    the output (needed unless the activation is "none").  The residual's
    gradient is ``grad``.  ``need``: which of the three to compute; None stands
    for the others."""
    _gpu(grad, "grad")
    _code(grad, "grad")
    act = _act_code(activation)
    if grad.dim() != 2 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("grad: [m, n]; x: [m, k]; weight: [n, k]")
    m, n = grad.shape
    k = weight.shape[1]
    _check(weight, "weight", grad, (n, k))
    _check(x, "x", grad, (m, k))
    if act:
        if pre is None:
            raise ValueError("pre: the pre-activation is needed")
        _check(pre, "pre", grad, (m, n))
    else:
        pre = None
    need = tuple(bool(b) for b in need)
    if len(need) != 3:
        raise ValueError("need: three truth values")
    if not any(need):
        return None, None, None
    with torch.no_grad():
        return _linear_grad_run(grad, x, weight, act, pre, need)


# ---------------------------------------------------------------- decode
def _selection(values, indices, rows, n):
    """The selection's struct: [rows, k] values hold latents, 1-D ones flattened places."""
    if values.dim() == 2:
        return _pack_selection(values.data_ptr(), indices.data_ptr(), values.shape[0], values.shape[1], n, 0,
                               _CODES[values.dtype])
    return _pack_selection(values.data_ptr(), indices.data_ptr(), rows, values.shape[0], n, 1,
                           _CODES[values.dtype])


def _decode_scratch(sel, d, like):
    size = ctypes.c_size_t()
    _lib.check(_lib.lib.topk_decode_workspace_size(sel, d, _byref(size)), "decode")
    return _scratch(size.value, like), size.value


def _decode_run(values, indices, weight, rows, bias):
    n, d = weight.shape
    dev = values.get_device()
    values, indices = values.contiguous(), indices.contiguous()
    weight, ldw, _ = _matrix(weight)
    if bias is not None:
        bias = bias.contiguous()
    with _on(dev):
        out = values.new_empty((rows, d))
        sel = _selection(values, indices, rows, n)
        stream = _stream(dev)
        args = (sel, weight.data_ptr(), ldw, d, _ptr(bias), out.data_ptr(), d or 1)
        # row-wise selections seldom need scratch: ask only when the call says so
        if values.dim() != 2 or _lib.lib.topk_decode(*args, None, 0, stream) != _lib.TOPK_OK:
            ws, size = _decode_scratch(sel, d, values)
            _lib.check(_lib.lib.topk_decode(*args, _ptr(ws), size, stream), "decode")
    return out


def _decode_grad_run(grad, values, indices, weight, need):
    _no_tangents(grad, values, weight)
    n, d = weight.shape
    rows = grad.shape[0]
    dev = grad.get_device()
    values, indices = values.contiguous(), indices.contiguous()
    weight, ldw, _ = _matrix(weight)
    grad, ldg, _ = _matrix(grad)
    with _on(dev):
        dv = torch.empty_like(values) if need[0] else None
        dw = grad.new_empty((n, d)) if need[1] else None
        db = grad.new_empty((d,)) if need[2] else None
        if _empty(dv, dw, db):
            return dv, dw, db
        sel = _selection(values, indices, rows, n)
        ws, size = _decode_scratch(sel, d, values)
        _lib.check(_lib.lib.topk_decode_grad(sel, weight.data_ptr(), ldw, d, grad.data_ptr(), ldg,
                                             _ptr(dv), _ptr(dw), max(d, 1), _ptr(db), _ptr(ws), size,
                                             _stream(dev)), "decode_grad")
    return dv, dw, db


class _Decode(torch.autograd.Function):
    @staticmethod
    def forward(ctx, values, indices, weight, rows, bias):
        ctx.save_for_backward(values, indices, weight)
        return _decode_run(values, indices, weight, rows, bias)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        values, indices, weight = ctx.saved_tensors
        nv, _, nw, _, nb = ctx.needs_input_grad
        dv, dw, db = _decode_grad_run(grad, values, indices, weight, (nv, nw, nb))
        return dv, None, dw, None, db


def _check_selection(values, indices, rows):
    _gpu(values, "values")
    _code(values, "values")
    if values.dim() not in (1, 2):
        raise ValueError("values, indices: [rows, k], or [k] of a flattened selection")
    _check(indices, "indices", values, values.shape, torch.int64)
    if values.dim() == 2:
        if rows is not None and rows != values.shape[0]:
            raise ValueError(f"rows is {rows}, values has {values.shape[0]}")
        return values.shape[0]
    if rows is None or rows < 0:
        raise ValueError("rows: needed for a flattened selection")
    return int(rows)


def decode(values: torch.Tensor, indices: torch.Tensor, weight: torch.Tensor, rows: int | None = None,
           bias: torch.Tensor | None = None) -> torch.Tensor:
    """Sparse decode of a selection: ``out[r] = bias + sum of v_e * weight[latent_e]``
    over the selected entries e of row r, without the dense activation.

    ``values``, ``indices`` as ``topk`` returns them: [rows, k] with latents in
    [0, n), or [k] of a flattened [rows, n] selection (then ``rows`` is
    needed; an index is row * n + latent).  ``weight`` [n, d], ``bias`` [d].
    Entries out of range (the -1 of padded slots) add nothing; an index that
    occurs twice counts twice.  Returns [rows, d].  Differentiable (once) in
    values, weight and bias; under graph capture with gradients off, and
    ``decode_grad``."""
    rows = _check_selection(values, indices, rows)
    _check(weight, "weight", values)
    if weight.dim() != 2:
        raise ValueError("weight: [n, d]")
    if bias is not None:
        _check(bias, "bias", values, (weight.shape[1],))
    if _wants_grad(values, weight, bias):
        return _Decode.apply(values, indices, weight, rows, bias)
    return _decode_run(values, indices, weight, rows, bias)


def decode_grad(grad: torch.Tensor, values: torch.Tensor, indices: torch.Tensor, weight: torch.Tensor,
                need: tuple = (True, True, True)) -> tuple:
    """Gradients (dvalues, dweight, dbias) of ``decode`` from ``grad`` = dL/dout
    [rows, d].  Entries out of range get a gradient of 0.  ``need``: which of
    the three to compute; None stands for the others."""
    _gpu(grad, "grad")
    if grad.dim() != 2 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("grad: [rows, d]; weight: [n, d]")
    rows = _check_selection(values, indices, grad.shape[0])
    _check(weight, "weight", values)
    _check(grad, "grad", values, (rows, weight.shape[1]))
    need = tuple(bool(b) for b in need)
    if len(need) != 3:
        raise ValueError("need: three truth values")
    if not any(need):
        return None, None, None
    with torch.no_grad():
        return _decode_grad_run(grad, values, indices, weight, need)


# ---------------------------------------------------------------- encode
def _encode_grad_run(grad_values, values, indices, x, weight, need):
    _no_tangents(grad_values, values, x, weight)
    n, d = weight.shape
    rows = x.shape[0]
    dev = x.get_device()
    grad_values, values, indices = grad_values.contiguous(), values.contiguous(), indices.contiguous()
    weight, ldw, _ = _matrix(weight)
    x, ldx, _ = _matrix(x)
    with _on(dev):
        dx = x.new_empty((rows, d)) if need[0] else None
        dw = x.new_empty((n, d)) if need[1] else None
        db = x.new_empty((n,)) if need[2] else None
        if _empty(dx, dw, db):
            return dx, dw, db
        sel = _selection(values, indices, rows, n)
        ws, size = _decode_scratch(sel, d, values)
        _lib.check(_lib.lib.topk_encode_grad(sel, grad_values.data_ptr(), x.data_ptr(), ldx,
                                             weight.data_ptr(), ldw, d, _ptr(dx), max(d, 1), _ptr(dw),
                                             max(d, 1), _ptr(db), _ptr(ws), size, _stream(dev)),
                   "encode_grad")
    return dx, dw, db


class _Encode(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, k_total, params, workspace):
        values, indices = _encode_run(x, weight, bias, k_total, params, workspace)
        ctx.save_for_backward(x, weight, values, indices)
        ctx.mark_non_differentiable(indices)
        return values, indices

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_values, _):
        x, weight, values, indices = ctx.saved_tensors
        nx, nw, nb = ctx.needs_input_grad[:3]
        dx, dw, db = _encode_grad_run(grad_values, values, indices, x, weight, (nx, nw, nb))
        return dx, dw, db, None, None, None


def _encode_run(x, weight, bias, k_total, params, workspace):
    from . import topk
    acts = _linear_run(x, weight, bias, _lib.ACTIVATIONS["relu"], None, False)[0]
    values, indices = topk(acts.reshape(1, -1), k_total, params=params, workspace=workspace)
    return values[0], indices[0]


def encode(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None, k_total: int,
           params=None, workspace=None) -> tuple:
    """The encoder of a BatchTopK sparse autoencoder (Prof-K section 5): the
    ``k_total`` largest entries of ``relu(x @ weight.T + bias)`` over the whole
    batch, as (values [k_total], flattened indices [k_total]) in rank order.

    ``x`` [rows, d], ``weight`` [n, d], ``bias`` [n]; float32 or bfloat16.
    Differentiable (once) in x, weight and bias through the selected entries
    above 0 (the others have no gradient); the backward touches those entries
    only.  Under graph capture with gradients off, and ``encode_grad``.
    ``params``, ``workspace``: as ``topk``'s (a captured call needs a workspace
    of its own)."""
    _gpu(x, "x")
    _code(x, "x")
    if x.dim() != 2 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("x: [rows, d]; weight: [n, d]")
    _check(weight, "weight", x)
    if weight.shape[1] != x.shape[1]:
        raise ValueError(f"x has {x.shape[1]} columns, weight {weight.shape[1]}")
    if bias is not None:
        _check(bias, "bias", x, (weight.shape[0],))
    if not 1 <= k_total <= x.shape[0] * weight.shape[0]:
        raise ValueError("k_total: from 1 to rows * n")
    if _wants_grad(x, weight, bias):
        return _Encode.apply(x, weight, bias, k_total, params, workspace)
    return _encode_run(x, weight, bias, k_total, params, workspace)


def encode_grad(grad_values: torch.Tensor, values: torch.Tensor, indices: torch.Tensor,
                x: torch.Tensor, weight: torch.Tensor, need: tuple = (True, True, True)) -> tuple:
    """Gradients (dx, dweight, dbias) of ``encode`` from ``grad_values`` =
    dL/dvalues: with c_e = grad_values[e] where values[e] > 0 and 0 elsewhere,
    ``dx[r] = sum of c_e * weight[latent_e]``, ``dweight[j] = sum of c_e * x[row_e]``,
    ``dbias[j] = sum of c_e``.  A selection of [rows, k] (row-wise) is taken
    as well.  ``need``: which of the three to compute; None stands for the others."""
    _gpu(x, "x")
    if x.dim() != 2 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("x: [rows, d]; weight: [n, d]")
    rows = _check_selection(values, indices, x.shape[0])
    _check(grad_values, "grad_values", values, values.shape)
    _check(weight, "weight", values, (weight.shape[0], x.shape[1]))
    _check(x, "x", values, (rows, weight.shape[1]))
    need = tuple(bool(b) for b in need)
    if len(need) != 3:
        raise ValueError("need: three truth values")
    if not any(need):
        return None, None, None
    with torch.no_grad():
        return _encode_grad_run(grad_values, values, indices, x, weight, need)


# ---------------------------------------------------------------- gradient norm
def _dense(t: torch.Tensor) -> bool:
    """Whether the elements fill one block of memory without gaps or overlap, in any order of the axes."""
    if t.is_contiguous():
        return True
    at = 1
    for stride, size in sorted((st, sz) for st, sz in zip(t.stride(), t.shape) if sz != 1):
        if stride != at:
            return False
        at *= size
    return True


def _norm_run(tensors, clip):
    if isinstance(tensors, torch.Tensor):
        tensors = [tensors]
    ts = list(tensors)
    try:
        devices = set(map(_T.get_device, ts))
    except TypeError:   # something that is no tensor: None is skipped
        ts = [t for t in ts if t is not None]
        devices = set(map(_T.get_device, ts))
    _no_tangents(*ts)
    if not ts:
        return torch.zeros((), device="cuda")
    index = devices.pop()
    if index < 0 or devices:
        raise ValueError(f"tensors: all on one GPU (found {', '.join(sorted({str(t.device) for t in ts}))})")
    dtypes = list(map(_dtype_of, ts))
    kinds = set(dtypes)
    for dtype in kinds:
        if dtype not in _CODES:
            raise TypeError(f"tensors: unsupported dtype {dtype}; use float32 or bfloat16")
    if not all(map(_T.is_contiguous, ts)) and not all(map(_dense, ts)):
        raise ValueError("tensors: need dense memory (no gaps, no expanded axes)")
    # flat host arrays, passed by address; they live until the call has read them
    ptrs = array("Q", map(_T.data_ptr, ts))
    counts = array("q", map(_T.numel, ts))
    codes = (array("i", map(_CODES.__getitem__, dtypes)) if len(kinds) > 1
             else array("i", [_CODES[dtypes[0]]]) * len(ts))
    args = (ptrs.buffer_info()[0], counts.buffer_info()[0], codes.buffer_info()[0], len(ts))
    with _on(index):
        norm = ts[0].new_empty((), dtype=torch.float32)
        size = ctypes.c_size_t()
        _lib.check(_lib.lib.topk_grad_norm_workspace_size(args[3], args[1], _byref(size)), "grad_norm")
        ws = _scratch(size.value, norm)
        if clip is None:
            _lib.check(_lib.lib.topk_grad_norm(*args, norm.data_ptr(), _ptr(ws), size.value, _stream(index)),
                       "grad_norm")
        else:
            _lib.check(_lib.lib.topk_clip_grad_norm(*args, *clip, norm.data_ptr(), _ptr(ws), size.value,
                                                    _stream(index)), "clip_grad_norm")
            torch.autograd.graph.increment_version(ts)   # changed in place, which autograd cannot see
    return norm


def grad_norm(tensors) -> torch.Tensor:
    """The 2-norm of all elements of ``tensors`` (one tensor or several, dense,
    float32 and bfloat16 mixed, None skipped), as a float32 scalar on their GPU."""
    return _norm_run(tensors, None)


def clip_grad_norm(tensors, max_norm: float, eps: float = 1e-6) -> torch.Tensor:
    """Scale ``tensors`` in place by min(1, max_norm / (norm + eps)), ``norm`` their
    global 2-norm, which is returned as a float32 scalar on the GPU (no
    synchronisation).  Tensors as in ``grad_norm``, none overlapping another
    (TopkError).  A norm of inf or NaN scales by 0 or NaN: read the norm to tell."""
    return _norm_run(tensors, (float(max_norm), float(eps)))
