"""The operators on a language model's selections: the next token, the experts
of a token and the way back, attention over a cache and the cache's eviction
(include/topk.h, "Operators on a language model's selections").

Argument checks and marshalling only; every step runs in the HIP library.
Scratch memory comes from torch's allocator for each call, so calls on
different streams, and captured graphs, never share any.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._ops import _CODES, _check, _code, _gpu, _matrix, _no_tangents, _on, _ptr, _scratch, _stream, _wants_grad

_byref = ctypes.byref
_STEP_MAX = 1 << 24    # entries of a cache that attend reads in place lie less than this many elements apart
_pack_dispatch = struct.Struct(_lib.DISPATCH_FORMAT).pack
_pack_combine = struct.Struct(_lib.COMBINE_FORMAT).pack
_pack_combine_grad = struct.Struct(_lib.COMBINE_GRAD_FORMAT).pack
_pack_attend = struct.Struct(_lib.ATTEND_FORMAT).pack
_pack_evict = struct.Struct(_lib.EVICT_FORMAT).pack
_pack_sample = struct.Struct(_lib.SAMPLE_FORMAT).pack


def _not_recorded(what: str, *tensors):
    """Operators without a gradient refuse tensors that want one: their results would be read as constants."""
    _no_tangents(*tensors)
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise RuntimeError(f"{what} has no gradient: call it under torch.no_grad, or with detached tensors")


_sizes: dict = {}    # workspace bytes by operator, device and what they depend on


def _run(name: str, args: bytes, like: torch.Tensor, dev: int, *key):
    """A call whose workspace is asked for with its own arguments, once for each
    ``key``: all of the arguments that its size depends on."""
    key = (name, dev, *key)
    size = _sizes.get(key)
    if size is None:
        out = ctypes.c_size_t()
        _lib.check(getattr(_lib.lib, f"topk_{name}_workspace_size")(args, _byref(out)), name)
        if len(_sizes) >= 4096:    # shapes that come once
            _sizes.clear()
        size = _sizes[key] = out.value
    ws = like.new_empty(size, dtype=torch.uint8) if size else None
    status = getattr(_lib.lib, "topk_" + name)(args, ws.data_ptr() if size else None, size, _stream(dev))
    if status:
        _lib.check(status, name)


# ---------------------------------------------------------------- tokens by expert
def _dispatch_run(x, experts, n_experts):
    t, d = x.shape
    k = experts.shape[1]
    dev = x.get_device()
    x, ldx, _ = _matrix(x)
    experts = experts.contiguous()
    with _on(dev):
        rows = x.new_empty((t * k, d))
        places = torch.empty_like(experts)
        offsets = experts.new_empty((n_experts + 1,))
        a = _pack_dispatch(x.data_ptr(), experts.data_ptr(), rows.data_ptr(), places.data_ptr(), offsets.data_ptr(),
                           t, k, n_experts, d, ldx, d or 1, _CODES[x.dtype], 0)
        # few entries need no scratch: ask only when the call says so
        if t * k > 4096 or _lib.lib.topk_dispatch(a, None, 0, _stream(dev)) != _lib.TOPK_OK:
            size = ctypes.c_size_t()
            _lib.check(_lib.lib.topk_dispatch_workspace_size(t, k, n_experts, _byref(size)), "dispatch")
            ws = _scratch(size.value, x)
            _lib.check(_lib.lib.topk_dispatch(a, _ptr(ws), size.value, _stream(dev)), "dispatch")
    return rows, places, offsets


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, experts, n_experts):
        rows, places, offsets = _dispatch_run(x, experts, n_experts)
        ctx.save_for_backward(places)
        ctx.mark_non_differentiable(places, offsets)
        return rows, places, offsets

    @staticmethod
    @once_differentiable
    def backward(ctx, grad, *_):
        _no_tangents(grad)
        return _combine_run(grad, ctx.saved_tensors[0], None), None, None


def dispatch(x: torch.Tensor, experts: torch.Tensor, n_experts: int) -> tuple:
    """Tokens sorted by expert: (rows, places, offsets).

    ``x`` [t, d] (float32 or bfloat16), ``experts`` [t, k] int64 as ``topk``
    returns the indices of a router's scores.  ``rows`` [t * k, d] holds a copy
    of a token's row for each of its experts, sorted by expert and, for one
    expert, in the order of (token, choice); expert i has the rows from
    ``offsets[i]`` to ``offsets[i + 1]`` (``offsets`` [n_experts + 1]).
    ``places`` [t, k] is where each copy lies, as ``combine`` takes it.  Entries
    out of range (the -1 of padded slots, or of copies dropped at a capacity)
    have the place -1; as many rows of zeros lie behind the last expert's.
    Differentiable (once) in x; its gradient is ``combine(grad, places)``, which
    is also how a captured step takes it."""
    _gpu(x, "x")
    _code(x, "x")
    if x.dim() != 2 or not isinstance(experts, torch.Tensor) or experts.dim() != 2:
        raise ValueError("x: [t, d]; experts: [t, k]")
    _check(experts, "experts", x, (x.shape[0], experts.shape[1]), torch.int64)
    n_experts = int(n_experts)
    if not 0 <= n_experts <= 8192:
        raise ValueError("n_experts: from 0 to 8192")
    if _wants_grad(x):
        return _Dispatch.apply(x, experts, n_experts)
    return _dispatch_run(x, experts, n_experts)


def _combine_run(y, places, weights):
    n, d = y.shape
    t, k = places.shape
    dev = y.get_device()
    y, ldy, _ = _matrix(y)
    places = places.contiguous()
    wcode = _CODES[y.dtype]
    if weights is not None:
        weights = weights.contiguous()
        wcode = _CODES[weights.dtype]
    with _on(dev):
        out = y.new_empty((t, d))
        a = _pack_combine(y.data_ptr(), places.data_ptr(), _ptr(weights), out.data_ptr(), t, k, n, d, ldy, d or 1,
                          _CODES[y.dtype], wcode)
        _lib.check(_lib.lib.topk_combine(a, _stream(dev)), "combine")
    return out


def _combine_grad_run(grad, y, places, weights, need):
    _no_tangents(grad, y, weights)
    n, d = y.shape
    t, k = places.shape
    dev = grad.get_device()
    grad, ldg, _ = _matrix(grad)
    y, ldy, _ = _matrix(y)
    places = places.contiguous()
    wcode = _CODES[y.dtype]
    if weights is not None:
        weights = weights.contiguous()
        wcode = _CODES[weights.dtype]
    with _on(dev):
        dy = y.new_empty((n, d)) if need[0] else None
        dw = torch.empty_like(weights) if need[1] else None
        if not ((dy is not None and dy.numel()) or (dw is not None and dw.numel())):
            return dy, dw
        a = _pack_combine_grad(grad.data_ptr(), y.data_ptr(), places.data_ptr(), _ptr(weights), _ptr(dy), _ptr(dw),
                               t, k, n, d, ldg, ldy, d or 1, _CODES[y.dtype], wcode)
        _run("combine_grad", a, grad, dev, t * k, n, d, need[0])
    return dy, dw


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, places, weights):
        ctx.save_for_backward(y, places, weights)
        return _combine_run(y, places, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        y, places, weights = ctx.saved_tensors
        ny, _, nw = ctx.needs_input_grad
        dy, dw = _combine_grad_run(grad, y, places, weights, (ny, nw))
        return dy, None, dw


def _check_combine(y, places, weights):
    _gpu(y, "y")
    _code(y, "y")
    if y.dim() != 2 or not isinstance(places, torch.Tensor) or places.dim() != 2:
        raise ValueError("y: [n, d]; places: [t, k]")
    _check(places, "places", y, dtype=torch.int64)
    if weights is not None:
        wide = isinstance(weights, torch.Tensor) and weights.dtype == torch.float32
        _check(weights, "weights", y, places.shape, torch.float32 if wide else None)


def combine(y: torch.Tensor, places: torch.Tensor, weights: torch.Tensor | None = None) -> torch.Tensor:
    """Rows back to their tokens: ``out[i] = sum over j of weights[i, j] * y[places[i, j]]``.

    ``y`` [n, d] (float32 or bfloat16), ``places`` [t, k] int64 as ``dispatch``
    returns them, ``weights`` [t, k] of y's type or float32 (None: all 1).
    Places out of range add nothing; one that occurs twice counts twice.  Sums
    are held in 32 bits.  Returns [t, d].  Differentiable (once) in y and
    weights; under graph capture with gradients off, and ``combine_grad``."""
    _check_combine(y, places, weights)
    if _wants_grad(y, weights):
        return _Combine.apply(y, places, weights)
    return _combine_run(y, places, weights)


def combine_grad(grad: torch.Tensor, y: torch.Tensor, places: torch.Tensor, weights: torch.Tensor | None = None,
                 need: tuple = (True, True)) -> tuple:
    """Gradients (dy, dweights) of ``combine`` from ``grad`` = dL/dout [t, d].
    Rows of y that no place names get 0, weights of places out of range too.
    Entries that name one row are added one after another (1.2 us each at 1024
    columns of bfloat16): dropped ones have the place -1, not one row for all.
    ``need``: which of the two to compute; None stands for the other, and for
    dweights where there are no weights."""
    _check_combine(y, places, weights)
    _check(grad, "grad", y, (places.shape[0], y.shape[1]))
    need = tuple(bool(b) for b in need)
    if len(need) != 2:
        raise ValueError("need: two truth values")
    need = (need[0], need[1] and weights is not None)
    if not any(need):
        return None, None
    with torch.no_grad():
        return _combine_grad_run(grad, y, places, weights, need)


# ---------------------------------------------------------------- attention over a cache
def _cache(t: torch.Tensor, what: str, like, shape=None) -> torch.Tensor:
    """[b, heads, n, d] with a contiguous last axis, by a copy where it is not."""
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError(f"{what}: [b, heads, n, d]")
    _check(t, what, like, shape)
    return t if t.stride(3) == 1 or t.shape[3] <= 1 else t.contiguous()


def _check_lengths(lengths, like, b):
    if lengths is None:
        return None
    _check(lengths, "lengths", like, (b,), torch.int64)
    return lengths.contiguous()


def _may_share(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two tensors with a contiguous last axis can have memory in common.
    Not if they lie apart; nor if they are interleaved, their rows beginning at
    multiples of one distance and not meeting within it (keys beside values)."""
    if not a.numel() or not b.numel():
        return False
    parts = []
    step = 0
    for t in (a, b):
        size = t.element_size()
        last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
        parts.append((t.data_ptr(), t.data_ptr() + (last + 1) * size, t.shape[-1] * size))
        for n, s in list(zip(t.shape, t.stride()))[:-1]:
            if n > 1:
                step = math.gcd(step, s * size)
    (a0, a1, wa), (b0, b1, wb) = parts
    if a1 <= b0 or b1 <= a0:
        return False
    if not step:
        return True
    return not (wa <= (b0 - a0) % step and wb <= (a0 - b0) % step)


def attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lengths: torch.Tensor | None = None,
           scores: torch.Tensor | None = None, scale: float | None = None) -> torch.Tensor:
    """Attention of one new token for each sequence over its cache.

    ``q`` [b, hq, d]; ``k``, ``v`` [b, h, n, d], hq a multiple of h (query head
    i reads head i // (hq / h)), d at most 256; float32 or bfloat16, all alike.
    Any strides but the last axis' (a [b, n, h, d] cache transposed is read in
    place).  ``lengths`` [b] int64: how many entries each sequence has (None:
    n); what lies behind them is not looked at.  ``scale``: d ** -0.5 if None.

    ``scores`` [b, h, n] float32, changed in place: each entry's probability,
    summed over the heads that share it, is added to it, as ``evict`` takes it.

    Returns [b, hq, d]; 0 for a sequence of length 0.  Softmax statistics and
    sums are held in 32 bits; in bfloat16 a probability's product with v is of
    two bfloat16 numbers, off by less than 2 ** -14 of it.  No gradient (tensors
    that want one are refused)."""
    _gpu(q, "q")
    _code(q, "q")
    if q.dim() != 3:
        raise ValueError("q: [b, hq, d]")
    b, hq, d = q.shape
    k = _cache(k, "k", q)
    _, h, n, _ = k.shape
    _check(k, "k", q, (b, h, n, d))
    v = _cache(v, "v", q, (b, h, n, d))
    k, v = (t if t.stride(2) < _STEP_MAX or n <= 1 else t.contiguous() for t in (k, v))
    if not 1 <= d <= 256 or h == 0 or hq % h or hq // h > 4096:
        raise ValueError(f"d: from 1 to 256; the heads of q a multiple of the cache's (up to 4096 times), not {hq} and {h}")
    lengths = _check_lengths(lengths, q, b)
    _not_recorded("attend", q, k, v, scores)
    sb = sh = 0
    if scores is not None:
        _check(scores, "scores", q, (b, h, n), torch.float32)
        if n > 1 and scores.stride(2) != 1:
            raise ValueError("scores: the last axis contiguous")
        sb, sh, _ = scores.stride()
    scale = d ** -0.5 if scale is None else ctypes.c_float(float(scale)).value
    if not math.isfinite(scale):
        raise ValueError("scale: a finite number")
    if q.stride(2) != 1 and d > 1:
        q = q.contiguous()
    dev = q.get_device()
    with _on(dev):
        out = q.new_empty((b, hq, d))
        a = _pack_attend(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(lengths), _ptr(scores), out.data_ptr(),
                         b, hq, h, n, d, *q.stride()[:2], *k.stride()[:3], *v.stride()[:3], sb, sh, hq * d, d,
                         scale, _CODES[q.dtype])
        _run("attend", a, q, dev, b, hq, h, n, d, q.dtype, scores is None)
        if scores is not None:
            torch.autograd.graph.increment_version(scores)   # changed in place, which autograd cannot see
    return out


def evict(k: torch.Tensor, v: torch.Tensor, scores: torch.Tensor, budget: int, recent: int = 0,
          lengths: torch.Tensor | None = None, out: tuple | None = None) -> tuple:
    """A cache cut to ``budget`` entries a head by accumulated attention weight:
    (k, v, scores, kept, lengths) of the entries that stay.

    ``k``, ``v`` [b, h, n, d] (float32 or bfloat16), ``scores`` [b, h, n]
    float32, as ``attend`` sums them; ``lengths`` [b] int64 (None: n).  Of a
    sequence with more than ``budget`` entries the ``recent`` last ones stay
    and, of the others, those with the largest scores (equal ones by lower
    index; NaN above all); a shorter one stays whole.  Entries keep their order.

    Returns new tensors of ``budget`` rows (k, v, scores; zeros behind a
    sequence's end), ``kept`` [b, h, budget] int64 (the old index of each row,
    -1 behind the end) and the new lengths [b].  ``out`` = (k, v, scores) takes
    the rows into tensors of at least ``budget`` rows instead, which may not
    share memory with the old cache; rows behind the end are left as they
    were.  No gradient (tensors that want one are refused)."""
    _gpu(k, "k")
    _code(k, "k")
    k = _cache(k, "k", k)
    b, h, n, d = k.shape
    v = _cache(v, "v", k, (b, h, n, d))
    _check(scores, "scores", k, (b, h, n), torch.float32)
    budget, recent = int(budget), int(recent)
    if budget < 1 or not 0 <= recent <= budget:
        raise ValueError("budget: at least 1; recent: from 0 to the budget")
    lengths = _check_lengths(lengths, k, b)
    _not_recorded("evict", k, v, scores)
    if n > 1 and scores.stride(2) != 1:
        scores = scores.contiguous()
    dev = k.get_device()
    with _on(dev):
        if out is None:
            ko, vo, so = k.new_empty((b, h, budget, d)), k.new_empty((b, h, budget, d)), scores.new_empty((b, h, budget))
        else:
            ko, vo, so = out
            for t, what in ((ko, "k"), (vo, "v"), (so, "scores")):
                if not isinstance(t, torch.Tensor) or t.dim() != (3 if what == "scores" else 4) or t.shape[2] < budget:
                    raise ValueError(f"out {what}: a tensor of at least {budget} rows")
                tail = () if what == "scores" else (d,)
                _check(t, "out " + what, k, (b, h, t.shape[2], *tail), torch.float32 if what == "scores" else None)
                last = t.stride(-1)
                if last != 1 and t.shape[-1] > 1:
                    raise ValueError(f"out {what}: the last axis contiguous")
            _not_recorded("evict", ko, vo, so)
            for i, t in enumerate((ko, vo, so)):
                if any(_may_share(t, o) for o in (k, v, scores, ko, vo)[:3 + min(i, 2)]):
                    raise ValueError("out: no memory shared with the old cache, or with one another")
        kept = torch.empty((b, h, budget), dtype=torch.int64, device=k.device)
        lengths_out = torch.empty((b,), dtype=torch.int64, device=k.device)
        if b and h:
            a = _pack_evict(k.data_ptr(), v.data_ptr(), scores.data_ptr(), _ptr(lengths), ko.data_ptr(), vo.data_ptr(),
                            so.data_ptr(), kept.data_ptr(), lengths_out.data_ptr(), b, h, n, d, budget, recent,
                            *k.stride()[:3], *v.stride()[:3], *scores.stride()[:2], *ko.stride()[:3], *vo.stride()[:3],
                            *so.stride()[:2], _CODES[k.dtype], 1 if out is None else 0)
            _lib.check(_lib.lib.topk_evict(a, None, 0, _stream(dev)), "evict")   # it takes no workspace
            if out is not None:
                torch.autograd.graph.increment_version((ko, vo, so))   # changed in place, which autograd cannot see
        elif b:   # no heads: only the lengths are left
            lengths_out.fill_(n) if lengths is None else lengths_out.copy_(lengths)
            lengths_out.clamp_(0, min(n, budget))
    return ko, vo, so, kept, lengths_out


# ---------------------------------------------------------------- the next token
def _setting(value, what, rows, like, lo, hi):
    """(number, tensor or None) of a setting of ``sample``."""
    if isinstance(value, torch.Tensor):
        _check(value, what, like, (rows,), torch.float32)
        return 0.0, value.contiguous()
    value = ctypes.c_float(float(value)).value   # as the library takes it
    if not lo <= value <= hi:
        raise ValueError(f"{what}: a number from {lo} to {hi}, or a float32 tensor of one for each row")
    return value, None


def sample(logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0) -> tuple:
    """The next token of each row, drawn by given random numbers: (tokens int64, logprobs float32).

    ``logits`` [rows, n] or [n] (float32 or bfloat16, n up to 2^24); ``u``
    [rows] float32, uniform in [0, 1).  With w_i = exp((z_i - max) /
    temperature) and the tokens in the order of their logits (the largest
    first, equal ones by lower index): the first ``top_k`` stay (0: all); of
    those the shortest beginning with ``top_p`` of their weight (1: all); of
    those the ones with w_i >= ``min_p``.  The token is the first, by index, at
    which the sum of what stayed exceeds u times its whole; logprobs are of
    that distribution.  A temperature of 0 takes the largest logit, with
    logprob 0.  Each setting is a number, or a tensor [rows] on the logits' GPU
    (int64 for top_k, float32 for the others; a temperature in it that is not
    above 0 counts as 0).

    A logit of -inf or NaN is never taken; a row of nothing else gives token -1
    and logprob -inf.  Sums are exact, so a row's token does not depend on the
    rows beside it.  No gradient (tensors that want one are refused)."""
    _gpu(logits, "logits")
    _code(logits, "logits")
    squeeze = logits.dim() == 1
    z = logits.unsqueeze(0) if squeeze else logits
    if z.dim() != 2 or z.shape[1] < 1:
        raise ValueError("logits: [rows, n] or [n], n at least 1")
    rows, n = z.shape
    _check(u, "u", z, dtype=torch.float32)
    if u.shape != (rows,) and not (squeeze and u.dim() == 0):
        raise ValueError(f"u: a float32 tensor of {rows} numbers")
    u = u.contiguous()
    temperature, ts = _setting(temperature, "temperature", rows, z, 0.0, math.inf)
    top_p, ps = _setting(top_p, "top_p", rows, z, 0.0, 1.0)
    min_p, ms = _setting(min_p, "min_p", rows, z, 0.0, 1.0)
    ks = None
    if isinstance(top_k, torch.Tensor):
        _check(top_k, "top_k", z, (rows,), torch.int64)
        top_k, ks = 0, top_k.contiguous()
    elif int(top_k) != top_k or top_k < 0:
        raise ValueError("top_k: a whole number from 0, or an int64 tensor of one for each row")
    _not_recorded("sample", logits, u, ts, ps, ms)
    z, ld, _ = _matrix(z)
    dev = z.get_device()
    with _on(dev):
        tokens = torch.empty((rows,), dtype=torch.int64, device=z.device)
        logprobs = torch.empty((rows,), dtype=torch.float32, device=z.device)
        a = _pack_sample(z.data_ptr(), u.data_ptr(), tokens.data_ptr(), logprobs.data_ptr(), _ptr(ts), _ptr(ks), _ptr(ps), _ptr(ms),
                         rows, n, ld, min(int(top_k), 1 << 62), temperature, top_p, min_p, _CODES[z.dtype])
        _run("sample", a, z, dev, rows, n, ts is None, ks is None, ps is None, temperature > 0, top_k, top_p < 1)
    return (tokens[0], logprobs[0]) if squeeze else (tokens, logprobs)
