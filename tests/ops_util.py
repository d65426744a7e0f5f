"""Plain 64-bit forms of the operators around the selection, and the bounds
their results are held to.

Bounds, derived from the types alone:
  - A sum of q products in 32 bits, in any order, is off by at most
    (q + 2) * 2^-24 times the sum of the products' magnitudes (each step rounds
    by at most 2^-24 of a partial sum that is no larger than that).
  - A value rounded once to its type is off by at most finfo.eps / 2 of it,
    and, below the normal range, by half of the least subnormal.
  - gelu and silu have slopes of at most 1.13, and their 32-bit evaluation is
    off by at most 16 * 2^-24 (1 + |z|): a few roundings of factors no larger
    than 1 + |z|.
"""
from __future__ import annotations

import math

U32 = 2.0 ** -24


def _torch():
    import torch
    return torch


def half_step(dtype) -> float:
    return _torch().finfo(dtype).eps / 2


def round_err(ref, dtype):
    torch = _torch()
    return ref.abs() * half_step(dtype) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def act64(z, kind):
    torch = _torch()
    if kind == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if kind == "gelu":
        return torch.where(z == -math.inf, torch.zeros_like(z), 0.5 * z * torch.special.erfc(-z / math.sqrt(2)))
    if kind == "silu":
        return torch.where(z == -math.inf, torch.zeros_like(z), z * torch.sigmoid(z))
    return z


def slope64(z, kind):
    torch = _torch()
    if kind == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), torch.ones_like(z))
    if kind == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def linear64(x, w, b, kind, res):
    """(y, bound on |result - y|, z)"""
    torch = _torch()
    x, w = x.double(), w.double()
    z = x @ w.t().contiguous()
    mag = x.abs() @ w.abs().t().contiguous()
    if b is not None:
        z = z + b.double()
        mag = mag + b.double().abs()
    y = act64(z, kind)
    err = 1.13 * (x.shape[1] + 3) * U32 * mag
    if kind in ("gelu", "silu"):
        err = err + 16 * U32 * (1 + z.abs())
    if res is not None:
        y = y + res.double()
        err = err + U32 * y.abs()
    return y, err, z


def linear_grad64(dy, x, w, pre, kind):
    """((dx, dw, db), bounds before the last rounding).  The two products take
    dz rounded to the type (exact for none and relu)."""
    torch = _torch()
    dt = dy.dtype
    dy, x, w = dy.double(), x.double(), w.double()
    rounding = half_step(dt) + torch.finfo(dt).smallest_normal if kind in ("gelu", "silu") else 0.0
    if kind == "none":
        dz = dy
    elif kind == "relu":
        dz = torch.where(pre.double() <= 0, torch.zeros_like(dy), dy)
    else:
        dz = dy * slope64(pre.double(), kind)
    off = torch.zeros_like(dz)
    if kind in ("gelu", "silu"):
        off = 16 * U32 * (1 + pre.double().abs()) * dy.abs()
    m, n = dy.shape
    dzm = dz.abs()
    dx = dz @ w
    dw = dz.t().contiguous() @ x
    db = dz.sum(0)
    ex = ((n + 3) * U32 + rounding) * (dzm @ w.abs()) + off @ w.abs()
    ew = ((m + 3) * U32 + rounding) * (dzm.t().contiguous() @ x.abs()) + off.t().contiguous() @ x.abs()
    eb = (m + 3) * U32 * dzm.sum(0) + off.sum(0)
    return (dx, dw, db), (ex, ew, eb)


def within(got, ref, err, label=""):
    """|got - ref| <= err + one rounding of the result, element by element."""
    torch = _torch()
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    bound = err + round_err(ref.abs() + err, got.dtype)
    g = got.double()
    diff = (g - ref).abs()
    same = (g == ref) | (torch.isnan(g) & torch.isnan(ref))
    bad = ~(same | (diff <= bound))
    if bool(bad.any()):
        at = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} outside; first at {at}: "
                             f"{float(g[at])} for {float(ref[at])}, bound {float(bound[at])}")


def entries(indices, rows, n):
    """(entry numbers, rows, latents) of the entries in range, flat or row-wise."""
    torch = _torch()
    i = indices.cpu()
    if i.dim() == 2:
        ok = (i >= 0) & (i < n)
        r = torch.arange(rows)[:, None].expand_as(i)
        return ok.reshape(-1).nonzero()[:, 0], r[ok], i[ok]
    ok = (i >= 0) & (i < rows * n)
    i = i[ok]
    return ok.nonzero()[:, 0], torch.div(i, n, rounding_mode="floor"), i % n


def group64(coef, by, other, keys, src):
    """(sum over entries of coef * src[other] by key, its bound), in 64 bits on the CPU."""
    torch = _torch()
    s = src.cpu().double()
    c = coef.double()
    out = torch.zeros(keys, s.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    out.index_add_(0, by, c[:, None] * s[other])
    mag.index_add_(0, by, (c[:, None] * s[other]).abs())
    count = torch.bincount(by, minlength=keys).double()
    return out, (count[:, None] + 3) * U32 * mag
