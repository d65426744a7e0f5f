"""Plain 64-bit forms of the operators on a language model's selections, on the
CPU, and the bounds their results are held to.

Bounds, derived from the types alone (U32 = 2^-24, half a step of float32):
  - combine, combine_grad: sums of q products in 32 bits, as in ops_util.
  - attend: a logit is a sum of d products, scaled once: off by at most
    e = (d + 4) U32 scale sum |q k|.  The exponent's difference to the maximum,
    its rounding and the hardware's exponential add (|s - m| + 4) U32 * 2 to a
    probability's relative error, the sum of n of them (n + 8) U32 (any order,
    with the factors of its parts).  So p is off by at most
      r = 2 max e + 2 (max |s - m| + 4) U32 + (n + 8) U32
    of itself (for r far below 1; 1.1 r holds its square).  The output adds a
    sum of n products, and in bfloat16 the rounding of p.
  - what is only moved or chosen is equal.
"""
from __future__ import annotations

import math

import ops_util as U

U32 = U.U32


def _torch():
    import torch
    return torch


# ---------------------------------------------------------------- tokens by expert
def places64(experts, count):
    """(order of the entries, places, offsets), by counting."""
    torch = _torch()
    e = experts.reshape(-1).tolist()
    bins = [[] for _ in range(count + 1)]
    for i, x in enumerate(e):
        bins[x if 0 <= x < count else count].append(i)
    order = [i for b in bins for i in b]
    place = [-1] * len(e)
    at = 0
    offsets = [0]
    for b in bins[:count]:
        for i in b:
            place[i] = at
            at += 1
        offsets.append(at)
    return (torch.tensor(order, dtype=torch.int64), torch.tensor(place, dtype=torch.int64).reshape(experts.shape),
            torch.tensor(offsets, dtype=torch.int64))


def dispatch64(x, experts, count):
    torch = _torch()
    x, experts = x.cpu(), experts.cpu()
    order, place, offsets = places64(experts, count)
    k = max(experts.shape[1], 1)
    rows = x[torch.div(order, k, rounding_mode="floor")].clone()
    rows[int(offsets[-1]):] = 0
    return rows, place, offsets


def combine64(y, places, weights):
    """(out, bound)"""
    torch = _torch()
    y, places = y.cpu().double(), places.cpu()
    n = y.shape[0]
    good = (places >= 0) & (places < n)
    w = torch.ones(places.shape, dtype=torch.float64) if weights is None else weights.cpu().double()
    rows = torch.zeros(*places.shape, y.shape[1], dtype=torch.float64)
    rows[good] = y[places[good]] * w[good][:, None]
    return rows.sum(1), (places.shape[1] + 2) * U32 * rows.abs().sum(1)


def combine_grad64(grad, y, places, weights):
    """((dy, dw), bounds)"""
    torch = _torch()
    grad, y, places = grad.cpu().double(), y.cpu().double(), places.cpu()
    n, d = y.shape
    good = (places >= 0) & (places < n)
    w = torch.ones(places.shape, dtype=torch.float64) if weights is None else weights.cpu().double()
    t = torch.arange(places.shape[0])[:, None].expand_as(places)
    dy, mag = torch.zeros(n, d, dtype=torch.float64), torch.zeros(n, d, dtype=torch.float64)
    part = w[good][:, None] * grad[t[good]]
    dy.index_add_(0, places[good], part)
    mag.index_add_(0, places[good], part.abs())
    count = torch.bincount(places[good], minlength=n).double() if n else torch.zeros(0, dtype=torch.float64)
    dw, ew = torch.zeros(places.shape, dtype=torch.float64), torch.zeros(places.shape, dtype=torch.float64)
    prod = grad[t[good]] * y[places[good]]
    dw[good] = prod.sum(1)
    ew[good] = (d + 3) * U32 * prod.abs().sum(1)
    return (dy, dw), ((count[:, None] + 2) * U32 * mag, ew)


# ---------------------------------------------------------------- a cache
def attend64(q, k, v, lengths, scale, dtype):
    """(out, its bound, added scores, their bound)"""
    torch = _torch()
    q, k, v = q.cpu().double(), k.cpu().double(), v.cpu().double()
    b, hq, d = q.shape
    _, h, n, _ = k.shape
    scale = d ** -0.5 if scale is None else scale
    out, eo = torch.zeros(b, hq, d, dtype=torch.float64), torch.zeros(b, hq, d, dtype=torch.float64)
    add, ea = torch.zeros(b, h, n, dtype=torch.float64), torch.zeros(b, h, n, dtype=torch.float64)
    for i in range(b):
        e = n if lengths is None else max(0, min(n, int(lengths[i])))
        if e == 0:
            continue
        for x in range(hq):
            j = x // (hq // h)
            kk, vv = k[i, j, :e], v[i, j, :e]
            s = kk @ q[i, x] * scale
            off = float(((d + 4) * U32 * abs(scale) * (kk.abs() @ q[i, x].abs())).max())
            p = torch.softmax(s, 0)
            r = 1.1 * (2 * off + 2 * (float((s - s.max()).abs().max()) + 4) * U32 + (e + 8) * U32)
            out[i, x] = p @ vv
            size = p @ vv.abs()
            eo[i, x] = size * (r + (e + 4) * U32 + (U.half_step(dtype) if dtype == torch.bfloat16 else 0.0))
            add[i, j, :e] += p
            ea[i, j, :e] += p * (r + hq // h * U32)
    return out, eo, add, ea


def evict64(scores, lengths, budget, recent):
    """kept [b, h, budget] and the new lengths."""
    torch = _torch()
    scores = scores.cpu()
    b, h, n = scores.shape
    kept = torch.full((b, h, budget), -1, dtype=torch.int64)
    ends = []
    for i in range(b):
        e = n if lengths is None else max(0, min(n, int(lengths[i])))
        ends.append(min(e, budget))
        for j in range(h):
            if e <= budget:
                ids = list(range(e))
            else:
                old = e - recent
                row = [(-math.inf if x != x else -x, 0 if x != x else 1, t) for t, x in enumerate(scores[i, j, :old].tolist())]
                ids = sorted(t for _, _, t in sorted(row)[:budget - recent]) + list(range(old, e))
            kept[i, j, :len(ids)] = torch.tensor(ids, dtype=torch.int64)
    return kept, torch.tensor(ends, dtype=torch.int64)


def rows_of(cache, kept):
    """The cache's rows that stay, zeros behind them."""
    torch = _torch()
    c = cache.cpu()
    good = kept >= 0
    at = kept.clamp(min=0)
    if c.dim() == 3:
        return torch.where(good, c.gather(2, at), torch.zeros((), dtype=c.dtype)) if c.shape[2] else torch.zeros(kept.shape, dtype=c.dtype)
    if not c.shape[2]:
        return torch.zeros(*kept.shape, c.shape[3], dtype=c.dtype)
    g = c.gather(2, at[..., None].expand(*kept.shape, c.shape[3]))
    return torch.where(good[..., None], g, torch.zeros((), dtype=c.dtype))


# ---------------------------------------------------------------- the next token
def f32(v):
    """A number as the operator gets it."""
    torch = _torch()
    return float(torch.tensor(float(v), dtype=torch.float32))


def sample64(z, u, temperature, top_k, top_p, min_p):
    """(token, logprob) of one row, by lists of numbers in 64 bits."""
    z = [(-math.inf if x != x else x) for x in z.double().tolist()]
    top = max(z)
    if top == -math.inf:
        return -1, -math.inf
    order = sorted((i for i in range(len(z)) if z[i] > -math.inf), key=lambda i: (-z[i], i))
    if not temperature > 0:
        return order[0], 0.0

    def weight(i):
        return 1.0 if z[i] == top else math.exp((z[i] - top) / temperature)

    if top_k > 0:
        order = order[:top_k]
    w = [weight(i) for i in order]
    if not top_p >= 1:
        limit, at, n = top_p * math.fsum(w), 0.0, 0
        while n < len(w) and (n == 0 or at < limit):
            at += w[n]
            n += 1
        order, w = order[:n], w[:n]
    kept = sorted((i, x) for i, x in zip(order, w) if x >= min(min_p, 1.0))
    total = math.fsum(x for _, x in kept)
    target, at = u * total, 0.0
    for i, x in kept:
        at += x
        if at > target:
            return i, math.log(x / total)
    return kept[-1][0], math.log(kept[-1][1] / total)
