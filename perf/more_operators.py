"""Operators that act on a selection of a language model, as cases to measure.

The package selects the largest entries of a row.  In a language model three
things hang on such a selection: which token comes next, which experts a token
goes to, and which entries of an attention cache stay.

  sample        the next token of each row of logits: temperature, then the top k,
                then the smallest set of them with probability top_p, then those of
                at least min_p times the largest; drawn by a given number u in [0, 1)
  dispatch      rows of x [t, d] sorted by expert (stable), a copy for each of a
                token's k experts; the place of each copy; where each expert begins
  combine       out[i] = sum over j of weights[i, j] y[places[i, j]]; without weights
                it is the gradient of dispatch
  combine_grad  (dy, dweights) of it
  attend        attention of one new token for each sequence over its cache, which
                adds the probabilities (summed over the heads that share a
                key-value head) to the cache's accumulated weights
  evict         the cache of `budget` entries a head: the `recent` newest ones and,
                of the others, those with the largest accumulated weights, in their
                old order

`run` computes them in elementary torch operations, or with the package's own
entry points where `own` is set.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one user's next token: latency; the selection's threshold inside a long row
        dict(name="sample one row", op="sample", rows=1, n=131072, dtype="f32", per_row=False, temperature=0.8, top_k=50, top_p=0.95, min_p=0.0, masked=0.0),
        # a serving batch, each request with settings of its own, logits in bfloat16 (many equal ones), a third masked by a grammar
        dict(name="sample 64 requests", op="sample", rows=64, n=100003, dtype="bf16", per_row=True, temperature=1.0, top_k=200, top_p=0.9, min_p=0.02, masked=0.3),
        # rollouts for training: a large batch at temperature 1, nothing but a floor on the probabilities
        dict(name="sample 256 rollouts", op="sample", rows=256, n=65536, dtype="f32", per_row=False, temperature=1.0, top_k=0, top_p=1.0, min_p=0.05, masked=0.0),
        # a decoding step of eight sequences through eight experts
        dict(name="dispatch 8 tokens", op="dispatch", t=8, k=2, experts=8, d=1024, dtype="bf16", dropped=0.0),
        # a training batch through 128 experts of uneven popularity
        dict(name="dispatch 16384 tokens", op="dispatch", t=16384, k=8, experts=128, d=1024, dtype="bf16", dropped=0.0),
        # back from the experts in the same decoding step
        dict(name="combine 8 tokens", op="combine", t=8, k=2, experts=8, d=1024, dtype="bf16", wdtype="f32", weighted=True, dropped=0.0),
        # odd sizes in float32, some copies dropped at their expert's capacity
        dict(name="combine ragged f32", op="combine", t=4099, k=4, experts=60, d=515, dtype="f32", wdtype="f32", weighted=True, dropped=0.05),
        # the gradient of a training batch; the router's weights in float32 beside bfloat16 rows
        dict(name="combine_grad 8192 tokens", op="combine_grad", t=8192, k=8, experts=128, d=1024, dtype="bf16", wdtype="f32", weighted=True, dropped=0.0),
        # one sequence, twelve heads on four, an odd length and a width that is no power of two, float32
        dict(name="attend one sequence f32", op="attend", b=1, hq=12, hkv=4, n=4099, d=80, dtype="f32", ragged=False),
        # a serving batch of long sequences of different lengths, 32 heads on 8
        dict(name="attend 16 sequences", op="attend", b=16, hq=32, hkv=8, n=8192, d=128, dtype="bf16", ragged=True),
        # one sequence's cache halved
        dict(name="evict one sequence f32", op="evict", b=1, hkv=4, n=2049, d=80, budget=1024, recent=64, dtype="f32", ragged=False),
        # the prompts of a batch cut to a quarter of the room
        dict(name="evict 16 prompts", op="evict", b=16, hkv=8, n=16384, d=128, budget=4096, recent=256, dtype="bf16", ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "dispatch", "combine", "combine_grad", "attend", "evict"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "sample":
        n = _log(rng, 1000, 200000)
        return dict(op=op, rows=_log(rng, 1, min(256, 16777216 // n)), n=n, dtype=dtype, per_row=rng.random() < 0.5,
                    temperature=rng.choice([0.6, 0.8, 1.0, 1.3]), top_k=rng.choice([0, 0, 1, 20, 50, 1000]), top_p=rng.choice([1.0, 0.95, 0.8, 0.5]),
                    min_p=rng.choice([0.0, 0.0, 0.02, 0.1]), masked=rng.choice([0.0, 0.0, 0.5]))
    if op in ("dispatch", "combine", "combine_grad"):
        k = rng.choice([1, 2, 4, 6, 8])
        d = _log(rng, 24, 4096)
        c = dict(op=op, t=_log(rng, 1, min(16384, 60000000 // (k * d))), k=k, experts=_log(rng, max(k, 4), 256), d=d, dtype=dtype,
                 dropped=rng.choice([0.0, 0.0, 0.1]))
        if op != "dispatch":
            c["wdtype"] = rng.choice(["f32", dtype])
            c["weighted"] = op == "combine_grad" or rng.random() < 0.7
        return c
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 80, 96, 128, 128, 256, rng.randint(8, 200)])
    n = _log(rng, 1, 20000)
    b = _log(rng, 1, max(1, min(32, 100000000 // (n * hkv * d))))
    if op == "attend":
        return dict(op=op, b=b, hq=hkv * rng.choice([1, 2, 3, 4, 8]), hkv=hkv, n=n, d=d, dtype=dtype, ragged=rng.random() < 0.5)
    budget = max(1, int(n * rng.choice([0.1, 0.25, 0.5, 0.9])))
    return dict(op=op, b=b, hkv=hkv, n=n, d=d, budget=budget, recent=int(budget * rng.choice([0.0, 0.1, 0.5])), dtype=dtype, ragged=rng.random() < 0.5)


# ---------------------------------------------------------------- the inputs
def _lengths(c, g):
    """Sequence lengths: all the room, or anything from one entry up, one of them all of it."""
    if not c["ragged"]:
        return None
    n = torch.randint(1, c["n"] + 1, (c["b"],), generator=g, device="cuda")
    n[c["b"] // 2] = c["n"]
    return n


def _experts(c, g):
    """The experts of each token, largest router score first: the popular ones are in many rows."""
    score = torch.randn(c["t"], c["experts"], generator=g, device="cuda") + torch.randn(c["experts"], generator=g, device="cuda")
    experts = score.topk(c["k"], dim=1).indices
    if c["dropped"]:
        experts[torch.rand(c["t"], c["k"], generator=g, device="cuda") < c["dropped"]] = -1
    return experts, score


def _places(experts, count):
    """Where each (token, expert) pair lies when all are sorted by expert; -1 for the dropped ones."""
    e = experts.reshape(-1)
    key = torch.where((e >= 0) & (e < count), e, count)
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    return torch.where(key < count, place, -1).reshape(experts.shape), order, key


def prepare(case, seed):
    c, dt = case, DT[case["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=None):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype or dt)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": c}
    op = c["op"]
    if op == "sample":
        rows, n = c["rows"], c["n"]
        z = torch.randn(rows, n, generator=g, device="cuda") * (1.5 + rand(rows, 1))
        if c["masked"]:
            z.masked_fill_(rand(rows, n) < c["masked"], -math.inf)
            z[:, n // 2] = 1.0   # a mask leaves something
        s["z"], s["u"] = z.to(dt), rand(rows)
        names = ("temperature", "top_k", "top_p", "min_p")
        if c["per_row"]:
            s["settings"] = {"temperature": c["temperature"] * (0.5 + rand(rows)), "top_p": c["top_p"] * (0.75 + 0.25 * rand(rows)),
                             "min_p": c["min_p"] * rand(rows),
                             "top_k": torch.randint(max(1, c["top_k"] // 2), c["top_k"] + 1, (rows,), generator=g, device="cuda") if c["top_k"] else
                             torch.zeros(rows, dtype=torch.int64, device="cuda")}
            s["settings"]["temperature"][0] = 0   # one request decodes greedily
        else:
            s["settings"] = {k: c[k] for k in names}
    elif op == "dispatch":
        s["x"] = randn(c["t"], c["d"])
        s["experts"] = _experts(c, g)[0]
    elif op in ("combine", "combine_grad"):
        experts, score = _experts(c, g)
        s["places"] = _places(experts, c["experts"])[0]
        s["y"] = randn(c["t"] * c["k"], c["d"])
        s["w"] = None
        if c["weighted"]:   # the router's softmax over the chosen experts
            s["w"] = score.gather(1, experts.clamp(min=0)).softmax(1).to(DT[c["wdtype"]])
        if op == "combine_grad":
            s["g"] = randn(c["t"], c["d"])
    elif op == "attend":
        s["q"] = randn(c["b"], c["hq"], c["d"], scale=1.5)
        s["k"], s["v"] = (randn(c["b"], c["hkv"], c["n"], c["d"]) for _ in range(2))
        s["lengths"] = _lengths(c, g)
        s["scores"] = rand(c["b"], c["hkv"], c["n"])
    else:
        s["k"], s["v"] = (randn(c["b"], c["hkv"], c["n"], c["d"]) for _ in range(2))
        # a few entries carry most of the weight; many were never looked at and are equal: 0
        w = torch.randn(c["b"], c["hkv"], c["n"], generator=g, device="cuda").mul_(2).exp_()
        s["scores"] = w.masked_fill_(rand(c["b"], c["hkv"], c["n"]) < 0.2, 0.0)
        s["lengths"] = _lengths(c, g)
    return s


# ---------------------------------------------------------------- the plain forms
def _column(v, rows, dtype):
    if not isinstance(v, torch.Tensor):
        v = torch.full((rows,), v, device="cuda")
    return v.to(dtype)[:, None]


def _plain_sample(s):
    """In 64 bits: which token it is hangs on sums over the whole row, next to a border."""
    z = s["z"].double()
    rows, n = z.shape
    # a number reaches the operator in 32 bits, as its tensors do
    temperature, top_p, min_p = (_column(s["settings"][k], rows, torch.float32).double() for k in ("temperature", "top_p", "min_p"))
    top_k = _column(s["settings"]["top_k"], rows, torch.int64)
    z = torch.where(torch.isnan(z), -math.inf, z)
    zs, order = z.sort(dim=1, descending=True, stable=True)
    top = zs[:, :1]
    w = torch.where(zs == top, 1.0, torch.exp((zs - top) / temperature))
    w = torch.where(zs == -math.inf, 0.0, w)
    rank = torch.arange(n, device=z.device)[None]
    w = torch.where((top_k <= 0) | (rank < top_k), w, 0.0)
    before = w.cumsum(1) - w
    keep = (top_p >= 1) | (before < top_p * w.sum(1, keepdim=True)) | (rank == 0)
    keep &= w >= min_p.clamp(max=1)
    keep &= (temperature > 0) | (rank == 0)
    w = torch.where(keep, w, 0.0)
    back = torch.zeros_like(w).scatter_(1, order, w)
    sums = back.cumsum(1)
    total = sums[:, -1:]
    token = (sums <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    last = torch.where(back > 0, rank, -1).amax(1, keepdim=True)
    token = torch.minimum(token, last)
    prob = torch.where(token >= 0, back.gather(1, token.clamp(min=0)) / total, 0.0)
    return token[:, 0], prob.log()[:, 0].float()


def _plain(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    op = c["op"]
    if op == "sample":
        return _plain_sample(s)
    if op == "dispatch":
        places, order, key = _places(s["experts"], c["experts"])
        rows = s["x"][order // c["k"]]
        rows = torch.where((key[order] < c["experts"])[:, None], rows, torch.zeros_like(rows))
        edges = torch.arange(c["experts"] + 1, device=key.device)
        return rows, places, (key[:, None] < edges).sum(0)
    if op in ("combine", "combine_grad"):
        keep = (s["places"] >= 0)[..., None]
        y = torch.where(keep, s["y"][s["places"].clamp(min=0)].float(), 0.0)
        if op == "combine":
            return (y if s["w"] is None else y * s["w"].float()[..., None]).sum(1).to(dt)
        g = s["g"].float()[:, None]
        dw = (y * g).sum(2)
        dy = torch.zeros(s["y"].shape, device=y.device)
        dy.index_add_(0, s["places"].clamp(min=0).reshape(-1), torch.where(keep, g * s["w"].float()[..., None], 0.0).flatten(0, 1))
        return dy.to(dt), dw.to(s["w"].dtype)
    n = c["n"]
    lengths = s["lengths"] if s["lengths"] is not None else torch.full((c["b"],), n, device="cuda")
    at = torch.arange(n, device="cuda")
    if op == "attend":
        k, v = s["k"].float(), s["v"].float()
        q = s["q"].float().reshape(c["b"], c["hkv"], c["hq"] // c["hkv"], c["d"])
        logits = (k @ q.transpose(2, 3).contiguous()).transpose(2, 3) * c["d"] ** -0.5
        logits = torch.where(at < lengths[:, None, None, None], logits, -math.inf)
        p = torch.exp(logits - logits.amax(3, keepdim=True))
        p = p / p.sum(3, keepdim=True)
        s["scores"] += p.sum(2)
        return (p.contiguous() @ v).reshape(s["q"].shape).to(dt), s["scores"]
    b, h, m = c["b"], c["hkv"], c["budget"]
    lengths = lengths[:, None, None]
    kept = lengths.clamp(max=m)
    value = torch.where(at >= lengths - min(c["recent"], m), math.inf, s["scores"])
    value = torch.where(at < lengths, value, -1.0)
    chosen = value.sort(dim=2, descending=True, stable=True).indices[..., :m]
    slot = torch.arange(m, device="cuda")
    chosen = torch.where(slot < kept, chosen, n).sort(dim=2).values
    good = chosen < n
    pick = torch.where(good, chosen, 0)
    rows = [torch.where(good[..., None], t.gather(2, pick[..., None].expand(b, h, m, c["d"])), torch.zeros((), dtype=dt, device="cuda")) for t in (s["k"], s["v"])]
    return rows[0], rows[1], torch.where(good, s["scores"].gather(2, pick), 0.0), torch.where(good, chosen, -1), kept[:, 0, 0]


# ---------------------------------------------------------------- the package's operators
def _own(s):
    import top_selection_sample_amd as tss
    c = s["case"]
    op = c["op"]
    if op == "sample":
        return tss.sample(s["z"], s["u"], **s["settings"])
    if op == "dispatch":
        return tss.dispatch(s["x"], s["experts"], c["experts"])
    if op == "combine":
        return tss.combine(s["y"], s["places"], s["w"])
    if op == "combine_grad":
        return tss.combine_grad(s["g"], s["y"], s["places"], s["w"])
    if op == "attend":
        return tss.attend(s["q"], s["k"], s["v"], lengths=s["lengths"], scores=s["scores"]), s["scores"]
    return tss.evict(s["k"], s["v"], s["scores"], c["budget"], recent=min(c["recent"], c["budget"]), lengths=s["lengths"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c, e = case, SIZE[case["dtype"]]
    op = c["op"]
    if op == "sample":   # a difference, a scaling and a sum for each logit beside its exponential
        return {"bytes": c["rows"] * (c["n"] * e + 16), "flops": 3 * c["rows"] * c["n"]}
    if op in ("dispatch", "combine", "combine_grad"):
        t, k, d = c["t"], c["k"], c["d"]
        entries = t * k * 8   # experts or places
        if op == "dispatch":
            return {"bytes": e * d * (t + t * k) + 2 * entries + 8 * (c["experts"] + 1), "flops": 0}
        w = SIZE[c["wdtype"]] * t * k if c["weighted"] else 0
        if op == "combine":
            return {"bytes": e * d * (t + t * k) + entries + w, "flops": 2 * t * k * d}
        return {"bytes": e * d * (t + 2 * t * k) + entries + 2 * w, "flops": 3 * t * k * d}
    # lengths are spread evenly up to all the room
    b, h, n, d = c["b"], c["hkv"], c["n"] * (0.5 if c["ragged"] and c["b"] > 1 else 1.0), c["d"]
    if op == "attend":
        return {"bytes": b * h * n * (2 * d * e + 8) + 2 * b * c["hq"] * d * e, "flops": 4 * b * c["hq"] * n * d}
    m = min(c["budget"], n)
    return {"bytes": b * h * (4 * n + m * (4 * d * e + 8 + 8)), "flops": b * h * n}


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_row(z, u, temperature, top_k, top_p, min_p):
    """One row by sets: the kept tokens as positions of the row sorted by (logit, position)."""
    z = torch.nan_to_num(z.double(), nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    live = (z > -math.inf).nonzero()[:, 0]
    if live.numel() == 0:
        return -1, -math.inf
    live = live[torch.argsort(-z[live], stable=True)]
    if temperature <= 0:
        return int(live[0]), 0.0
    if 0 < top_k < live.numel():
        live = live[:top_k]
    v = z[live]
    p = torch.softmax(torch.where(v == v[0], 0.0, (v - v[0]) / temperature), 0)
    if top_p < 1:
        reach = torch.cumsum(p, 0)
        count = int((reach < top_p).sum()) + 1
        live, p = live[:count], p[:count]
    good = p >= min(min_p, 1.0) * p[0]
    live, p = live[good], p[good] / p[good].sum()
    place = torch.argsort(live)
    at = int(torch.searchsorted(torch.cumsum(p[place], 0), torch.tensor([u], dtype=torch.float64, device=z.device), right=True))
    at = place[min(at, live.numel() - 1)]
    return int(live[at]), math.log(float(p[at]))


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    op = c["op"]
    if op == "sample":
        got = []
        for r in range(c["rows"]):
            single = {k: (v[r].item() if isinstance(v, torch.Tensor) else torch.tensor(float(v)).item()) for k, v in s["settings"].items()}
            single["top_k"] = int(single["top_k"])
            got.append(_exact_row(s["z"][r], s["u"][r].item(), **single))
        return (torch.tensor([t for t, _ in got], device="cuda"), torch.tensor([p for _, p in got], dtype=torch.float64, device="cuda"))
    if op == "dispatch":
        ids = s["experts"]
        rows, place, edges = [], torch.full_like(ids, -1), [0]
        for e in range(c["experts"]):
            where = (ids == e).nonzero()   # token by token, in order
            rows.append(s["x"][where[:, 0]].double())
            place[where[:, 0], where[:, 1]] = edges[-1] + torch.arange(len(where), device="cuda")
            edges.append(edges[-1] + len(where))
        rows.append(torch.zeros(ids.numel() - edges[-1], c["d"], dtype=torch.float64, device="cuda"))
        return torch.cat(rows), place, torch.tensor(edges, device="cuda")
    if op in ("combine", "combine_grad"):
        t, k = c["t"], c["k"]
        w = torch.ones(t, k, dtype=torch.float64, device="cuda") if s["w"] is None else s["w"].double()
        if op == "combine":
            out = torch.zeros(t, c["d"], dtype=torch.float64, device="cuda")
            for j in range(k):
                good = s["places"][:, j] >= 0
                out[good] += w[good, j, None] * s["y"][s["places"][good, j]].double()
            return out
        dy = torch.zeros(t * k, c["d"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(t, k, dtype=torch.float64, device="cuda")
        for j in range(k):   # no place occurs twice
            good = (s["places"][:, j] >= 0).nonzero()[:, 0]
            at, g = s["places"][good, j], s["g"][good].double()
            dy[at] = w[good, j, None] * g
            dw[good, j] = torch.linalg.vecdot(s["y"][at].double(), g)
        return dy, dw
    ends = [c["n"]] * c["b"] if s["lengths"] is None else s["lengths"].tolist()
    if op == "attend":
        out, scores = torch.zeros(c["b"], c["hq"], c["d"], dtype=torch.float64, device="cuda"), s["scores"].double()
        share = c["hq"] // c["hkv"]
        for i, e in enumerate(ends):
            for h in range(c["hkv"]):
                k, v = s["k"][i, h, :e].double(), s["v"][i, h, :e].double()
                for x in range(h * share, (h + 1) * share):
                    p = torch.softmax(torch.mv(k, s["q"][i, x].double()) / math.sqrt(c["d"]), 0)
                    out[i, x] = torch.mv(v.t().contiguous(), p)
                    scores[i, h, :e] += p
        return out, scores
    m, recent = c["budget"], min(c["recent"], c["budget"])
    k2, v2 = (torch.zeros(c["b"], c["hkv"], m, c["d"], dtype=torch.float64, device="cuda") for _ in range(2))
    s2 = torch.zeros(c["b"], c["hkv"], m, dtype=torch.float64, device="cuda")
    kept = torch.full((c["b"], c["hkv"], m), -1, device="cuda")
    for i, e in enumerate(ends):
        for h in range(c["hkv"]):
            old = e - min(recent, e)
            best = torch.argsort(-s["scores"][i, h, :old].double(), stable=True)[: max(0, min(m, e) - (e - old))]
            ids = torch.cat([best.sort().values, torch.arange(old, e, device="cuda")])
            x = ids.numel()
            kept[i, h, :x] = ids
            k2[i, h, :x], v2[i, h, :x] = s["k"][i, h, ids].double(), s["v"][i, h, ids].double()
            s2[i, h, :x] = s["scores"][i, h, ids].double()
    return k2, v2, s2, kept, torch.tensor([min(e, m) for e in ends], device="cuda")
