"""The training and serving operators around the BatchTopK selection, as cases to measure.

A BatchTopK sparse autoencoder encodes activations with one product (bias and
activation in its epilogue), keeps the largest latents of the whole batch,
decodes those few latents against the rows of a dictionary, and clips the
global norm of its gradients before the update.  The selection itself is
`top_selection_sample_amd.topk`; the operators measured here are the ones on
either side of it:

  linear       y = act(x W^T + b) + residual           x [m, k], W [n, k]
  linear_grad  (dx, dW, db) of it, from dy and the pre-activation z
  decode       out[r] = b + sum of v_e W[j_e] over the selected entries e of row r
  decode_grad  (dv, dW, db) of it
  encode_grad  (dx, dW, db) of the encoder through the selection: only the
               selected places of relu(x W^T + b) have a gradient
  clip         the global 2-norm of many gradients, and their scaling to at most max_norm

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
        # one token through the encoder of a 12288-latent dictionary: the product of serving
        dict(name="linear one token", op="linear", m=1, k=512, n=12288, dtype="bf16", act="relu", bias=True, residual=False),
        # the encoder of the 4096 x 65536 bfloat16 BatchTopK workload
        dict(name="linear encoder 65536", op="linear", m=4096, k=512, n=65536, dtype="bf16", act="relu", bias=True, residual=False),
        # odd sizes in float32, with a feed-forward epilogue: activation, then the residual stream
        dict(name="linear ragged f32", op="linear", m=1001, k=515, n=4099, dtype="f32", act="gelu", bias=True, residual=True),
        # dense backward of the encoder at 4096 x 12288, the paper's BatchTopK batch
        dict(name="linear_grad 12288 bf16", op="linear_grad", m=4096, k=512, n=12288, dtype="bf16", act="relu"),
        # dense backward in float32 with a smooth activation
        dict(name="linear_grad f32", op="linear_grad", m=2048, k=1024, n=4096, dtype="f32", act="silu"),
        # eight tokens, each with its own 32 latents (a batch of row-wise selections), one slot padded
        dict(name="decode 8 tokens", op="decode", rows=8, per_row=32, latents=12288, d=512, dtype="bf16", flat=False, bias=True, padded=1),
        # the flattened selection of the 4096 x 65536 workload: 131072 entries, rows of uneven counts
        dict(name="decode batch 65536", op="decode", rows=4096, per_row=32, latents=65536, d=512, dtype="bf16", flat=True, bias=True, padded=0),
        # its gradient at 12288 latents in float32
        dict(name="decode_grad 12288 f32", op="decode_grad", rows=4096, per_row=32, latents=12288, d=512, dtype="f32", flat=True, padded=0),
        # the encoder's gradient through the selection of the 65536-latent workload
        dict(name="encode_grad 65536 bf16", op="encode_grad", rows=4096, per_row=32, latents=65536, d=512, dtype="bf16", flat=True, padded=0),
        # a small model's worth of little tensors, scalars and odd lengths among them: launches count
        dict(name="clip 48 small", op="clip", tensors=48, least=1, most=4099, dtype="f32", bucket=False, max_norm=1.0),
        # an autoencoder of 65536 latents: encoder, decoder and the two biases
        dict(name="clip autoencoder f32", op="clip", tensors=0, latents=65536, d=512, dtype="f32", bucket=False, max_norm=1.0),
        # bfloat16 gradients of a middle-sized model, ragged, as the views of one packed bucket that data-parallel training keeps
        dict(name="clip 160 bf16", op="clip", tensors=160, least=17, most=1000003, dtype="bf16", bucket=True, max_norm=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "decode", "decode_grad", "encode_grad", "clip"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "linear":
        return dict(op=op, m=_log(rng, 1, 4096), k=_log(rng, 24, 1024), n=_log(rng, 24, 16384), dtype=dtype,
                    act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.7, residual=rng.random() < 0.4)
    if op == "linear_grad":
        return dict(op=op, m=_log(rng, 1, 4096), k=_log(rng, 24, 1024), n=_log(rng, 24, 8192), dtype=dtype,
                    act=rng.choice(["none", "relu", "gelu", "silu"]))
    if op == "clip":
        most = _log(rng, 10, 300000)
        bucket = rng.random() < 0.5
        return dict(op=op, tensors=_log(rng, 1, 200 if bucket else 60), least=rng.randint(1, 9), most=most, dtype=dtype, bucket=bucket,
                    max_norm=rng.choice([0.1, 0.5, 1.0]))
    rows, per = _log(rng, 1, 4096), _log(rng, 1, 64)
    c = dict(op=op, rows=rows, per_row=per, latents=_log(rng, 4 * per, 40000), d=_log(rng, 24, 1024), dtype=dtype,
             flat=rng.random() < 0.6, padded=rng.choice([0, 0, 1, 3]))
    if op == "decode":
        c["bias"] = rng.random() < 0.7
    if op == "encode_grad":
        c["flat"] = True   # the encoder selects over the whole batch
    c["padded"] = min(c["padded"], per - 1)
    return c


# ---------------------------------------------------------------- the inputs
def _selection(c, g):
    """Values and indices as the selection returns them: rank order (largest
    value first), places distinct, latents of very uneven popularity, the
    padded slots of a relaxed-recall selection at the end."""
    rows, per, n = c["rows"], c["per_row"], c["latents"]
    dev = "cuda"
    if c["flat"]:
        total = rows * per
        order = torch.randperm(n, generator=g, device=dev)
        places, want = None, 2 * total + 64
        while places is None or places.numel() < total:
            # a cubed uniform number: a few latents are in nearly every row, most in hardly any
            u = torch.rand(want, generator=g, device=dev, dtype=torch.float64)
            j = (u * u * u * n).long().clamp_(max=n - 1)
            r = torch.randint(0, rows, (want,), generator=g, device=dev)
            got = r * n + order[j]
            places = torch.unique(got if places is None else torch.cat([places, got]))
            want *= 2
        idx = places[torch.randperm(places.numel(), generator=g, device=dev)[:total]]
        shape = (total,)
    else:
        idx = torch.rand(rows, n, generator=g, device=dev).argsort(1)[:, :per].contiguous()
        shape = (rows, per)
    vals = torch.randn(shape, generator=g, device=dev).abs().add(0.25).sort(-1, descending=True).values.to(DT[c["dtype"]])
    if c["padded"]:
        idx[..., -c["padded"]:] = -1
        vals[..., -c["padded"]:] = -math.inf
    return vals, idx


def _clip_sizes(c, seed):
    if not c["tensors"]:
        return [(c["latents"], c["d"]), (c["latents"],), (c["latents"], c["d"]), (c["d"],)]
    import random
    r = random.Random(seed)
    return [(_log(r, c["least"], max(c["least"], c["most"])),) for _ in range(c["tensors"])]


def prepare(case, seed):
    c, dt = case, DT[case["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)

    s = {"case": c}
    if c["op"] == "linear":
        s["x"] = randn(c["m"], c["k"])
        s["w"] = randn(c["n"], c["k"], scale=c["k"] ** -0.5)
        s["b"] = randn(c["n"], scale=0.1) if c["bias"] else None
        s["res"] = randn(c["m"], c["n"]) if c["residual"] else None
    elif c["op"] == "linear_grad":
        s["x"] = randn(c["m"], c["k"])
        s["w"] = randn(c["n"], c["k"], scale=c["k"] ** -0.5)
        s["dy"] = randn(c["m"], c["n"])
        s["pre"] = randn(c["m"], c["n"]) if c["act"] != "none" else None
    elif c["op"] == "clip":
        # gradients of one model: each tensor has a scale of its own
        sizes = _clip_sizes(c, 77)   # the model's shapes are the same whatever its gradients
        scales = torch.rand(len(sizes), generator=g, device="cuda").mul(4).add(0.05)
        s["grads"] = [(torch.randn(*z, generator=g, device="cuda") * scales[i]).to(dt) for i, z in enumerate(sizes)]
        s["held"] = s["grads"]
        if c["bucket"]:   # packed without gaps: the views start at any multiple of the element size
            s["held"] = [torch.cat([t.reshape(-1) for t in s["grads"]])]
            s["grads"] = list(s["held"][0].split([t.numel() for t in s["grads"]]))
    else:
        s["v"], s["idx"] = _selection(c, g)
        if c["op"] == "encode_grad":
            s["x"] = randn(c["rows"], c["d"])
            s["gv"] = randn(*s["v"].shape)
        elif c["op"] == "decode_grad":
            s["g"] = randn(c["rows"], c["d"])
        else:
            s["b"] = randn(c["d"], scale=0.1) if c["bias"] else None
        s["w"] = randn(c["latents"], c["d"], scale=c["d"] ** -0.5)
    return s


# ---------------------------------------------------------------- the plain forms
def _act(z, kind):
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _slope(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    p = 1 / (1 + torch.exp(-z))
    return p * (1 + z * (1 - p))


def _places(idx, rows, n):
    """Row and latent of each entry, and whether it is one (padded slots are not)."""
    keep = idx >= 0
    at = idx.clamp(min=0)
    if idx.dim() == 2:
        r = torch.arange(rows, device=idx.device)[:, None].expand_as(idx).reshape(-1)
        return r, at.reshape(-1), keep.reshape(-1)
    return at // n, at % n, keep


def _plain(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    op = c["op"]
    if op == "linear":
        z = s["x"].float() @ s["w"].float().t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, c["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        return y.to(dt)
    if op == "linear_grad":
        dz = s["dy"].float()
        if c["act"] != "none":
            dz = dz * _slope(s["pre"].float(), c["act"])
        return (dz @ s["w"].float()).to(dt), (dz.t() @ s["x"].float()).to(dt), dz.sum(0).to(dt)
    if op == "clip":
        grads = s["grads"]
        norm = torch.stack([t.float().square().sum() for t in grads]).sum().sqrt()
        scale = (c["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        done = [t.copy_(t.float() * scale) for t in grads]
        return [norm, s["held"] if c["bucket"] else done]
    r, j, keep = _places(s["idx"], c["rows"], c["latents"])
    v = torch.where(keep, s["v"].reshape(-1).float(), 0.0)
    d = c["d"]
    if op == "decode":
        out = torch.zeros(c["rows"], d, device=v.device).index_add_(0, r, v[:, None] * s["w"][j].float())
        if s["b"] is not None:
            out = out + s["b"].float()
        return out.to(dt)
    if op == "decode_grad":
        g = s["g"][r].float()
        dv = torch.where(keep, (g * s["w"][j].float()).sum(1), 0.0).reshape(s["v"].shape)
        dw = torch.zeros(c["latents"], d, device=v.device).index_add_(0, j, v[:, None] * g)
        return dv.to(dt), dw.to(dt), s["g"].float().sum(0).to(dt)
    gp = torch.where(keep & (v > 0), s["gv"].reshape(-1).float(), 0.0)
    dx = torch.zeros(c["rows"], d, device=v.device).index_add_(0, r, gp[:, None] * s["w"][j].float())
    dw = torch.zeros(c["latents"], d, device=v.device).index_add_(0, j, gp[:, None] * s["x"][r].float())
    db = torch.zeros(c["latents"], device=v.device).index_add_(0, j, gp)
    return dx.to(dt), dw.to(dt), db.to(dt)


# ---------------------------------------------------------------- the package's operators
def _own(s):
    import top_selection_sample_amd as tss
    c = s["case"]
    op = c["op"]
    if op == "linear":
        return tss.linear(s["x"], s["w"], s["b"], activation=c["act"], residual=s["res"])
    if op == "linear_grad":
        return tss.linear_grad(s["dy"], s["x"], s["w"], activation=c["act"], pre=s["pre"])
    if op == "clip":
        return [tss.clip_grad_norm(s["grads"], c["max_norm"]), s["held"]]
    if op == "decode":
        return tss.decode(s["v"], s["idx"], s["w"], rows=c["rows"], bias=s["b"])
    if op == "decode_grad":
        return tss.decode_grad(s["g"], s["v"], s["idx"], s["w"])
    return tss.encode_grad(s["gv"], s["v"], s["idx"], s["x"], s["w"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c, e = case, SIZE[case["dtype"]]
    op = c["op"]
    if op == "linear":
        m, k, n = c["m"], c["k"], c["n"]
        return {"bytes": e * (m * k + n * k + (n if c["bias"] else 0) + m * n * (2 if c["residual"] else 1)), "flops": 2 * m * n * k}
    if op == "linear_grad":
        m, k, n = c["m"], c["k"], c["n"]
        return {"bytes": e * (m * n * (1 if c["act"] == "none" else 2) + 2 * (m * k + n * k) + n), "flops": 4 * m * n * k}
    if op == "clip":
        n = sum(math.prod(z) for z in _clip_sizes(c, 77))
        return {"bytes": 2 * e * n + 4, "flops": 3 * n}
    rows, d, n, total = c["rows"], c["d"], c["latents"], c["rows"] * c["per_row"]
    used = min(total, n)   # weight rows that an entry can name
    if op == "decode":
        return {"bytes": total * (8 + e) + e * d * (used + rows + (1 if c["bias"] else 0)), "flops": 2 * total * d}
    if op == "decode_grad":
        return {"bytes": total * (8 + 2 * e) + e * d * (rows + used + n + 1), "flops": 4 * total * d}
    return {"bytes": total * (8 + 2 * e) + e * (d * (2 * rows + used + n) + n), "flops": 4 * total * d}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    c = case
    s = prepare(case, seed)
    f = {k: (v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v) for k, v in s.items()}
    op = c["op"]
    if op == "linear":
        z = torch.mm(f["x"], f["w"].t().contiguous())
        if f["b"] is not None:
            z += f["b"][None, :]
        if c["act"] == "relu":
            z = torch.where(z > 0, z, torch.zeros_like(z))
        elif c["act"] == "gelu":
            z = z * torch.special.ndtr(z)
        elif c["act"] == "silu":
            z = z * torch.sigmoid(z)
        return z if f["res"] is None else z + f["res"]
    if op == "linear_grad":
        dz = f["dy"]
        if c["act"] == "relu":
            dz = torch.where(f["pre"] > 0, dz, torch.zeros_like(dz))
        elif c["act"] == "gelu":
            z = f["pre"]
            dz = dz * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
        elif c["act"] == "silu":
            p = torch.sigmoid(f["pre"])
            dz = dz * (p + f["pre"] * p * (1 - p))
        return torch.mm(dz, f["w"]), torch.mm(dz.t().contiguous(), f["x"]), torch.sum(dz, 0)
    if op == "clip":
        flat = torch.cat([t.double().reshape(-1) for t in s["held"]])
        norm = torch.linalg.vector_norm(flat)
        scale = min(1.0, c["max_norm"] / (float(norm) + 1e-6))
        return [norm, [t.double() * scale for t in s["held"]]]
    # through the dense activation that the selection stands for, when that fits; entry by entry otherwise
    rows, n, d = c["rows"], c["latents"], c["d"]
    good = s["idx"] >= 0
    if s["idx"].dim() == 2:
        flat = (torch.arange(rows, device="cuda")[:, None] * n + s["idx"])[good]
    else:
        flat = s["idx"][good]
    row, col = torch.div(flat, n, rounding_mode="floor"), torch.remainder(flat, n)

    def product(coef, by_row, matrix):
        """sum over entries of coef * matrix[other], into the rows of `by_row`."""
        if by_row:
            a = torch.sparse_coo_tensor(torch.stack([row, col]), coef, (rows, n))
        else:
            a = torch.sparse_coo_tensor(torch.stack([col, row]), coef, (n, rows))
        return torch.sparse.mm(a, matrix)

    if op == "decode":
        out = product(f["v"][good], True, f["w"])
        return out if f["b"] is None else out + f["b"]
    if op == "decode_grad":
        dv = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
        dv[good] = torch.linalg.vecdot(f["g"].index_select(0, row), f["w"].index_select(0, col))
        return dv, product(f["v"][good], False, f["g"]), torch.sum(f["g"], 0)
    coef = torch.where(f["v"] > 0, f["gv"], torch.zeros_like(f["gv"]))[good]
    return product(coef, True, f["w"]), product(coef, False, f["x"]), torch.bincount(col, weights=coef, minlength=n)
