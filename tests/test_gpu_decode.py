"""The sparse decode of a selection, its gradients, and the encoder's gradient
through the selection, against 64 bits: flattened and row-wise selections,
empty rows, one row with every entry, padded slots, repeated places, widths
around the vectors, strides and alignment, streams and graphs."""
import math

import pytest

import ops_util as U

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def tss():
    import top_selection_sample_amd
    return top_selection_sample_amd


def rnd(seed, *shape, dt="f32", scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(DT[dt]).cuda()


def ints(seed, hi, *shape):
    return torch.randint(0, hi, shape, generator=torch.Generator().manual_seed(seed)).cuda()


def check_all(v, idx, rows, n, d, dt, label, seed=100):
    """decode, decode_grad and encode_grad of one selection against 64 bits."""
    T = tss()
    w, b = rnd(seed, n, d, dt=dt), rnd(seed + 1, d, dt=dt)
    g, x, gv = rnd(seed + 2, rows, d, dt=dt), rnd(seed + 3, rows, d, dt=dt), rnd(seed + 4, *v.shape, dt=dt)
    e, r, j = U.entries(idx, rows, n)
    vals = v.reshape(-1).cpu()[e].double()
    ref, err = U.group64(vals, r, j, rows, w)
    b64 = b.cpu().double()
    U.within(T.decode(v, idx, w, rows=rows).cpu(), ref, err, label + " decode")
    U.within(T.decode(v, idx, w, rows=rows, bias=b).cpu(), ref + b64,
             err + U.U32 * (ref.abs() + b64.abs()), label + " decode with bias")
    dv, dw, db = T.decode_grad(g, v, idx, w)
    gr, wj = g.cpu().double()[r], w.cpu().double()[j]
    want = torch.zeros(v.numel(), dtype=torch.float64)
    bound = torch.zeros_like(want)
    want[e] = (gr * wj).sum(1)
    bound[e] = (d + 3) * U.U32 * (gr * wj).abs().sum(1)
    U.within(dv.reshape(-1).cpu(), want, bound, label + " dvalues")
    ref, err = U.group64(vals, j, r, n, g)
    U.within(dw.cpu(), ref, err, label + " dweight")
    U.within(db.cpu(), g.cpu().double().sum(0), (rows + 3) * U.U32 * g.cpu().double().abs().sum(0), label + " dbias")
    dx, dwe, dbe = T.encode_grad(gv, v, idx, x, w)
    c = torch.where(vals > 0, gv.reshape(-1).cpu()[e].double(), torch.zeros_like(vals))
    ref, err = U.group64(c, r, j, rows, w)
    U.within(dx.cpu(), ref, err, label + " encoder dx")
    ref, err = U.group64(c, j, r, n, x)
    U.within(dwe.cpu(), ref, err, label + " encoder dweight")
    ref, err = U.group64(c, j, torch.zeros_like(j), n, torch.ones(1, 1))
    U.within(dbe.cpu(), ref[:, 0], err[:, 0], label + " encoder dbias")
    only = T.encode_grad(gv, v, idx, x, w, need=(0, 0, 1))
    assert only[0] is None and only[1] is None and torch.equal(only[2], dbe)
    some = T.decode_grad(g, v, idx, w, need=(0, 1, 0))
    assert some[0] is None and some[2] is None and torch.equal(some[1], dw)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,n,d", [(1, 1, 1, 1), (1, 32, 100, 512), (3, 7, 50, 33), (8, 32, 12288, 512),
                                        (70, 5, 300, 64), (2, 64, 64, 1030), (300, 1, 9, 8), (5, 200, 400, 257),
                                        (1, 3000, 5000, 40)])
def test_row_wise(rows, k, n, d, dt):
    idx = torch.stack([torch.randperm(n, generator=torch.Generator().manual_seed(i))[:k] for i in range(rows)]).cuda()
    v = rnd(1, rows, k, dt=dt).abs().sort(1, descending=True).values
    check_all(v, idx, rows, n, d, dt, f"row-wise {rows}x{k} of {n}, {d} wide")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,total,n,d", [(1, 1, 1, 1), (1, 50, 300, 512), (4, 64, 40, 65), (33, 500, 70, 512),
                                            (100, 4097, 1000, 96), (257, 9000, 300, 40), (64, 5000, 80, 520),
                                            (5000, 6000, 3, 16), (3, 20000, 9001, 8), (700, 30000, 66000, 24)])
def test_flattened(rows, total, n, d, dt):
    places = torch.randperm(rows * n, generator=torch.Generator().manual_seed(2))[:total].cuda()
    v = rnd(3, total, dt=dt).abs().sort(descending=True).values
    check_all(v, places, rows, n, d, dt, f"flat {total} of {rows}x{n}, {d} wide")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,total,n,d", [(2000, 1_200_000, 3001, 9), (3, 4096, 300_000, 20), (3, 4097, 300_000, 20),
                                            (9, 100_000, 20_000, 17)])
def test_many_entries_and_many_latents(rows, total, n, d, dt):
    idx = ints(14, rows * n, total)      # places may repeat
    check_all(rnd(15, total, dt=dt), idx, rows, n, d, dt, f"{total} of {rows}x{n}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shape", ["one row", "one latent", "every fourth row", "last place"])
def test_uneven(shape, dt):
    rows, n, d = 200, 6000, 48
    if shape == "one row":
        idx = 37 * n + torch.randperm(n, generator=torch.Generator().manual_seed(4))[:5900].cuda()
    elif shape == "one latent":
        idx = torch.randperm(rows, generator=torch.Generator().manual_seed(5)).cuda() * n + 4321
    elif shape == "every fourth row":
        idx = ints(6, rows // 4, 7000) * 4 * n + ints(7, n, 7000)
    else:
        idx = torch.tensor([rows * n - 1]).cuda()
    check_all(rnd(8, idx.numel(), dt=dt), idx, rows, n, d, dt, shape)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("total", [300, 9000])
def test_padded_and_out_of_range_and_repeated(total, dt):
    rows, n, d = 40, 500, 72
    idx = ints(9, rows * n, total)
    idx[100:120] = idx[:20]              # places that occur twice
    idx[-30:] = -1
    idx[50], idx[60], idx[70] = rows * n, -7, 2 ** 62
    v = rnd(10, total, dt=dt)
    v[-30:] = -math.inf
    check_all(v, idx, rows, n, d, dt, f"flat padded {total}")
    idx2 = ints(11, n, rows, total // 30)
    idx2[:, -2:] = -1
    idx2[3] = -1                         # a row with no entry
    idx2[5, 0], idx2[6, 1] = n, 2 ** 40
    v2 = rnd(12, rows, total // 30, dt=dt)
    v2[:, -2:] = -math.inf
    check_all(v2, idx2, rows, n, d, dt, f"row-wise padded {total}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nothing_selected(dt):
    rows, n, d = 30, 20, 24
    for v, idx in ((torch.empty(0), torch.empty(0, dtype=torch.int64)), (torch.ones(5), torch.full((5,), -1)),
                   (torch.ones(rows, 0), torch.empty(rows, 0, dtype=torch.int64))):
        check_all(v.to(DT[dt]).cuda(), idx.cuda(), rows, n, d, dt, "nothing")
    T = tss()
    for r, nn, dd in ((0, 5, 4), (3, 0, 4), (3, 5, 0), (0, 0, 0)):
        v, idx = torch.full((2,), 1.0, dtype=DT[dt]).cuda(), torch.full((2,), -1).cuda()
        w, g = rnd(1, nn, dd, dt=dt), rnd(2, r, dd, dt=dt)
        assert T.decode(v, idx, w, rows=r).shape == (r, dd)
        dv, dw, db = T.decode_grad(g, v, idx, w)
        assert not dv.any() and dw.shape == (nn, dd) and not dw.any() and db.shape == (dd,)
        dx, dw, db = T.encode_grad(v, v, idx, g, w)
        assert dx.shape == (r, dd) and not dx.any() and not dw.any() and db.shape == (nn,) and not db.any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strides_and_alignment(dt):
    T = tss()
    rows, total, n, d = 60, 3000, 200, 128
    idx, v = ints(13, rows * n, total), rnd(14, total, dt=dt)
    base_w, base_g = rnd(15, n, d, dt=dt), rnd(16, rows, d, dt=dt)
    want = T.decode(v, idx, base_w, rows=rows)
    wants = T.decode_grad(base_g, v, idx, base_w)
    wante = T.encode_grad(v, v, idx, base_g, base_w)

    def odd(t):
        big = torch.full((t.shape[0], t.shape[1] + 3), 9.0, dtype=t.dtype, device="cuda")
        big[:, 1:1 + t.shape[1]] = t
        return big[:, 1:1 + t.shape[1]]

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    for form in (odd, shifted, lambda t: t.t().contiguous().t(), lambda t: t.repeat_interleave(2, 0)[::2]):
        w, g = form(base_w), form(base_g)
        close = [(want, T.decode(v, idx, w, rows=rows))] + list(zip(wants, T.decode_grad(g, v, idx, w)))
        close += list(zip(wante, T.encode_grad(shifted(v[None])[0], shifted(v[None])[0], idx, g, w)))
        for a, b in close:   # sums of at most 60 entries or 128 columns, in another order at most
            scale = a.double().abs().max() + 30
            assert float((a.double() - b.double()).abs().max()) <= float(scale) * (140 * U.U32 + 2 * U.half_step(a.dtype))


def test_autograd_against_differences():
    T = tss()
    rows, n, d, total = 7, 12, 10, 25
    idx = torch.randperm(rows * n, generator=torch.Generator().manual_seed(17))[:total].cuda()
    v, w, b, c = rnd(18, total), rnd(19, n, d), rnd(20, d), rnd(21, rows, d)
    for t in (v, w, b):
        t.requires_grad_(True)
    grads = torch.autograd.grad((T.decode(v, idx, w, rows=rows, bias=b) * c).sum(), (v, w, b))
    dense = lambda vv, ww, bb: float(((torch.zeros(rows * n, dtype=torch.float64, device="cuda").index_add(0, idx, vv)  # noqa: E731
                                       .view(rows, n) @ ww + bb) * c.double()).sum())
    base = [t.detach().double() for t in (v, w, b)]
    for i, g in enumerate(grads):
        way = rnd(22 + i, *base[i].shape).double()
        ends = []
        for s in (1e-4, -1e-4):
            at = list(base)
            at[i] = at[i] + s * way
            ends.append(dense(*at))
        want = (ends[0] - ends[1]) / 2e-4     # linear in each argument: exact but for 64-bit rounding
        scale = float((g.double() * way).abs().sum())
        assert abs(float((g.double() * way).sum()) - want) <= 100 * U.U32 * scale + 1e-9


def test_encode_is_the_selection_of_the_product_and_differentiates():
    T = tss()
    rows, d, n, k = 64, 48, 500, 2000
    x, w, b = rnd(23, rows, d), rnd(24, n, d, scale=0.2), rnd(25, n, scale=0.1)
    acts = T.linear(x, w, b, activation="relu")
    want = T.topk(acts.reshape(1, -1), k)
    for t in (x, w, b):
        t.requires_grad_(True)
    v, idx = T.encode(x, w, b, k)
    assert torch.equal(v, want[0][0]) and torch.equal(idx, want[1][0]) and not idx.requires_grad
    gv = rnd(26, k)
    got = torch.autograd.grad((v * gv).sum(), (x, w, b))
    for a, c in zip(got, T.encode_grad(gv, v.detach(), idx, x.detach(), w.detach())):
        assert torch.equal(a, c)
    # the same through the dense activation in 64 bits
    z = x.detach().double().requires_grad_(True)
    ww, bb = w.detach().double().requires_grad_(True), b.detach().double().requires_grad_(True)
    dense = torch.relu(z @ ww.t() + bb).reshape(-1)[idx]
    for a, c in zip(got, torch.autograd.grad((dense * gv.double()).sum(), (z, ww, bb))):
        assert float((a.double() - c).abs().max()) <= 1e-4 * float(c.abs().max())


def test_encode_with_fewer_positive_than_selected_and_relaxed_recall():
    T = tss()
    x, w = rnd(27, 16, 24), rnd(28, 40, 24)
    v, idx = T.encode(x, w, None, 640)     # every place: half of them are 0 after relu
    dx, dw, db = T.encode_grad(torch.ones_like(v), v, idx, x, w)
    mask = (x.double() @ w.double().t() > 0).double()
    assert float((dx.double() - mask @ w.double()).abs().max()) < 1e-4
    assert torch.equal(db.double(), mask.sum(0))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("total", [400, 9000])
def test_graphs_streams_and_repeats(total, dt):
    T = tss()
    rows, n, d = 90, 300, 72
    idx, v, gv = ints(29, rows * n, total), rnd(30, total, dt=dt), rnd(31, total, dt=dt)
    w, g = rnd(32, n, d, dt=dt), rnd(33, rows, d, dt=dt)

    def step():
        return (T.decode(v, idx, w, rows=rows),) + T.decode_grad(g, v, idx, w) + T.encode_grad(gv, v, idx, g, w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(warm, step()):
        assert torch.equal(a, b)
    graphs = []
    for _ in range(2):
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            out = step()
        graphs.append((cg, out))
    for i in range(3):
        idx.copy_(ints(40 + i, rows * n, total))
        v.copy_(rnd(50 + i, total, dt=dt))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):       # the two graphs side by side
            graphs[1][0].replay()
        graphs[0][0].replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for _, out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,n,d", [(1, 257, 3000, 512), (1, 40_000, 5000, 20), (5, 700, 900, 1), (7, 1030, 300, 3), (3, 2048, 8192, 1028),
                                        (40, 5000, 70, 65), (2047, 600, 50, 8), (2049, 300, 50, 8)])
def test_few_rows_of_many_entries(rows, k, n, d, dt):
    idx = ints(31, n, rows, k)
    idx[:, -3:] = -1
    if rows > 2:
        idx[1] = -1                      # a row with no entry, a row with one part without any
        idx[2, :300] = n
    check_all(rnd(32, rows, k, dt=dt), idx, rows, n, d, dt, f"row-wise {rows}x{k} of {n}, {d} wide")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,total,n,d", [(1, 8192, 9000, 40), (3, 8191, 70, 520), (64, 2000, 300, 5), (900, 6000, 8, 65)])
def test_short_flattened_selections_in_parts(rows, total, n, d, dt):
    idx = ints(33, rows * n, total)
    idx[::5] = idx[0]
    check_all(rnd(34, total, dt=dt), idx, rows, n, d, dt, f"flat {total} of {rows}x{n}, {d} wide")
