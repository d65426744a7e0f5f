"""Tokens sorted by expert and back, and the gradients, against plain forms:
few and many entries and experts, dropped and out-of-range ones, one expert
with everything, widths around the vectors, strides and alignment, places that
occur twice, weights of either type, streams and graphs."""
import pytest

import model_util as M
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


def ints(seed, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=torch.Generator().manual_seed(seed)).cuda()


def check_dispatch(x, experts, count, label):
    got = tss().dispatch(x, experts, count)
    for g, w, what in zip(got, M.dispatch64(x, experts, count), ("rows", "places", "offsets")):
        assert g.shape == w.shape, (label, what)
        assert torch.equal(g.cpu(), w), (label, what)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("t,k,count", [(0, 2, 4), (0, 3, 8192), (0, 0, 2000), (5, 0, 1500), (1, 1, 1), (3, 0, 5), (1, 8, 8), (7, 2, 3), (64, 1, 64), (100, 6, 257), (512, 8, 1024),
                                       (513, 8, 7), (4096, 1, 1025), (3, 2, 8192), (2500, 4, 8192), (40000, 2, 16), (5000, 3, 63)])
def test_dispatch_counts(t, k, count, dt):
    check_dispatch(rnd(t, t, 24, dt=dt), ints(k, -1, count + 1, t, k), count, (t, k, count))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [0, 1, 3, 4, 5, 7, 8, 9, 64, 515, 1024, 2049])
@pytest.mark.parametrize("t", [9, 3000])
def test_dispatch_widths(t, d, dt):
    x = rnd(d, t, d, dt=dt)
    e = ints(d + 1, -1, 12, t, 2)
    check_dispatch(x, e, 12, (t, d))
    wide = torch.zeros(t, d + 3, dtype=DT[dt], device="cuda")
    wide[:, 1:1 + d] = x
    check_dispatch(wide[:, 1:1 + d], e, 12, (t, d, "rows apart and unaligned"))
    check_dispatch(x.t().contiguous().t(), e, 12, (t, d, "columns"))


def test_dispatch_extremes():
    x = rnd(1, 3000, 16)
    for e in (torch.full((3000, 2), -1), torch.full((3000, 2), 5), torch.full((3000, 2), 2 ** 62), torch.full((3000, 2), -2 ** 63),
              torch.arange(6000).reshape(3000, 2) % 6):
        check_dispatch(x, e.cuda(), 6, "extremes")
        check_dispatch(x[:100], e[:100].cuda(), 6, "extremes of few")
    check_dispatch(x, torch.zeros(3000, 2, dtype=torch.int64, device="cuda"), 0, "no experts")
    same = ints(5, 0, 6, 3000, 1).expand(3000, 4)      # the same expert four times
    check_dispatch(x, same, 6, "an expert twice")


def test_dispatch_keeps_bits():
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).reshape(256, 256).cuda()
    e = ints(3, 0, 9, 256, 2)
    rows, places, _ = tss().dispatch(bits.view(torch.bfloat16), e, 9)
    assert torch.equal(rows.view(torch.int16)[places[:, 1]], bits)


def check_combine(y, places, w, label):
    out, err = M.combine64(y, places, w)
    U.within(tss().combine(y, places, w).cpu(), out, err, label)


@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("bf16", None), ("f32", None)])
@pytest.mark.parametrize("t,k,n,d", [(0, 2, 4, 8), (1, 1, 1, 1), (5, 3, 0, 9), (3, 0, 5, 16), (1, 2, 2, 1024), (8, 2, 16, 515), (50, 9, 300, 7),
                                     (40, 17, 100, 8), (1000, 8, 8000, 64), (700, 1, 50, 130), (33, 4, 200, 0)])
def test_combine(t, k, n, d, dt, wdt):
    y = rnd(t, n, d, dt=dt)
    places = ints(k, -2, n + 2, t, k)       # out of range at both ends, many twice
    w = rnd(d, t, k, dt=wdt) if wdt else None
    check_combine(y, places, w, (t, k, n, d))
    g = rnd(7, t, d, dt=dt)
    (dy, dw), (ey, ew) = M.combine_grad64(g, y, places, w)
    for need in ((True, True), (True, False), (False, True)):
        gy, gw = tss().combine_grad(g, y, places, w, need=need)
        assert (gy is not None) == need[0] and (gw is not None) == (need[1] and w is not None)
        if gy is not None:
            U.within(gy.cpu(), dy, ey, "dy")
        if gw is not None:
            U.within(gw.cpu(), dw, ew, "dw")


def test_combine_strides():
    wide = rnd(1, 300, 75, dt="bf16")
    places, w = ints(2, -1, 300, 90, 3), rnd(3, 90, 6)[:, ::2]
    check_combine(wide[:, 3:70], places, w, "rows apart")
    check_combine(rnd(4, 67, 300).t(), places, w, "columns")
    check_combine(rnd(4, 1, 67).expand(300, 67), places, w, "one row for all")
    g = rnd(5, 1, 1, dt="bf16").expand(90, 67)      # as the gradient of a sum comes
    (dy, dw), (ey, ew) = M.combine_grad64(g, wide[:, 3:70], places, w)
    gy, gw = tss().combine_grad(g, wide[:, 3:70], places, w)
    U.within(gy.cpu(), dy, ey, "dy")
    U.within(gw.cpu(), dw, ew, "dw")


def test_infinities_stay_where_they_are():
    # a dropped place adds nothing, whatever the weight or the rows hold
    y = rnd(1, 8, 16)
    y[5] = float("nan")
    places = torch.tensor([[0, -1], [1, 9], [-1, -1]]).cuda()
    w = torch.tensor([[1.0, float("inf")], [2.0, float("nan")], [float("inf"), 1.0]]).cuda()
    out = tss().combine(y, places, w)
    assert torch.equal(out, torch.stack([y[0], 2 * y[1], torch.zeros_like(y[0])]))
    dy, dw = tss().combine_grad(torch.ones(3, 16, device="cuda"), y, places, w)
    assert bool(torch.isfinite(dy).all()) and bool((dy[2:] == 0).all()) and bool((dw[:, 1] == 0).all()) and float(dw[2, 0]) == 0


def test_many_entries_at_one_place():
    places = torch.zeros(500, 3, dtype=torch.int64, device="cuda")
    y, w, g = rnd(1, 4, 40), rnd(2, 500, 3), rnd(3, 500, 40)
    (dy, _), (ey, _) = M.combine_grad64(g, y, places, w)
    first, _ = tss().combine_grad(g, y, places, w)
    U.within(first.cpu(), dy, ey, "dy")
    for _ in range(5):     # in whatever order the entries came
        assert torch.equal(tss().combine_grad(g, y, places, w)[0], first)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_very_many_entries_at_few_places(dt):
    # linear in the entries, however they crowd; more of them than one launch maps
    t, k, d = 40000, 3, 20
    places = ints(1, 0, 5, t, k)
    places[:1000] = ints(2, 0, 900, 1000, k)
    y, w, g = rnd(3, 1000, d, dt=dt), rnd(4, t, k), rnd(5, t, d, dt=dt)
    (dy, dw), (ey, ew) = M.combine_grad64(g, y, places, w)
    gy, gw = tss().combine_grad(g, y, places, w)
    U.within(gy.cpu(), dy, ey, "dy")
    U.within(gw.cpu(), dw, ew, "dw")
    assert torch.equal(tss().combine_grad(g, y, places, w)[0], gy)


def test_chains_of_extremes():
    inf, nan, big = float("inf"), float("nan"), 3e38
    places = torch.zeros(4, 1, dtype=torch.int64, device="cuda")
    g = torch.tensor([[1.0, big, inf, inf, nan, 1e-45, 0.0, big], [1.0, big, 1.0, -inf, 1.0, 1e-45, 0.0, -big],
                      [1e-20, -big, 1.0, 1.0, 1.0, 1e-45, -0.0, big], [-2.0, -big, 1.0, 1.0, 1.0, -1e-45, 0.0, -big]], device="cuda")
    dy, _ = tss().combine_grad(g, torch.zeros(2, 8, device="cuda"), places)
    # terms up to 2 are multiples of 2^-57 (62 bits, less 3 for up to 7 terms and 2 for the largest): four roundings
    assert abs(float(dy[0, 0]) - 1e-20) <= 4 * 2.0 ** -58
    assert dy[0, 1:3].tolist() == [0.0, inf] and bool(torch.isnan(dy[0, 3:5]).all())
    assert float(dy[0, 5]) == float(torch.tensor(1e-45) * 2) and dy[0, 6:].tolist() == [0.0, 0.0] and bool((dy[1] == 0).all())


@pytest.mark.parametrize("t", [40, 3000])
def test_gradients(t):
    T = tss()
    x, e = rnd(1, t, 20).requires_grad_(), ints(2, -1, 9, t, 3)
    w = rnd(3, t, 3).requires_grad_()
    rows, places, offsets = T.dispatch(x, e, 9)
    assert not places.requires_grad and not offsets.requires_grad
    y = rows * rows
    T.combine(y, places, w).square().sum().backward()
    # the same in 64 bits, through torch
    x64, w64 = x.detach().cpu().double().requires_grad_(), w.detach().cpu().double().requires_grad_()
    good = (e.cpu() >= 0).double()
    out = (x64.square()[:, None] * (w64 * good)[..., None]).sum(1)
    out.square().sum().backward()
    # |values| here are below 300 and every one comes from fewer than 60 operations of 32 bits
    for got, want in ((x.grad, x64.grad), (w.grad, w64.grad)):
        assert float((got.cpu().double() - want).abs().max()) <= 60 * U.U32 * float(want.abs().max())


def test_gradients_against_differences():
    T = tss()
    e = ints(1, -1, 5, 6, 2)
    x, w, g = rnd(2, 6, 8), rnd(3, 6, 2), rnd(4, 6, 8)

    def loss(x, w):
        rows, places, _ = T.dispatch(x, e, 5)
        return float((T.combine(rows, places, w).double() * g.double()).sum())

    xr, wr = x.clone().requires_grad_(), w.clone().requires_grad_()
    rows, places, _ = T.dispatch(xr, e, 5)
    (T.combine(rows, places, wr) * g).sum().backward()
    # linear in each: a difference over a whole step is the slope, but for 32-bit roundings of sums below 100
    for t, grad, at in ((x, xr.grad, (3, 5)), (x, xr.grad, (0, 0)), (w, wr.grad, (2, 1)), (w, wr.grad, (5, 0))):
        step = t.clone()
        step[at] += 1.0
        diff = (loss(step, w) if t is x else loss(x, step)) - loss(x, w)
        assert abs(diff - float(grad[at])) <= 1e-3


def test_gradient_needs_and_refusals():
    T = tss()
    x, e = rnd(1, 6, 8), ints(2, 0, 4, 6, 2)
    rows, places, _ = T.dispatch(x, e, 4)
    w = rnd(3, 6, 2).requires_grad_()
    T.combine(rows, places, w).sum().backward()
    assert w.grad is not None
    with pytest.raises(ValueError):
        T.dispatch(x, e[:5], 4)
    with pytest.raises(ValueError):
        T.dispatch(x, e.int(), 4)
    with pytest.raises(ValueError):
        T.dispatch(x, e, 8193)
    with pytest.raises(ValueError):
        T.dispatch(x, e, -1)
    with pytest.raises(TypeError):
        T.dispatch(x.half(), e, 4)
    with pytest.raises(ValueError):
        T.dispatch(x[0], e, 4)
    with pytest.raises(ValueError):
        T.combine(rows, places, w.detach()[:5])
    with pytest.raises(ValueError):
        T.combine(rows, places, w.detach().bfloat16())     # rows of float32 take weights of float32
    with pytest.raises(ValueError):
        T.combine(rows, places.int())
    with pytest.raises(ValueError):
        T.combine_grad(x[:, :4], rows, places, w.detach())
    with pytest.raises(ValueError):
        T.combine_grad(x, rows, places, w.detach(), need=(True,))
    assert T.combine_grad(x, rows, places, None, need=(False, True)) == (None, None)
    from torch.autograd import forward_ad as F
    with F.dual_level():
        for f in (lambda: T.dispatch(F.make_dual(x, x), e, 4), lambda: T.combine(F.make_dual(rows, rows), places),
                  lambda: T.combine_grad(F.make_dual(x, x), rows, places)):
            with pytest.raises(RuntimeError, match="forward-mode"):
                f()


def test_graph_and_stream():
    T = tss()
    for t in (20, 4000):
        x, e, w, g = rnd(1, t, 72, dt="bf16"), ints(2, -1, 17, t, 4), rnd(3, t, 4), rnd(4, t, 72, dt="bf16")

        def step():
            rows, places, offsets = T.dispatch(x, e, 17)
            out = T.combine(rows, places, w)
            dy, dw = T.combine_grad(g, rows, places, w)
            return rows, places, offsets, out, dy, dw, T.combine(dy, places)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
        for i in range(4):
            x.copy_(rnd(10 + i, t, 72, dt="bf16"))
            e.copy_(ints(20 + i, -1, 17, t, 4))
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(held, step()):
                assert torch.equal(a, b)
        xr = x.float().requires_grad_()
        with pytest.raises(RuntimeError, match="capture"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                T.dispatch(xr, e, 17)
