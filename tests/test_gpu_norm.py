"""The global norm of many tensors and their clipping, against 64 bits: many
tensors, ragged and empty ones, views at odd addresses, mixed types, extreme
and non-finite values, graphs."""
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


def norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def check(ts, max_norm, eps=1e-6):
    want = norm64(ts)
    before = [t.clone() for t in ts]
    got = tss().clip_grad_norm(ts, max_norm, eps)
    assert got.shape == () and got.dtype == torch.float32
    # 64-bit sums, one square root and one rounding to 32 bits
    assert abs(float(got) - want) <= 2 * U.U32 * want
    f = min(1.0, max_norm / (want + eps)) if want + eps else 1.0
    for a, b in zip(ts, before):
        if f == 1.0:
            assert torch.equal(a, b)
        else:   # the factor: a rounded norm, a sum and a quotient; then one product
            U.within(a, b.double() * f, b.double().abs() * f * 6 * U.U32, "scaled")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", [[1], [7], [16384], [16385], [5, 0, 300], [100000], [3, 4096, 4097, 1, 0, 65536],
                                   [1000003, 17]])
def test_sizes(sizes, dt):
    ts = [rnd(i, s, dt=dt, scale=1 + i) for i, s in enumerate(sizes)]
    check(ts, 0.5)
    check([rnd(i, s, dt=dt, scale=1e-3) for i, s in enumerate(sizes)], 1e4)


def test_many_tensors_and_mixed_types():
    ts = [rnd(i, 1 + (i * 37) % 900, dt="bf16" if i % 3 else "f32") for i in range(401)]
    check(ts, 1.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_views_of_one_bucket(dt):
    flat = rnd(1, 70000, dt=dt)
    edge = flat.clone()
    sizes = [1, 2, 3, 5, 8, 13, 40001, 7, 9, 64, 65, 1000]
    views = list(flat[3:3 + sum(sizes)].split(sizes))
    check(views, 0.3)
    assert torch.equal(flat[:3], edge[:3]) and torch.equal(flat[3 + sum(sizes):], edge[3 + sum(sizes):])


def test_orders_of_axes_and_refusals():
    T = tss()
    t = rnd(2, 40, 50).t()
    check([t, rnd(3, 4, 5, 6).permute(2, 0, 1)], 0.1)
    with pytest.raises(ValueError):
        T.clip_grad_norm([rnd(4, 10, 10)[:, :5]], 1.0)
    with pytest.raises(ValueError):
        T.clip_grad_norm([rnd(4, 10, 1).expand(10, 3)], 1.0)
    a = rnd(5, 100)
    keep = a.clone()
    for twice in ([a, a], [a, a[50:]], [a[:51], a[50:]]):
        with pytest.raises(T.TopkError):
            T.clip_grad_norm(twice, 1e-3)
    assert torch.equal(a, keep)
    assert abs(float(T.grad_norm([a, a])) - math.sqrt(2) * norm64([a])) < 1e-4
    for bad in (-1.0, math.nan):
        with pytest.raises(T.TopkError):
            T.clip_grad_norm([a], bad)
    with pytest.raises(TypeError):
        T.grad_norm([a.half()])
    with pytest.raises(ValueError):
        T.grad_norm([a, a.cpu()])


def test_nothing_and_zeros():
    T = tss()
    assert float(T.clip_grad_norm([], 1.0)) == 0.0
    assert float(T.clip_grad_norm([torch.empty(0, device="cuda"), None], 1.0)) == 0.0
    z = torch.zeros(1000, device="cuda")
    for eps in (1e-6, 0.0):
        assert float(T.clip_grad_norm([z], 0.0, eps)) == 0.0
        assert not z.any()
    assert float(T.grad_norm(rnd(6, 3).mul_(0).add_(2.0))) == pytest.approx(math.sqrt(12), rel=1e-6)


def test_extremes_and_non_finite():
    T = tss()
    big = torch.full((1000,), 1e30, device="cuda")
    check([big], 1.0)
    tiny = torch.full((1000,), 1e-30, device="cuda")
    assert abs(float(T.grad_norm([tiny])) / (1e-30 * math.sqrt(1000)) - 1) < 1e-6
    a = rnd(7, 100)
    a[3] = math.inf
    b = a.clone()
    assert float(T.clip_grad_norm([b], 1.0)) == math.inf
    assert torch.isnan(b[3]) and not b[:3].any() and not b[4:].any()
    a[4] = math.nan
    n = T.clip_grad_norm([a], 1.0)
    assert torch.isnan(n) and bool(torch.isnan(a).all())
    c = rnd(8, 50)
    keep = c.clone()
    T.clip_grad_norm([c], math.inf)
    assert torch.equal(c, keep)


def test_version_counter_and_gradients_of_parameters():
    p = torch.nn.Parameter(rnd(9, 30, 20))
    (p * 3).sum().backward()
    v = p.grad._version
    n = tss().clip_grad_norm([p.grad], 1.0)
    assert p.grad._version > v
    assert float(n) == pytest.approx(3 * math.sqrt(600), rel=1e-6)


def test_graph_replays_and_streams():
    T = tss()
    ts = [rnd(i, s, dt=d) for i, (s, d) in enumerate([(70000, "f32"), (33, "bf16"), (4097, "bf16")])]
    src = [t.clone() for t in ts]
    g = torch.cuda.CUDAGraph()
    T.clip_grad_norm([t.clone() for t in ts], 0.7)
    with torch.cuda.graph(g):
        out = T.clip_grad_norm(ts, 0.7)
    side = torch.cuda.Stream()
    for i in range(3):
        for t, s in zip(ts, src):
            t.copy_(s * (i + 1))
        g.replay()
        mine = [s * (i + 1) for s in src]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want = T.clip_grad_norm(mine, 0.7)
        torch.cuda.synchronize()
        assert float(out) == float(want)
        for a, b in zip(ts, mine):
            assert torch.equal(a, b)
