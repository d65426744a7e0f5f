"""The next token against 64 bits, token for token: lengths around the chunks,
every setting as a number and as a tensor, rows whose mask leaves nothing or
one token, equal logits on the cut, infinities and NaN, numbers at the ends of
[0, 1), strides, streams and graphs."""
import math

import pytest

import model_util as M
import ops_util as U

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LAST = 1 - 2.0 ** -24     # the largest float32 below 1


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


def uni(seed, rows):
    return torch.rand(rows, generator=torch.Generator().manual_seed(seed)).cuda()


def at(v, r):
    return v[r].item() if isinstance(v, torch.Tensor) else v


def check(z, u, label="", temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    token, logprob = tss().sample(z, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    rows = z.shape[0]
    assert token.dtype == torch.int64 and logprob.dtype == torch.float32 and token.shape == logprob.shape == (rows,)
    zc, uc = z.cpu(), u.tolist()
    want, prob = [], []
    for r in range(rows):
        t, p = M.sample64(zc[r], uc[r], M.f32(at(temperature, r)), int(at(top_k, r)), M.f32(at(top_p, r)), M.f32(at(min_p, r)))
        want.append(t)
        prob.append(p)
    assert token.tolist() == want, label
    U.within(logprob.cpu(), torch.tensor(prob, dtype=torch.float64), torch.full((rows,), 1e-9, dtype=torch.float64), label)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 3, 63, 64, 65, 255, 1000, 1024, 1025, 4097, 30011])
def test_lengths(n, dt):
    z = rnd(n, 3, n, dt=dt, scale=2.0)
    for i, kw in enumerate((dict(), dict(top_k=5), dict(top_p=0.7), dict(min_p=0.1), dict(top_k=40, top_p=0.9, min_p=0.01, temperature=0.7),
                            dict(top_k=max(1, n // 2), top_p=0.5), dict(temperature=0.0), dict(top_k=1), dict(top_p=0.0), dict(min_p=1.0))):
        check(z, uni(i, 3), (n, kw), **kw)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 40])
def test_settings_of_each_row(rows, dt):
    z = rnd(rows, rows, 3001, dt=dt, scale=3.0)
    g = torch.Generator().manual_seed(rows)
    t = torch.rand(rows, generator=g).mul(2).cuda()
    t[0] = 0
    k = torch.randint(-1, 4000, (rows,), generator=g).cuda()
    p = torch.rand(rows, generator=g).mul(1.2).cuda()
    m = torch.rand(rows, generator=g).mul(0.2).cuda()
    check(z, uni(1, rows), "all", temperature=t, top_k=k, top_p=p, min_p=m)
    check(z, uni(2, rows), "temperature", temperature=t, top_k=7)
    check(z, uni(3, rows), "top_k", top_k=k)
    check(z, uni(4, rows), "top_p", top_p=p)
    check(z, uni(5, rows), "min_p", min_p=m)


def test_long_rows():
    for dt, n, seed in (("f32", 200003, 1), ("bf16", 131072, 2), ("bf16", 400001, 3)):
        z = rnd(seed, 2, n, dt=dt, scale=2.0)
        for i, kw in enumerate((dict(), dict(top_k=50, top_p=0.95), dict(top_p=0.9), dict(top_k=n // 4, top_p=0.3), dict(top_k=n // 3),
                                dict(top_p=0.999, temperature=1.5))):
            check(z, uni(seed * 10 + i, 2), (n, kw), **kw)


def test_longest_row():
    n = 1 << 24
    z = torch.full((1, n), -3.0, dtype=torch.bfloat16, device="cuda")
    z[0, n - 5] = 2.0
    # weights 1 and n - 1 times e^-5: every border is known
    w = math.exp(-5.0)
    total = 1 + (n - 1) * w
    for u in (0.0, 0.25, 0.5, LAST):
        token, logprob = tss().sample(z, torch.tensor([u], device="cuda"))
        want = min(int(u * total / w), n - 1)
        if want >= n - 5:     # behind the heavy token the borders lie 1 - w further
            want = n - 5 if u * total < (n - 5) * w + 1 else int((u * total - 1) / w) + 1
        assert abs(int(token) - want) <= 1
        assert abs(float(logprob) - math.log((1 if int(token) == n - 5 else w) / total)) <= 1e-5
    assert int(tss().sample(z, torch.tensor([0.5], device="cuda"), top_k=1)[0]) == n - 5
    # all but one equal: the cut by index
    assert int(tss().sample(z, torch.tensor([LAST], device="cuda"), top_k=1001, temperature=100.0)[0]) == n - 5
    z[0, n - 5] = -3.0
    assert int(tss().sample(z, torch.tensor([LAST], device="cuda"), top_k=1001)[0]) == 1000
    assert int(tss().sample(z, torch.tensor([LAST], device="cuda"), top_p=0.25)[0]) == n // 4 - 1


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_equal_logits(dt):
    # more equal ones on the cut than are sorted (4096), and borders that are exact
    for n in (8, 1000, 4096, 4097, 20000):
        z = torch.full((9, n), 0.5, dtype=DT[dt], device="cuda")
        u = torch.tensor([0.0, 0.125, 0.25, 0.5, 0.75, 0.875, LAST, 0.3, 0.999], device="cuda")
        for kw in (dict(), dict(top_k=n // 2), dict(top_p=0.5), dict(top_k=3 * n // 4, top_p=0.25), dict(top_p=0.7, min_p=1.0)):
            check(z, u, (n, kw), **kw)
    z = (torch.arange(30000) % 3).to(DT[dt]).expand(4, 30000).contiguous().cuda()
    for kw in (dict(top_k=15000), dict(top_p=0.8), dict(top_k=25000, top_p=0.95), dict(top_k=10000), dict(top_k=10001), dict(top_k=12000, top_p=0.9999)):
        check(z, uni(3, 4), kw, **kw)


@pytest.mark.parametrize("n", [65535, 65536, 65537, 131072])
def test_equal_logits_by_index(n):
    # of equal logits the lowest indices stay: the last of them is the largest number's token
    z = torch.zeros(1, n, device="cuda")
    u = torch.tensor([LAST], device="cuda")
    for k in (5000, 32768, n - 1, n):
        assert int(tss().sample(z, u, top_k=k)[0]) == k - 1, k
    for p in (0.25, 0.5, 0.75):
        assert int(tss().sample(z, u, top_p=p)[0]) == math.ceil(p * n) - 1, p
    assert int(tss().sample(z, u, top_k=40000, top_p=0.5)[0]) == 19999


def test_cut_in_two_places():
    # the k-th and the nucleus' end are many bins apart, with too many entries between to sort them all
    z = rnd(1, 3, 60000, scale=1.0)
    for kw in (dict(top_k=40000, top_p=0.3), dict(top_k=30000, top_p=0.05), dict(top_k=59999, top_p=0.6), dict(top_k=20000, top_p=0.99)):
        check(z, uni(4, 3), kw, **kw)


def test_cut_inside_the_first_logits():
    # the nucleus ends among a few logits next to the largest, the k-th is far behind, and most of what p counts lies between
    z = rnd(2, 4, 60000, scale=0.5) - 3.0
    z[:, 100:105] = torch.tensor([5.0, 4.9999, 4.9998, 4.9997, 4.9996])
    z[1:3, 7] = 4.99985
    for k in (40000, 59000, 0):
        for p in (0.02, 0.05, 0.08, 0.1):
            check(z, uni(5, 4), (k, p), top_k=k, top_p=p)
    check(z[:, :3000].contiguous(), uni(6, 4), "short", top_k=2000, top_p=0.5)


@pytest.mark.parametrize("n", [511, 512, 513, 700, 2000, 4096, 6143, 6144, 20000])
def test_limits_of_the_ways(n):
    # k around those at which another way is taken, with and without top_p
    z = rnd(n, 2, n, scale=1.5)
    for k in sorted({3 * n // 64, 3 * n // 64 + 1, n // 64, n // 64 + 1, 384, 385, 512, 513, n - 1}):
        if 0 < k <= n:
            check(z, uni(k, 2), (n, k), top_k=k)
            check(z, uni(k + 1, 2), (n, k, "p"), top_k=k, top_p=0.9)
    for p in (0.3, 0.9, 0.99):
        check(z, uni(n, 2), (n, p), top_p=p)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(), dict(top_k=3), dict(top_p=0.9), dict(top_k=2, top_p=0.5, min_p=0.1), dict(temperature=0.0)])
def test_masks(dt, kw):
    inf, nan, low = math.inf, math.nan, torch.finfo(DT[dt]).min
    z = rnd(5, 10, 3000, dt=dt)
    z[0] = -inf
    z[1] = -inf
    z[1, 2999] = -5.0
    z[2] = low
    z[3] = low
    z[3, 7] = 1.0
    z[4, ::2] = nan
    z[5] = nan
    z[6, 10] = z[6, 2000] = z[6, 2500] = inf
    z[7, :] = -inf
    z[7, 5:9] = torch.tensor([-0.0, 0.0, -0.0, 0.0])
    z[8] = torch.finfo(DT[dt]).max
    z[9, 1:] = -inf
    check(z, uni(6, 10), kw, **kw)
    check(z, torch.full((10,), LAST).cuda(), kw, **kw)
    check(z, torch.zeros(10).cuda(), kw, **kw)


def test_extreme_settings():
    z = rnd(7, 4, 5000, scale=4.0)
    u = uni(8, 4)
    for t in (1e-30, 1e-44, 1e-3, 1e3, 1e30, math.inf):
        for kw in (dict(), dict(top_p=0.5), dict(top_k=100)):
            check(z, u, (t, kw), temperature=t, **kw)
    for p in (1e-45, 1e-38, 1e-10, 1 - 2.0 ** -24, 0.5):
        check(z, u, p, top_p=p)
    for k in (4999, 5000, 5001, 2 ** 40):
        check(z, u, k, top_k=k)
    got = tss().sample(z, torch.tensor([-1.0, 1.0, math.nan, 7.0], device="cuda"), top_k=6)   # outside [0, 1): the ends
    ends = [tss().sample(z, torch.full((4,), v, device="cuda"), top_k=6) for v in (0.0, LAST)]
    assert got[0].tolist() == [ends[0][0][0], ends[1][0][1], ends[1][0][2], ends[1][0][3]]
    nan = torch.full((4,), math.nan, device="cuda")
    assert tss().sample(z, u, temperature=nan)[0].tolist() == z.argmax(1).tolist()
    assert tss().sample(z, u, top_p=nan)[0].tolist() == z.argmax(1).tolist()
    assert tss().sample(z, u, min_p=nan)[0].tolist() == [-1] * 4


def test_settings_are_float32():
    # a number counts as the float32 next to it, also for what the call's scratch memory is sized by
    z = rnd(13, 3, 1501, scale=2.0)
    u = uni(14, 3)
    check(z, u, "as 1", top_p=1 - 1e-12)
    check(z, u, "below 1", top_p=0.8)
    check(z, u, "as 0", temperature=1e-50)
    check(z, u, "above 0", temperature=0.9)
    check(z, u, "as inf", temperature=1e39)
    check(z, u, "as 0, of everything", min_p=1e-60)


def test_distribution():
    # the shares of 2^16 evenly spaced numbers are the probabilities, to one of them
    z = torch.tensor([[0.5, -1.0, 2.0, 0.0, 1.0, -3.0]], device="cuda")
    rows = 1 << 16
    u = (torch.arange(rows, device="cuda") / rows).float()
    token, logprob = tss().sample(z.expand(rows, 6), u, temperature=0.7)
    p = torch.softmax(z[0].double() / M.f32(0.7), 0)
    share = torch.bincount(token, minlength=6).double() / rows
    assert float((share - p).abs().max()) <= 1.01 / rows
    assert torch.equal(logprob.exp() > 0, torch.ones(rows, dtype=torch.bool, device="cuda"))


def test_rows_do_not_depend_on_their_batch():
    z = rnd(9, 600, 2500, scale=2.0)
    u = uni(10, 600)
    whole = tss().sample(z, u, top_k=60, top_p=0.9)
    for r in (0, 17, 599):
        one = tss().sample(z[r], u[r], top_k=60, top_p=0.9)
        assert one[0].dim() == 0 and int(one[0]) == int(whole[0][r]) and float(one[1]) == float(whole[1][r])
    many = tss().sample(z[:, :40], u, top_p=0.5)
    check(z[:50, :40], u[:50], "rows apart", top_p=0.5)
    assert int(many[0].max()) < 40
    big = tss().sample(z[0:1, :16].expand(70000, 16), u[0:1].expand(70000), top_k=4)
    assert bool((big[0] == big[0][0]).all())


def test_layouts():
    z = rnd(11, 6, 2003, dt="bf16", scale=2.0)
    wide = torch.zeros(6, 2010, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:2006] = z
    check(wide[:, 3:2006], uni(12, 6), "unaligned", top_p=0.9)
    check(z.t().contiguous().t(), uni(12, 6), "columns", top_p=0.9)
    check(z, uni(12, 12)[::2], "every other number", top_k=9)
    empty = tss().sample(z[:0], uni(1, 0))
    assert empty[0].shape == (0,) and empty[1].shape == (0,)


def test_refusals():
    T, z, u = tss(), rnd(1, 4, 10), uni(2, 4)
    for kw in (dict(temperature=-1.0), dict(temperature=math.nan), dict(top_k=-1), dict(top_k=1.5), dict(top_p=-0.1), dict(top_p=1.1),
               dict(min_p=2.0), dict(min_p=math.nan), dict(top_k=u), dict(top_p=u.double()), dict(temperature=u[:3]), dict(min_p=u.cpu())):
        with pytest.raises(ValueError):
            T.sample(z, u, **kw)
    for bad in (lambda: T.sample(z, u[:3]), lambda: T.sample(z, u.double()), lambda: T.sample(z, u.cpu()), lambda: T.sample(z[:, :0], u),
                lambda: T.sample(z[None], u)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        T.sample(z.half(), u)
    with pytest.raises(RuntimeError, match="no gradient"):
        T.sample(z.clone().requires_grad_(), u)
    with torch.no_grad():
        T.sample(z.clone().requires_grad_(), u)


def test_graph_and_streams():
    T = tss()
    z, u = rnd(1, 5, 9000, scale=2.0), uni(2, 5)
    calls = [dict(top_k=30, top_p=0.9), dict(min_p=0.05), dict(top_p=0.6, temperature=1.2)]

    def step():
        return [t for kw in calls for t in T.sample(z, u, **kw)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        z.copy_(rnd(10 + i, 5, 9000, scale=2.0))
        if i == 2:
            z.fill_(1.0)       # equal logits: the way past the sort
        u.copy_(uni(20 + i, 5))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b)
    want = [t.clone() for t in step()]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append(step())
        torch.cuda.synchronize()
        for g in got:
            assert all(torch.equal(a, b) for a, b in zip(g, want))
