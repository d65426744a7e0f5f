"""Attention over a cache, the weights it adds up, and the cache's eviction,
against 64 bits: lengths from 0, head layouts, widths around the vectors,
rows behind a sequence's end that hold NaN, strides and expanded axes, equal
scores on the cut, buffers that are filled in place, streams and graphs."""
import math

import pytest

import model_util as M
import ops_util as U

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN = float("nan")


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


def ends(*v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def check_attend(q, k, v, lengths=None, scale=None, label="", layout=None):
    b, h, n, _ = k.shape
    out, eo, add, ea = M.attend64(q, k, v, lengths, scale, q.dtype)
    U.within(tss().attend(q, k, v, lengths, scale=scale).cpu(), out, eo, f"{label} out alone")
    before = torch.rand(b, h, n, generator=torch.Generator().manual_seed(1)).cuda()
    scores = before.clone() if layout is None else layout(before)
    U.within(tss().attend(q, k, v, lengths, scores, scale).cpu(), out, eo, f"{label} out")
    U.within(scores.cpu(), before.cpu().double() + add, ea, f"{label} scores")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [1, 3, 4, 7, 8, 9, 20, 63, 64, 65, 80, 96, 97, 128, 130, 192, 200, 256])
def test_attend_widths(d, dt):
    for hq, h, n in ((4, 2, 70), (16, 1, 33)):
        check_attend(rnd(d, 2, hq, d, dt=dt), rnd(d + 1, 2, h, n, d, dt=dt), rnd(d + 2, 2, h, n, d, dt=dt), label=(d, hq, h))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 127, 128, 129, 255, 257, 1000, 5003])
def test_attend_lengths(n, dt):
    check_attend(rnd(n, 3, 6, 40, dt=dt, scale=2.0), rnd(n + 1, 3, 2, n, 40, dt=dt), rnd(n + 2, 3, 2, n, 40, dt=dt), label=n)
    check_attend(rnd(n, 3, 6, 40, dt=dt), rnd(n + 1, 3, 2, n, 40, dt=dt), rnd(n + 2, 3, 2, n, 40, dt=dt), ends(0, n, max(1, n // 2)), label=(n, "ragged"))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("hq,h", [(1, 1), (5, 5), (8, 1), (15, 1), (17, 1), (32, 2), (40, 2), (33, 1), (96, 2), (64, 64)])
def test_attend_heads(hq, h, dt):
    for n in (50, 700):
        check_attend(rnd(hq, 2, hq, 64, dt=dt), rnd(h, 2, h, n, 64, dt=dt), rnd(h + 1, 2, h, n, 64, dt=dt), ends(n, n - 13), label=(hq, h, n))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attend_room_behind_the_end(dt):
    # what lies behind a sequence is never looked at, and its scores stay
    for n, lens in ((300, (0, 1, 17, 130)), (3000, (2999, 5, 0, 1024)), (40, (-3, 41, 2 ** 40, 39))):
        q, k, v = rnd(1, 4, 4, 48, dt=dt), rnd(2, 4, 2, n, 48, dt=dt), rnd(3, 4, 2, n, 48, dt=dt)
        for i, e in enumerate(lens):
            e = max(0, min(n, e))
            k[i, :, e:] = NAN
            v[i, :, e:] = math.inf if i % 2 else NAN
        lengths = ends(*lens)
        out, eo, add, ea = M.attend64(q, k, v, lengths, None, q.dtype)
        scores = torch.full((4, 2, n), 0.5, device="cuda")
        for i, e in enumerate(lens):
            scores[i, :, max(0, min(n, e)):] = NAN
        U.within(tss().attend(q, k, v, lengths, scores).cpu(), out, eo, "out")
        for i, e in enumerate(lens):
            e = max(0, min(n, e))
            U.within(scores[i, :, :e].cpu(), 0.5 + add[i, :, :e], ea[i, :, :e], "scores")
            assert bool(torch.isnan(scores[i, :, e:]).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attend_layouts(dt):
    b, hq, h, n, d = 2, 6, 3, 150, 36
    q, k, v = rnd(1, b, hq, d, dt=dt), rnd(2, b, n, h, d, dt=dt), rnd(3, b, n, h, d, dt=dt)
    check_attend(q, k.transpose(1, 2), v.transpose(1, 2), label="[b, n, h, d]")
    packed = rnd(4, b, n, 2 * h * d + 1, dt=dt)          # keys beside values, rows unaligned
    check_attend(q, packed[..., 1:1 + h * d].unflatten(2, (h, d)).transpose(1, 2), packed[..., 1 + h * d:].unflatten(2, (h, d)).transpose(1, 2), label="packed")
    check_attend(q, k[:, :, :1].transpose(1, 2).expand(b, h, n, d), v[:1, :, :].transpose(1, 2).expand(b, h, n, d), label="expanded")
    check_attend(rnd(5, hq, b, d, dt=dt).transpose(0, 1), rnd(6, b, h, d, n, dt=dt).transpose(2, 3), rnd(7, b, h, d, n, dt=dt).transpose(2, 3), label="columns")

    def heads_first(s):
        t = torch.zeros(h, b, n + 5, device="cuda")[:, :, 3:3 + n].transpose(0, 1)
        t.copy_(s)
        return t
    check_attend(q, k.transpose(1, 2), v.transpose(1, 2), layout=heads_first, label="scores apart")
    check_attend(q, k.transpose(1, 2), v.transpose(1, 2), scale=-0.3, label="scale")
    check_attend(q, k.transpose(1, 2), v.transpose(1, 2), scale=0.0, label="no scale")


def test_attend_large_logits():
    # one entry takes all; the running maximum rises late, and by a lot
    for dt in ("bf16", "f32"):
        k = rnd(1, 1, 1, 3000, 64, dt=dt)
        k[0, 0, 2900] = 30.0
        q = torch.ones(1, 2, 64, dtype=DT[dt], device="cuda")
        v = rnd(2, 1, 1, 3000, 64, dt=dt)
        check_attend(q, k, v, scale=1.0, label="late")
        check_attend(-q, k, v, scale=1.0, label="never")
        scores = torch.zeros(1, 1, 3000, device="cuda")
        out = tss().attend(q, k, v, scores=scores, scale=1.0)
        assert float(scores[0, 0, 2900]) == 2.0 and torch.equal(out[0, 0], v[0, 0, 2900])


def test_attend_not_finite():
    for dt in ("bf16", "f32"):
        q, k, v = rnd(1, 2, 4, 64, dt=dt), rnd(2, 2, 2, 200, 64, dt=dt), rnd(3, 2, 2, 200, 64, dt=dt)
        k[0, 1, 100, 5] = NAN
        v[1, 0, 50, 7] = math.inf
        out = tss().attend(q, k, v)
        assert bool(torch.isnan(out[0, 2:]).all()) and bool(torch.isfinite(out[0, :2]).all())
        assert bool((out[1, :2, 7] == math.inf).all()) and bool(torch.isfinite(out[1, :2, :7]).all()) and bool(torch.isfinite(out[1, 2:]).all())


def test_attend_offsets_beyond_32_bits():
    # a cache of 2^31 elements and more; keys and values are the same rows
    n, d = (1 << 24) + 1000, 128
    kv = torch.empty(1, 1, n, d, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for i in range(0, n, 1 << 20):
        kv[0, 0, i:i + (1 << 20)].normal_(generator=g)
    q = rnd(2, 1, 3, d, dt="bf16")
    scores = torch.zeros(1, 1, n, device="cuda")
    out = tss().attend(q, kv, kv, scores=scores)
    # in 64 bits, in pieces on the GPU
    s = torch.cat([(kv[0, 0, i:i + (1 << 20)].double() @ q[0].double().t().contiguous()) for i in range(0, n, 1 << 20)]) * d ** -0.5
    p = torch.softmax(s, 0)
    want = torch.zeros(3, d, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for i in range(0, n, 1 << 20):
        rows = kv[0, 0, i:i + (1 << 20)].double()
        want += p[i:i + (1 << 20)].t().contiguous() @ rows
        size += p[i:i + (1 << 20)].t().contiguous() @ rows.abs()
    # the sums here are of 2^24 entries, most of them far from the maximum: (n + ..) U32 with n = 2^24 is 1; the
    # kernel's longest chain is what one lane or one register adds in a split, joined by waves and splits
    chain = 20000
    r = 1.1 * (2 * (d + 4) * U.U32 * 50 + 2 * 60 * U.U32 + chain * U.U32)
    U.within(out[0].cpu(), want.cpu(), (size * (r + chain * U.U32 + 2.0 ** -8)).cpu(), "out")
    add = p.sum(1)
    U.within(scores[0, 0].cpu(), add.cpu(), (add * r).cpu(), "scores")
    k2, v2, s2, kept, lengths = tss().evict(kv, kv, scores, 1000, recent=100)
    order = torch.argsort(scores[0, 0, :n - 100], descending=True, stable=True)[:900].sort().values
    ids = torch.cat([order, torch.arange(n - 100, n, device="cuda")])
    assert torch.equal(kept[0, 0], ids) and torch.equal(k2[0, 0], kv[0, 0, ids]) and torch.equal(v2, k2)
    assert torch.equal(s2[0, 0], scores[0, 0, ids]) and lengths.tolist() == [1000]


def test_attend_refusals():
    T = tss()
    q, k = rnd(1, 2, 4, 16), rnd(2, 2, 2, 9, 16)
    s = torch.zeros(2, 2, 9, device="cuda")
    for bad in (lambda: T.attend(q[0], k, k), lambda: T.attend(q, k[0], k), lambda: T.attend(q, k, k[:, :, :8]), lambda: T.attend(q, k.bfloat16(), k),
                lambda: T.attend(q[:, :3], k, k), lambda: T.attend(rnd(1, 2, 4, 257), rnd(1, 2, 2, 9, 257), rnd(1, 2, 2, 9, 257)),
                lambda: T.attend(q, k, k, ends(1)), lambda: T.attend(q, k, k, ends(1, 2).int()), lambda: T.attend(q, k, k, scores=s.double()),
                lambda: T.attend(q, k, k, scores=s[:, :, :8]), lambda: T.attend(q, k, k, scores=s.transpose(1, 2).contiguous().transpose(1, 2)),
                lambda: T.attend(q, k, k, scale=math.inf), lambda: T.attend(q, k[:, :0], k[:, :0])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(T.TopkError):
        T.attend(q, k, k, scores=s[:, :1].expand(2, 2, 9))       # two heads would add to one row
    with pytest.raises(TypeError):
        T.attend(q.half(), k.half(), k.half())
    for bad in (lambda: T.attend(q.clone().requires_grad_(), k, k), lambda: T.attend(q, k, k.clone().requires_grad_())):
        with pytest.raises(RuntimeError, match="no gradient"):
            bad()
    assert T.attend(q[:0], k[:0], k[:0]).shape == (0, 4, 16)
    assert bool((T.attend(q, k[:, :, :0], k[:, :, :0], scores=s[:, :, :0]) == 0).all())


# ---------------------------------------------------------------- evict
def check_evict(k, v, s, budget, recent=0, lengths=None, label=""):
    k2, v2, s2, kept, ln = tss().evict(k, v, s, budget, recent, lengths)
    want, end = M.evict64(s, lengths, budget, recent)
    assert torch.equal(kept.cpu(), want), label
    assert torch.equal(ln.cpu(), end), label
    for got, old in ((k2, k), (v2, v), (s2, s)):
        assert torch.equal(got.cpu(), M.rows_of(old, want)), label


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 1000, 1023, 1024, 1025, 2049, 5000])
def test_evict_lengths(n, dt):
    k, v = rnd(n, 3, 2, n, 24, dt=dt), rnd(n + 1, 3, 2, n, 24, dt=dt)
    s = rnd(n + 2, 3, 2, n).abs()
    for budget in sorted({1, max(1, n // 3), max(1, n - 1), n, n + 7}):
        for recent in sorted({0, budget // 2, budget}):
            check_evict(k, v, s, budget, recent, label=(n, budget, recent))
    check_evict(k, v, s, max(1, n // 2), 0, ends(0, n, n // 2 + 1), "ragged")
    check_evict(k, v, s, max(1, n // 2), max(1, n // 4), ends(-5, n + 9, 1), "lengths out of range")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [0, 1, 3, 4, 7, 8, 9, 80, 128, 515, 1100])
def test_evict_widths(d, dt):
    k, v, s = rnd(1, 2, 2, 90, d, dt=dt), rnd(2, 2, 2, 90, d, dt=dt), rnd(3, 2, 2, 90).abs()
    check_evict(k, v, s, 37, 5, ends(90, 40), d)


def test_evict_equal_scores():
    k, v = rnd(1, 1, 1, 6000, 8), rnd(2, 1, 1, 6000, 8)
    for s in (torch.zeros(6000), torch.ones(6000), (torch.arange(6000) % 2).float(), (torch.arange(6000) % 7 == 0).float() * 0.5):
        for budget, recent in ((100, 0), (3000, 10), (5999, 0), (1, 1)):
            check_evict(k, v, s.reshape(1, 1, -1).cuda(), budget, recent, label=(budget, recent))


def test_evict_strange_scores():
    k, v = rnd(1, 1, 2, 500, 16), rnd(2, 1, 2, 500, 16)
    s = rnd(3, 1, 2, 500)
    s[0, 0, ::7] = math.inf
    s[0, 0, 1::7] = -math.inf
    s[0, 1, ::5] = 0.0
    s[0, 1, 1::5] = -0.0
    s[0, 1, 2::5] = 1e-45
    for budget in (30, 120, 300, 450):
        check_evict(k, v, s, budget, 9, label=budget)
    s[0, 1, 40:60] = NAN
    got = tss().evict(k, v, s, 25, 2)[3].cpu()
    assert torch.equal(got, M.evict64(s, None, 25, 2)[0])
    assert got[0, 1, :20].tolist() == list(range(40, 60))


def test_evict_layouts_and_bits():
    b, h, n, d = 2, 3, 200, 20
    k, v, s = rnd(1, b, n, h, d), rnd(2, b, n, h, d), rnd(3, h, b, n + 1).abs()[:, :, 1:].transpose(0, 1)
    check_evict(k.transpose(1, 2), v.transpose(1, 2), s, 77, 8, label="[b, n, h, d]")
    check_evict(k.transpose(1, 2)[..., 1:18], rnd(4, b, h, n, 34)[..., ::2], s, 77, 8, label="unaligned, stepped")
    check_evict(k.transpose(1, 2), v[:, :1].transpose(1, 2).expand(b, h, n, d), s[:, :, :1].expand(b, h, n), 77, 8, label="expanded")
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).reshape(1, 1, 256, 256).cuda()
    c = bits.view(torch.bfloat16)
    k2, _, _, kept, _ = tss().evict(c, c, torch.rand(1, 1, 256, device="cuda"), 100)
    assert torch.equal(k2.view(torch.int16)[0, 0], bits[0, 0, kept[0, 0]])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_evict_into_buffers(dt):
    b, h, n, d, room = 3, 2, 300, 33, 130
    k, v, s = rnd(1, b, h, n, d, dt=dt), rnd(2, b, h, n, d, dt=dt), rnd(3, b, h, n).abs()
    lengths = ends(300, 40, 0)
    ko = torch.full((b, room, h, d), 7.0, dtype=DT[dt], device="cuda").transpose(1, 2)
    vo = torch.full((b, h, room, d + 2), 8.0, dtype=DT[dt], device="cuda")[..., 1:d + 1]
    so = torch.full((b, h, room), 9.0, device="cuda")
    version = ko._version
    got = tss().evict(k, v, s, 100, 10, lengths, out=(ko, vo, so))
    assert got[0] is ko and got[1] is vo and got[2] is so and ko._version > version
    want, end = M.evict64(s, lengths, 100, 10)
    assert torch.equal(got[3].cpu(), want) and torch.equal(got[4].cpu(), end)
    for i, e in enumerate(end.tolist()):
        for t, old, mark in ((ko, k, 7.0), (vo, v, 8.0), (so, s, 9.0)):
            assert torch.equal(t[i, :, :e].cpu(), M.rows_of(old, want)[i, :, :e])
            assert bool((t[i, :, e:] == mark).all())      # rows behind the last, as they were


def test_evict_into_interleaved_buffers():
    # keys beside values, old ones and new ones in one tensor
    b, h, n, d = 2, 2, 60, 8
    pool = rnd(1, b, h, n, 4, d)
    k, v, ko, vo = (pool[:, :, :, i] for i in range(4))
    s = rnd(2, b, h, n, 2).abs()
    want = M.evict64(s[..., 0], None, 20, 3)[0]
    k0, v0 = k.clone(), v.clone()
    got = tss().evict(k, v, s[..., 0].contiguous(), 20, 3, out=(ko, vo, torch.zeros(b, h, 20, device="cuda")))
    assert torch.equal(got[3].cpu(), want)
    assert torch.equal(ko[:, :, :20].cpu(), M.rows_of(k0, want)) and torch.equal(vo[:, :, :20].cpu(), M.rows_of(v0, want))
    assert torch.equal(k, k0) and torch.equal(v, v0)


def test_attend_many_sequences():
    # more of them than lanes, and than lanes squared; most are empty, and one is long
    for b, n, d in ((70, 400, 16), (700, 300, 8), (5000, 300, 8)):
        q, k, v = rnd(1, b, 2, d), rnd(2, b, 1, n, d), rnd(3, b, 1, n, d)
        lengths = torch.randint(-n, n + 1, (b,), generator=torch.Generator().manual_seed(b)).cuda()
        lengths[b // 3] = n
        check_attend(q, k, v, lengths, label=b)


def test_attend_nothing_at_all():
    for n in (5, 5000):
        q, k = rnd(1, 3, 4, 40), torch.full((3, 2, n, 40), NAN, device="cuda")
        s = torch.ones(3, 2, n, device="cuda")
        assert bool((tss().attend(q, k, k, ends(0, 0, 0), s) == 0).all()) and bool((s == 1).all())
        assert bool((tss().attend(q, k, k, ends(0, 0, -1)) == 0).all())


def test_evict_refusals():
    T = tss()
    k, s = rnd(1, 2, 2, 50, 16), torch.rand(2, 2, 50, device="cuda")
    out = (rnd(2, 2, 2, 20, 16), rnd(3, 2, 2, 20, 16), torch.zeros(2, 2, 20, device="cuda"))
    wide = rnd(4, 2, 2, 20, 32)
    for bad in (lambda: T.evict(k, k, s, 0), lambda: T.evict(k, k, s, 10, 11), lambda: T.evict(k, k, s, 10, -1), lambda: T.evict(k, k[:, :, :9], s, 10),
                lambda: T.evict(k, k, s[:, :, :9], 10), lambda: T.evict(k, k, s.double(), 10), lambda: T.evict(k, k, s, 10, lengths=ends(1)),
                lambda: T.evict(k[0], k[0], s[0], 10), lambda: T.evict(k, k, s, 21, out=out), lambda: T.evict(k, k, s, 10, out=(out[0], out[0], out[2])),
                lambda: T.evict(k, k, s, 10, out=(k, out[1], out[2])), lambda: T.evict(k, k, s, 10, out=(out[0], out[1], s)),
                lambda: T.evict(k, k, s, 10, out=(out[0].bfloat16(), out[1], out[2])), lambda: T.evict(k, k, s, 10, out=(out[0][:1], out[1], out[2])),
                lambda: T.evict(k, k, s, 10, out=(k[:, :, 30:], out[1], out[2])),
                lambda: T.evict(k, k, s, 10, out=(wide[..., :16], wide[..., 8:24], out[2]))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(T.TopkError):
        T.evict(k, k, s, 10, out=(out[0][:, :1].expand(2, 2, 20, 16), out[1], out[2]))
    with pytest.raises(RuntimeError, match="no gradient"):
        T.evict(k.clone().requires_grad_(), k, s, 10)
    assert T.evict(k[:0], k[:0], s[:0], 10)[3].shape == (0, 2, 10)
    assert T.evict(k[:, :0], k[:, :0], s[:, :0], 10)[4].tolist() == [10, 10]
    assert T.evict(k[:, :, :0], k[:, :, :0], s[:, :, :0], 10)[3].eq(-1).all()


def test_graph_and_streams():
    T = tss()
    b, hq, h, n, d = 3, 8, 2, 700, 64
    q, k, v, s = rnd(1, b, hq, d, dt="bf16"), rnd(2, b, h, n, d, dt="bf16"), rnd(3, b, h, n, d, dt="bf16"), torch.zeros(b, h, n, device="cuda")
    lengths = ends(700, 3, 350)

    def step():
        s.zero_()
        out = T.attend(q, k, v, lengths, s)
        return (out, s.clone(), *T.evict(k, v, s, 200, 16, lengths))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        q.copy_(rnd(10 + i, b, hq, d, dt="bf16", scale=1.0 + i))
        k.copy_(rnd(20 + i, b, h, n, d, dt="bf16"))
        lengths.copy_(ends(700 - i, 3 + 100 * i, 350))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for x, y in zip(got, step()):
            assert torch.equal(x, y)
    caches = [(rnd(30 + i, b, hq, d), rnd(40 + i, b, h, n, d), torch.zeros(b, h, n, device="cuda")) for i in range(3)]
    want = []
    for cq, ck, cs in caches:
        T.attend(cq, ck, ck, scores=cs)
        want.append((cs.clone(), T.evict(ck, ck, cs, 100)[3]))
        cs.zero_()
    torch.cuda.synchronize()
    got = []
    for cq, ck, cs in caches:
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            T.attend(cq, ck, ck, scores=cs)
            got.append((cs, T.evict(ck, ck, cs, 100)[3]))
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
