"""Attention over a cache and its eviction where the ways differ: keys shared
over workgroups at every width, caches read past the caches, outputs stored
past them, many heads to a key-value head, long rows with equal and odd scores,
infinite keys, and how exactly a probability counts."""
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


# A probability that is multiplied with v as two bf16 numbers: the first has its leading bits less half a step (2^-7 of it at
# most is a step), the second is the rest, at most one and a half steps, off by half a step of its own, 2^-8 of it.
TWO_STEPS = 1.5 * 2.0 ** -7 * 2.0 ** -8


def attend_bound(q, k, v, lengths=None, scale=None):
    """attend64, its output's bound without a rounding of the probabilities to bf16."""
    out, eo, add, ea = M.attend64(q, k, v, lengths, scale, torch.float32)
    if q.dtype == torch.bfloat16:
        size = M.attend64(q, k, v.abs(), lengths, scale, torch.float32)[0]
        eo = eo + size * TWO_STEPS
    return out, eo, add, ea


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_probabilities_count_unrounded(dt):
    # two entries, of which the values cancel but for a hundredth: what a rounding of a probability adds is all that is left
    t = (torch.arange(64) * 0.0371 + 0.02).to(DT[dt])
    q = torch.zeros(1, 64, 8, dtype=DT[dt])
    q[0, :, 0] = t
    k = torch.zeros(1, 1, 2, 8, dtype=DT[dt])
    k[0, 0, 1, 0] = -1.0
    v = torch.empty(1, 1, 2, 8, dtype=DT[dt])
    for c in range(24):      # values from 0.08 to 1
        v[0, 0, 0] = torch.exp(-(torch.arange(8) + 8 * c) * 0.013).to(DT[dt])
        v[0, 0, 1] = -1.0
        a = [x.cuda() for x in (q, k, v)]
        out, eo, _, _ = attend_bound(*a, scale=1.0)
        U.within(tss().attend(*a, scale=1.0).cpu(), out, eo, c)
        # the same entries at the ends of 600, the others far below: pieces that are joined
        far = torch.full((1, 1, 600, 8), -1e4, dtype=DT[dt])
        far[:, :, :, 1:] = 0
        some = torch.ones(1, 1, 600, 8, dtype=DT[dt])
        for i, at in enumerate((0, 599)):
            far[:, :, at], some[:, :, at] = k[:, :, i], v[:, :, i]
        far, some = far.cuda(), some.cuda()
        U.within(tss().attend(a[0], far, some, scale=1.0).cpu(), out, eo + 600 * U.U32, (c, "far"))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_infinite_values_stay_infinite(dt):
    # of however small a probability, down to 2^-124, and at every position of its bits
    t = (torch.arange(512) / 512 * 85.9).to(DT[dt])
    q = torch.zeros(1, 512, 4, dtype=DT[dt], device="cuda")
    q[0, :, 0] = t.cuda()
    k = torch.zeros(1, 1, 2, 4, dtype=DT[dt], device="cuda")
    k[0, 0, 1, 0] = -1.0
    v = torch.tensor([[1.0, 2.0, 3.0, -4.0], [math.inf, -math.inf, 5.0, NAN]], device="cuda").to(DT[dt])[None, None]
    out = tss().attend(q, k, v, scale=1.0)[0]
    assert bool((out[:, 0] == math.inf).all()) and bool((out[:, 1] == -math.inf).all())
    assert bool(torch.isfinite(out[:, 2]).all()) and bool(torch.isnan(out[:, 3]).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [1, 3, 7, 8, 9, 15, 17, 20, 31, 33, 40, 50, 63, 65, 75, 80, 95, 97, 100, 127, 129, 130, 150, 161, 191, 193, 200, 225, 255, 256])
def test_keys_of_minus_infinity(d, dt):
    # whichever column is infinite, the entry has no probability and all others keep theirs
    for n in (40, 700):
        q, k, v = rnd(d, 1, 3, d, dt=dt).abs() + 0.25, rnd(d + 1, 1, 1, n, d, dt=dt, scale=0.5), rnd(d + 2, 1, 1, n, d, dt=dt)
        cols = sorted({0, d - 1, max(0, d - 2), max(0, d - 3), max(0, d - 4), max(0, d - 5), max(0, d - 8), max(0, d - 9), d // 2, d // 3})
        bad = [(7 * i + 3) % n for i in range(len(cols))]
        for c, j in zip(cols, bad):
            k[0, 0, j, c] = -math.inf
        good = [j for j in range(n) if j not in bad]
        out, eo, add, ea = M.attend64(q, k[:, :, good], v[:, :, good], None, None, q.dtype)
        scores = torch.full((1, 1, n), 0.25, device="cuda")
        U.within(tss().attend(q, k, v, scores=scores).cpu(), out, eo, (n, "out"))
        U.within(tss().attend(q, k, v).cpu(), out, eo, (n, "out alone"))
        U.within(scores[:, :, good].cpu(), 0.25 + add, ea, (n, "scores"))
        assert bool((scores[0, 0, bad] == 0.25).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_pieces_of_minus_infinity(dt):
    # whole workgroups' shares of entries without a probability, and all other logits far below 0
    for n, first, last in ((1000, 0, 513), (1000, 300, 999), (3000, 0, 2999), (3000, 1, 3000), (200, 0, 199), (260, 0, 256)):
        q = torch.zeros(2, 20, 16, dtype=DT[dt], device="cuda")
        q[..., 0] = 1.0
        k, v = rnd(n, 2, 1, n, 16, dt=dt), rnd(n + 1, 2, 1, n, 16, dt=dt)
        k[..., 0] -= 200.0
        k[:, :, first:last, 0] = -math.inf
        good = [j for j in range(n) if not first <= j < last]
        out, eo, add, ea = M.attend64(q, k[:, :, good], v[:, :, good], None, 1.0, q.dtype)
        scores = torch.full((2, 1, n), 0.25, device="cuda")
        U.within(tss().attend(q, k, v, scores=scores, scale=1.0).cpu(), out, eo, (n, "out"))
        U.within(tss().attend(q, k, v, scale=1.0).cpu(), out, eo, (n, "out alone"))
        U.within(scores[:, :, good].cpu(), 0.25 + add, ea, (n, "scores"))
        assert bool((scores[:, :, first:last] == 0.25).all())


def check_attend(q, k, v, lengths=None, label=""):
    b, h, n, _ = k.shape
    out, eo, add, ea = attend_bound(q, k, v, lengths)
    U.within(tss().attend(q, k, v, lengths).cpu(), out, eo, f"{label} out alone")
    before = torch.rand(b, h, n, generator=torch.Generator().manual_seed(1)).cuda()
    scores = before.clone()
    U.within(tss().attend(q, k, v, lengths, scores).cpu(), out, eo, f"{label} out")
    U.within(scores.cpu(), before.cpu().double() + add, ea, f"{label} scores")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [5, 36, 65, 80, 96, 100, 128, 130, 192, 200, 256])
def test_attend_shared_keys_of_every_width(d, dt):
    check_attend(rnd(d, 3, 6, d, dt=dt), rnd(d + 1, 3, 2, 700, d, dt=dt), rnd(d + 2, 3, 2, 700, d, dt=dt), ends(700, 0, 411), d)
    # more units than workgroups: several steps to a wave, pieces that end inside a row
    check_attend(rnd(d, 9, 34, d, dt=dt), rnd(d + 1, 9, 2, 5003, d, dt=dt), rnd(d + 2, 9, 2, 5003, d, dt=dt),
                 ends(5003, 1, 4096, 4097, 0, 2500, 5002, 3333, 4700), (d, "long"))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("hq,h,n", [(100, 1, 70), (100, 1, 700), (1000, 2, 300), (4096, 1, 40), (4096, 1, 600), (8192, 2, 130)])
def test_attend_many_heads_on_one(hq, h, n, dt):
    check_attend(rnd(hq, 2, hq, 16, dt=dt), rnd(h, 2, h, n, 16, dt=dt), rnd(h + 1, 2, h, n, 16, dt=dt), ends(n, n - 13), (hq, h, n))


@pytest.mark.parametrize("dt,d", [("f32", 80), ("f32", 128), ("bf16", 96), ("bf16", 200)])
def test_attend_past_the_caches(dt, d):
    # 64 MB of keys and values and more, every head its own rows
    n = (1 << 26) // (2 * 8 * d * (4 if dt == "f32" else 2)) + 5
    check_attend(rnd(d, 2, 8, d, dt=dt), rnd(d + 1, 2, 4, n, d, dt=dt), rnd(d + 2, 2, 4, n, d, dt=dt), ends(n, n - 77), (dt, d))


def test_attend_f32_offsets_beyond_32_bits():
    n, d = (1 << 24) + 1000, 128
    kv = torch.empty(1, 1, n, d, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for i in range(0, n, 1 << 20):
        kv[0, 0, i:i + (1 << 20)].normal_(generator=g)
    # the last entries, far beyond 2^31 elements, take nearly all
    kv[0, 0, n - 3:] = torch.eye(3, d, device="cuda") * 60
    q = torch.zeros(1, 3, d, device="cuda")
    for i in range(3):
        q[0, i, i] = 12.0
    scores = torch.zeros(1, 1, n, device="cuda")
    out = tss().attend(q, kv, kv, scores=scores)
    s = torch.cat([(kv[0, 0, i:i + (1 << 20)].double() @ q[0].double().t().contiguous()) for i in range(0, n, 1 << 20)]) * d ** -0.5
    p = torch.softmax(s, 0)
    # a logit of the others is below 10, that of the last ones 63: 2^24 of them have less than 2^24 e^-53 together
    near = torch.zeros(3, d, dtype=torch.float64, device="cuda")
    for i in range(0, n, 1 << 20):
        near += p[i:i + (1 << 20)].t().contiguous() @ kv[0, 0, i:i + (1 << 20)].double()
    r = 1.1 * (2 * (d + 4) * U.U32 * 64 + 2 * (64 + 15 + 4) * U.U32 + 20000 * U.U32)
    U.within(out[0].cpu(), near.cpu(), torch.full((3, d), 60 * r, dtype=torch.float64), "out")
    U.within(scores[0, 0].cpu(), p.sum(1).cpu(), p.sum(1).cpu() * r, "scores")
    assert bool((scores[0, 0, n - 3:] > 0.99).all())


# ---------------------------------------------------------------- evict
def bits(t):
    """NaN are equal to themselves."""
    return t.cpu().contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def check_evict(k, v, s, budget, recent=0, lengths=None, out=None, label=""):
    want, end = M.evict64(s, lengths, budget, recent)
    marks = None if out is None else [t.clone() for t in out]
    k2, v2, s2, kept, ln = tss().evict(k, v, s, budget, recent, lengths, out=out)
    assert torch.equal(kept.cpu(), want), label
    assert torch.equal(ln.cpu(), end), label
    for x, (got, old) in enumerate(((k2, k), (v2, v), (s2, s))):
        if out is None:
            assert torch.equal(bits(got), bits(M.rows_of(old, want))), label
            continue
        for i, e in enumerate(end.tolist()):     # rows behind the last, as they were
            assert torch.equal(bits(got[i, :, :e]), bits(M.rows_of(old, want)[i, :, :e])), label
            assert torch.equal(bits(got[i, :, e:]), bits(marks[x][i, :, e:])), label


@pytest.mark.parametrize("n", [16383, 16384, 16385, 20000, 40001])
def test_evict_long_rows(n):
    g = torch.Generator().manual_seed(n)
    k, v = rnd(1, 3, 2, n, 6), rnd(2, 3, 2, n, 6, dt="f32")
    for name, s in (("spread", torch.rand(3, 2, n, generator=g)), ("few values", torch.randint(0, 4, (3, 2, n), generator=g).float()),
                    ("zeros", torch.zeros(3, 2, n)), ("ones", torch.ones(3, 2, n)),
                    ("signs", torch.randn(3, 2, n, generator=g).mul(100).round().div(100))):
        s = s.clone()
        if name == "signs":
            s[0, 0, ::5] = -0.0
            s[0, 1, 1::7] = NAN
            s[1, 0, ::3] = math.inf
            s[1, 0, 1::3] = -math.inf
            s[2, 1, ::2] = 1e-45
        s = s.cuda()
        for budget, recent in ((1, 0), (n // 4, 100), (n - 1, 0), (12000, 12000), (5000, 1)):
            check_evict(k, v, s, budget, recent, ends(n, n - 3000, 5001), label=(name, budget, recent))
        check_evict(k, v, s, 4000, 64, label=(name, "all"))


@pytest.mark.parametrize("dt,d", [("f32", 515), ("bf16", 515), ("bf16", 128), ("f32", 3)])
def test_evict_past_the_caches(dt, d):
    # 16 MB of rows and more in each output
    size = 4 if dt == "f32" else 2
    budget = (1 << 24) // (2 * 2 * d * size) + 3
    n = budget + budget // 3
    k, v = rnd(1, 2, 2, n, d, dt=dt), rnd(2, 2, 2, n, d, dt=dt)
    s = torch.rand(2, 2, n, generator=torch.Generator().manual_seed(3)).cuda()
    for lengths in (ends(n, n - 5), ends(budget // 2, n)):
        check_evict(k, v, s, budget, budget // 8, lengths, label=(dt, d))
        out = (torch.full((2, 2, budget + 2, d), 7.0, dtype=DT[dt], device="cuda"),
               torch.full((2, budget + 1, 2, d), 8.0, dtype=DT[dt], device="cuda").transpose(1, 2),
               torch.full((2, 2, budget), 9.0, device="cuda"))
        check_evict(k, v, s, budget, budget // 8, lengths, out=out, label=(dt, d, "out"))
