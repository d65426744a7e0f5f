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
