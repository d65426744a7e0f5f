"""The next token at the ends of its ranges: tokens of little weight and their
probabilities, distances that overflow float32, settings that want a gradient."""
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


def check(z, u, label="", off=1e-9, **kw):
    full = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0) | kw
    token, logprob = tss().sample(z, u, **kw)
    rows = z.shape[0]
    zc, uc = z.cpu(), u.tolist()
    want = [M.sample64(zc[r], uc[r], *(M.f32(full["temperature"]), full["top_k"], M.f32(full["top_p"]), M.f32(full["min_p"]))) for r in range(rows)]
    assert token.tolist() == [t for t, _ in want], label
    U.within(logprob.cpu(), torch.tensor([p for _, p in want], dtype=torch.float64), torch.full((rows,), off, dtype=torch.float64), label)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [12, 400, 3000, 9000])
def test_distances_that_overflow(n, dt):
    # logits at both ends of the type, at temperatures that make something of their distance: it is no float32, but counts
    z = rnd(n, 4, n, scale=1e38).cpu().clamp(-3.2e38, 3.2e38)
    z[0, 0], z[0, 1:] = 3.2e38, -3.2e38
    z[1, n // 2] = 3.3e38
    z[1, ::3] = -3.3e38
    z[2, :] = -3.3e38
    z[2, n - 1] = 3.3e38
    z = z.to(DT[dt]).cuda()
    assert bool(torch.isfinite(z).all())
    for u in (2.0 ** -20, 0.5, 0.9, LAST):
        for t in (1e37, 1.5e38, 3.4e38):
            for kw in (dict(), dict(top_k=1), dict(top_k=2), dict(top_k=7), dict(top_k=n - 1), dict(top_k=n), dict(top_p=0.5), dict(top_p=0.97),
                       dict(top_k=9, top_p=0.9), dict(min_p=0.02)):
                check(z, torch.full((4,), u, device="cuda"), (u, t, kw), temperature=t, **kw)


@pytest.mark.parametrize("n", [40, 300, 513, 3000, 131072, 300007])
def test_probability_of_a_rare_token(n):
    # a number of 0 draws the first token with any weight, here one of down to 2^-40 of the largest.  Its own weight counts
    # as it is; the sum of all is of weights rounded to multiples of 2^-(62 - log2 n), off by less than n^2 2^-63 of the
    # largest one, of which the logprob has as much
    unit = 2.0 ** -(62 - math.ceil(math.log2(n)))
    off = 1e-9 + n * unit
    for others in (-math.inf, -2.0):
        low = [2.0, 9.7, 16.1, 20.3, 23.9, 26.8, 28.1] if n <= 3000 or others == -math.inf else [16.1, 20.3, 26.8]
        z = torch.full((len(low), n), others)
        if others > -math.inf:
            z += torch.randn(len(low), n, generator=torch.Generator().manual_seed(n)) * 0.5
        for r, far in enumerate(low):
            assert math.exp(-far) > 2 * unit
            z[r, 0] = -far
            z[r, n // 2] = 0.0
        z = z.cuda()
        u = torch.zeros(len(low), device="cuda")
        check(z, u, "plain", off)
        check(z, u, "top_k", off, top_k=n - 1)
        if n <= 3000:
            check(z, u, "top_k and p", off, top_k=n, top_p=LAST)
        for kw in (dict(top_k=2), dict(top_k=20)):
            if others == -math.inf:
                check(z, u, kw, off, **kw)


def test_settings_that_want_a_gradient():
    # the results would be constants to autograd: refused, as logits that want one are
    T, z, u = tss(), rnd(1, 3, 50), torch.rand(3, device="cuda")
    one = torch.full((3,), 0.5, device="cuda", requires_grad=True)
    for f in (lambda: T.sample(z, u, temperature=one), lambda: T.sample(z, u, top_p=one), lambda: T.sample(z, u, min_p=one), lambda: T.sample(z, one)):
        with pytest.raises(RuntimeError, match="no gradient"):
            f()
        with torch.no_grad():
            f()
    from torch.autograd import forward_ad as F
    with F.dual_level():
        dual = F.make_dual(one.detach(), torch.ones(3, device="cuda"))
        for f in (lambda: T.sample(z, u, temperature=dual), lambda: T.sample(z, u, top_p=dual), lambda: T.sample(z, u, min_p=dual)):
            with pytest.raises(RuntimeError, match="forward-mode"):
                f()
