"""Tokens by expert and back at sizes that are stored past the caches, and at
offsets beyond 2^31 elements."""
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


@pytest.mark.parametrize("dt,wdt,d", [("f32", "f32", 515), ("bf16", "f32", 515), ("bf16", "bf16", 128), ("bf16", None, 7), ("f32", "f32", 3)])
def test_gradient_past_the_caches(dt, wdt, d):
    # 16 MB of dy and more: distinct places, some dropped, some named by several entries, some by none
    n = (1 << 24) // (d * (4 if dt == "f32" else 2)) + 77
    t, k = n // 4 + 1, 3
    places = torch.randperm(n, generator=torch.Generator().manual_seed(d))[:t * k].reshape(t, k).cuda()
    places[::5, 1] = places[0, 1]
    places[1::7, 2] = -1
    places[2::11, 0] = n + 3
    places[3::13, 0] = ints(d, 0, n, len(range(3, t, 13)))
    if t > 60000:       # a place that very many name is slow, and tested elsewhere
        places[::5, 1] = ints(d + 1, 0, 500, len(range(0, t, 5)))
    y, g = rnd(1, n, d, dt=dt), rnd(2, t, d, dt=dt)
    w = rnd(3, t, k, dt=wdt) if wdt else None
    (dy, dw), (ey, ew) = M.combine_grad64(g, y, places, w)
    got, gw = tss().combine_grad(g, y, places, w)
    U.within(got.cpu(), dy, ey, "dy")
    if w is not None:
        U.within(gw.cpu(), dw, ew, "dw")
    out, err = M.combine64(y, places, w)
    U.within(tss().combine(y, places, w).cpu(), out, err, "out")


def test_rows_beyond_32_bits():
    # 2^31 elements and more in rows, and in what is gathered from them
    t, k, d, e = 600001, 4, 1024, 9
    x = torch.empty(t, d, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x.normal_(generator=g)
    experts = ints(2, -1, e, t, k)
    rows, places, offsets = tss().dispatch(x, experts, e)
    key = torch.where(experts.reshape(-1) < 0, e, experts.reshape(-1))
    order = torch.argsort(key, stable=True)
    end = int(offsets[-1])
    assert end == int((key < e).sum()) and rows.numel() > 1 << 31
    for i in range(0, end, 200000):
        j = min(i + 200000, end)
        assert torch.equal(rows[i:j], x[order[i:j] // k])
    assert not bool(rows[end:].any())
    # rows of a token are equal: the sum of k is exact in 32 bits, and rounded once
    want = x.float() * (experts >= 0).sum(1, keepdim=True)
    assert torch.equal(tss().combine(rows, places), want.to(torch.bfloat16))
    dy, _ = tss().combine_grad(x, rows, places, need=(True, False))
    assert torch.equal(dy, rows)
