"""The dense product with its epilogue, and its gradients, against 64 bits:
sizes around the tiles and the vector widths, both types, operands in either
order, strided and misaligned, empty axes, non-finite values, streams and
graphs."""
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


def check(x, w, b, act, res, label):
    y = tss().linear(x, w, b, activation=act, residual=res)
    ref, err, _ = U.linear64(x, w, b, act, res)
    U.within(y, ref, err, label)
    return y


SIZES = [(1, 1, 1), (1, 1, 64), (1, 130, 512), (2, 257, 96), (5, 16, 33), (15, 300, 64), (16, 128, 128),
         (17, 129, 515), (33, 4099, 72), (64, 64, 64), (65, 127, 40), (127, 128, 31), (128, 256, 96),
         (129, 255, 264), (130, 513, 1000), (256, 256, 32), (257, 300, 8), (300, 260, 2049), (511, 1, 100),
         (1000, 72, 7), (8, 2048, 4096), (40, 24, 20000), (513, 1030, 192)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_sizes(m, n, k, dt):
    act = ["none", "relu", "gelu", "silu"][(m + n + k) % 4]
    x, w = rnd(1, m, k, dt=dt), rnd(2, n, k, dt=dt, scale=k ** -0.5)
    check(x, w, rnd(3, n, dt=dt), act, rnd(4, m, n, dt=dt) if (m + n) % 2 else None, f"{m}x{n}x{k} {dt} {act}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(2100, 4100, 136), (4136, 2049, 72), (4096, 4096, 64), (5000, 700, 1032), (300, 17000, 200)])
def test_large_tiles(m, n, k, dt):
    # the larger tiles, outputs that are stored past the caches, edges in both directions, either order of the operands
    x, w, b, r = rnd(70, m, k, dt=dt), rnd(71, n, k, dt=dt, scale=k ** -0.5), rnd(72, n, dt=dt), rnd(73, m, n, dt=dt)
    want = U.linear64(x, w, b, "silu", r)
    xt, wt = x.t().contiguous().t(), w.t().contiguous().t()
    for xx, ww in ((x, w), (x, wt), (xt, w), (xt, wt)):
        U.within(tss().linear(xx, ww, b, activation="silu", residual=r), want[0], want[1], f"{m}x{n}x{k}")
    dy = rnd(74, m, n, dt=dt)
    refs, errs = U.linear_grad64(dy, x, w, r, "gelu")
    for got, ref, err in zip(tss().linear_grad(dy, x, w, activation="gelu", pre=r), refs, errs):
        U.within(got, ref, err, f"gradient {m}x{n}x{k}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(4, 40, 64), (70, 130, 96), (4100, 4104, 64)])
def test_residual_in_place_and_pre_activation_through_the_abi(m, n, k, dt):
    import ctypes
    lib = tss()._lib
    x, w, y = rnd(75, m, k, dt=dt), rnd(76, n, k, dt=dt, scale=0.2), rnd(77, m, n + 3, dt=dt)
    start, pre = y.clone(), torch.full((m, n + 1), 5.0, dtype=DT[dt], device="cuda")
    a = lib.LinearArgs(x.data_ptr(), w.data_ptr(), None, y.data_ptr(), y.data_ptr(), pre.data_ptr(), m, n, k, k, k,
                       n + 3, n + 3, n + 1, tss().dtype_code(DT[dt]), lib.ACTIVATIONS["gelu"], 0, 0)
    size = ctypes.c_size_t()
    assert lib.lib.topk_linear_workspace_size(ctypes.byref(a), ctypes.byref(size)) == 0
    ws = torch.empty(size.value + 1, dtype=torch.uint8, device="cuda")
    assert lib.lib.topk_linear(ctypes.byref(a), ws.data_ptr(), size.value, torch.cuda.current_stream().cuda_stream) == 0
    ref, err, z = U.linear64(x, w, None, "gelu", start[:, :n])
    U.within(y[:, :n], ref, err)
    U.within(pre[:, :n], z, (k + 3) * U.U32 * (x.double().abs() @ w.double().abs().t().contiguous()))
    assert torch.equal(y[:, n:], start[:, n:]) and bool((pre[:, n:] == 5).all())   # nothing behind the rows


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("with_bias,with_res", [(0, 0), (1, 0), (0, 1), (1, 1)])
def test_epilogue(act, with_bias, with_res, dt):
    for m, n, k in ((7, 190, 136), (150, 190, 136)):
        x, w = rnd(5, m, k, dt=dt), rnd(6, n, k, dt=dt, scale=0.3)
        check(x, w, rnd(7, n, dt=dt) if with_bias else None, act, rnd(8, m, n, dt=dt) if with_res else None,
              f"{act} bias {with_bias} residual {with_res} {m} rows")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(3, 200, 144), (140, 136, 200), (300, 1000, 520)])
def test_orders_and_strides(m, n, k, dt):
    base_x, base_w = rnd(9, m, k, dt=dt), rnd(10, n, k, dt=dt, scale=0.1)
    want = U.linear64(base_x, base_w, None, "none", None)

    def strided(t, pad, off):
        big = torch.full((t.shape[0], t.shape[1] + pad), 3.0, dtype=t.dtype, device="cuda")
        big[:, off:off + t.shape[1]] = t
        return big[:, off:off + t.shape[1]]

    def misaligned(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    forms = {"plain": lambda t: t, "transposed": lambda t: t.t().contiguous().t(),
             "stride 16": lambda t: strided(t, 16, 8), "odd stride": lambda t: strided(t, 3, 1),
             "misaligned": misaligned, "transposed odd": lambda t: strided(t.t().contiguous(), 5, 2).t(),
             "stepped": lambda t: t.repeat_interleave(2, 1)[:, ::2]}
    for fx in forms:
        for fw in forms:
            if fx != "plain" and fw not in ("plain", fx):
                continue
            x, w = forms[fx](base_x), forms[fw](base_w)
            assert torch.equal(x, base_x) and torch.equal(w, base_w)
            U.within(tss().linear(x, w), want[0], want[1], f"x {fx}, w {fw}")


def test_residual_layouts_and_leading_axes():
    x, w = rnd(11, 2, 3, 40, dt="bf16"), rnd(12, 50, 40, dt="bf16")
    res = rnd(13, 50, dt="bf16").expand(2, 3, 50)
    y = tss().linear(x, w, activation="relu", residual=res)
    assert y.shape == (2, 3, 50)
    ref, err, _ = U.linear64(x.reshape(6, 40), w, None, "relu", res.reshape(6, 50))
    U.within(y.reshape(6, 50), ref, err)
    one = tss().linear(x[0, 0], w)
    assert one.shape == (50,)
    assert torch.equal(one, tss().linear(x[0, :1], w)[0])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_empty_axes(dt):
    for m, n, k in ((0, 5, 4), (4, 0, 5), (3, 6, 0), (0, 0, 0), (200, 300, 0)):
        x, w, b, r = rnd(1, m, k, dt=dt), rnd(2, n, k, dt=dt), rnd(3, n, dt=dt), rnd(4, m, n, dt=dt)
        y = tss().linear(x, w, b, activation="silu", residual=r)
        assert y.shape == (m, n)
        ref, err, _ = U.linear64(x, w, b, "silu", r)
        U.within(y, ref, err)
        dx, dw, db = tss().linear_grad(r, x, w, activation="silu", pre=r)
        assert dx.shape == (m, k) and dw.shape == (n, k) and db.shape == (n,)
        refs, errs = U.linear_grad64(r, x, w, r, "silu")
        for got, ref, err in zip((dx, dw, db), refs, errs):
            U.within(got, ref, err)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("m", [3, 200])
def test_non_finite_stays_in_its_row_and_column(act, dt, m):
    n, k = 150, 70
    x, w = rnd(14, m, k, dt=dt), rnd(15, n, k, dt=dt)
    clean = tss().linear(x, w, activation=act)
    x[1, 69] = math.inf
    x[2, 3] = math.nan
    w[140, 0] = -math.inf
    y = tss().linear(x, w, activation=act)
    ref = U.act64(x.double() @ w.double().t().contiguous(), act)
    keep = torch.ones(m, n, dtype=torch.bool, device="cuda")
    keep[1], keep[2], keep[:, 140] = False, False, False
    assert torch.equal(y[keep], clean[keep])
    odd = ~keep
    assert torch.equal(torch.isnan(y[odd]), torch.isnan(ref[odd]))
    inf = odd & torch.isinf(ref)
    assert torch.equal(y[inf].double(), ref[inf])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_huge_and_tiny_values(dt):
    # products that leave the type's range only after the sum, and values near the ends of the range
    big, tiny = 1e30, 1e-30
    x = torch.tensor([[big, -big, 1.0, tiny], [tiny, tiny, 0.0, big]], dtype=DT[dt], device="cuda")
    w = torch.tensor([[1.0, 1.0, 2.0, 0.0], [tiny, 0.0, 1.0, big]], dtype=DT[dt], device="cuda")
    ref, err, _ = U.linear64(x, w, None, "none", None)
    U.within(tss().linear(x, w), ref.clamp(-3.4e38, 3.4e38) * (ref.abs() < 3.4e38) + torch.where(
        ref.abs() < 3.4e38, torch.zeros_like(ref), torch.sign(ref) * math.inf).nan_to_num(0, math.inf, -math.inf), err)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 300, 64), (9, 70, 130), (16, 512, 128), (130, 257, 65), (300, 136, 264),
                                   (700, 40, 24), (257, 1030, 96), (2100, 64, 72)])
def test_gradients(m, n, k, act, dt):
    x, w, dy = rnd(16, m, k, dt=dt), rnd(17, n, k, dt=dt, scale=0.2), rnd(18, m, n, dt=dt)
    pre = rnd(19, m, n, dt=dt)
    got = tss().linear_grad(dy, x, w, activation=act, pre=None if act == "none" else pre)
    refs, errs = U.linear_grad64(dy, x, w, pre, act)
    for g, ref, err, what in zip(got, refs, errs, ("dx", "dw", "db")):
        U.within(g, ref, err, f"{what} {m}x{n}x{k} {act} {dt}")
    some = tss().linear_grad(dy, x, w, activation=act, pre=pre, need=(False, True, False))
    assert some[0] is None and some[2] is None and torch.equal(some[1], got[1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradients_of_strided_operands(dt):
    m, n, k = 140, 90, 77
    x = rnd(20, k, m, dt=dt).t()
    w = rnd(21, n, k + 5, dt=dt)[:, 2:2 + k]
    dy = rnd(22, m, n + 1, dt=dt)[:, 1:]
    pre = rnd(23, m, n + 3, dt=dt)[:, :n]
    refs, errs = U.linear_grad64(dy, x, w, pre, "gelu")
    for g, ref, err in zip(tss().linear_grad(dy, x, w, activation="gelu", pre=pre), refs, errs):
        U.within(g, ref, err)
    dyb = rnd(24, n, dt=dt).expand(m, n)   # a broadcast gradient, as a sum's backward gives
    refs, errs = U.linear_grad64(dyb, x, w, pre, "relu")
    for g, ref, err in zip(tss().linear_grad(dyb, x, w, activation="relu", pre=pre), refs, errs):
        U.within(g, ref, err)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("with_res", [0, 1])
def test_autograd_against_differences(act, with_res):
    # central differences of a weighted sum of the outputs in 64 bits, along random directions
    m, n, k = 6, 9, 11
    x, w, b = rnd(25, m, k), rnd(26, n, k, scale=0.4), rnd(27, n)
    r, c = rnd(28, m, n), rnd(29, m, n)
    leaves = [x, w, b] + ([r] if with_res else [])
    for t in leaves:
        t.requires_grad_(True)
    y = tss().linear(x, w, b, activation=act, residual=r if with_res else None)
    grads = torch.autograd.grad((y * c).sum(), leaves)
    h = 1e-5

    def f(vals):
        z = vals[0] @ vals[1].t() + vals[2]
        return float(((U.act64(z, act) + (vals[3] if with_res else 0)) * c.double()).sum())

    base = [t.detach().double() for t in leaves]
    for i, g in enumerate(grads):
        way = rnd(30 + i, *leaves[i].shape).double()
        up, down = [t.clone() for t in base], [t.clone() for t in base]
        up[i] += h * way
        down[i] -= h * way
        want = (f(up) - f(down)) / (2 * h)
        got = float((g.double() * way).sum())
        # the difference quotient: h^2 times the third derivative (below 1e-8 of the magnitudes), and a kink of
        # relu crossed within h changes it by at most the crossing term's size h; the gradient: 32-bit sums
        scale = float((g.double().abs() * way.abs()).sum()) + float((c.double().abs()).sum()) * h
        assert abs(got - want) <= scale * 1e-4 + 1e-6


def test_autograd_matches_linear_grad_and_skips():
    m, n, k = 50, 70, 40
    x, w, b, r = (rnd(31, m, k, dt="bf16"), rnd(32, n, k, dt="bf16"), rnd(33, n, dt="bf16"), rnd(34, m, n, dt="bf16"))
    dy = rnd(35, m, n, dt="bf16")
    x.requires_grad_(True)
    r.requires_grad_(True)
    y = tss().linear(x, w, b, activation="gelu", residual=r)
    y.backward(dy)
    pre = tss().linear(x.detach(), w, b)
    dx = tss().linear_grad(dy, x.detach(), w, activation="gelu", pre=pre, need=(1, 0, 0))[0]
    assert torch.equal(x.grad, dx) and torch.equal(r.grad, dy)
    assert w.grad is None
    with torch.no_grad():
        assert not tss().linear(x, w, b).requires_grad


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_same_result_every_time(dt):
    x, w, dy = rnd(36, 300, 2000, dt=dt), rnd(37, 72, 2000, dt=dt), rnd(38, 300, 72, dt=dt)
    first = (tss().linear(x, w),) + tss().linear_grad(dy, x, w)
    for _ in range(3):
        for a, b in zip(first, (tss().linear(x, w),) + tss().linear_grad(dy, x, w)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 200])
def test_graph_replays_and_other_streams(dt, m):
    n, k = 130, 1500
    x, w, b = rnd(39, m, k, dt=dt), rnd(40, n, k, dt=dt), rnd(41, n, dt=dt)
    dy, pre = rnd(42, m, n, dt=dt), rnd(43, m, n, dt=dt)

    def step():
        return (tss().linear(x, w, b, activation="silu"),) + tss().linear_grad(dy, x, w, activation="silu", pre=pre)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = step()
    torch.cuda.current_stream().wait_stream(side)
    eager = step()
    torch.cuda.synchronize()
    for a, c in zip(warm, eager):
        assert torch.equal(a, c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(3):
        x.copy_(rnd(50 + i, m, k, dt=dt))
        dy.copy_(rnd(60 + i, m, n, dt=dt))
        g.replay()
        want = step()
        torch.cuda.synchronize()
        for a, c in zip(out, want):
            assert torch.equal(a, c)
