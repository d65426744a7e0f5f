"""GPU: operators at the edges of their operands: what lies beside and behind a
matrix stays out of the results, and outputs at odd argument combinations."""
import ctypes
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


def among_nan(t, left, right):
    """The same matrix as columns of a wider one, NaN on both sides and behind the last row."""
    rows, cols = t.shape
    big = torch.full((rows + 1, left + cols + right), math.nan, dtype=t.dtype, device="cuda")
    big[:rows, left:left + cols] = t
    return big[:rows, left:left + cols]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("left,right", [(0, 8), (0, 1), (3, 10)])
@pytest.mark.parametrize("m,n,k", [(1, 13, 48), (3, 35, 48), (8, 13, 48), (17, 13, 64), (20, 35, 40), (32, 7, 200),
                                   (200, 13, 48), (200, 35, 72), (300, 259, 130)])
def test_gradients_of_a_weight_stored_by_columns(m, n, k, left, right, act, dt):
    # tied weights: linear(x, v.t()); few rows and small products read such a weight where it lies
    x, w, dy, pre = (rnd(1, m, k, dt=dt), rnd(2, n, k, dt=dt, scale=0.2), rnd(3, m, n, dt=dt), rnd(4, m, n, dt=dt))
    refs, errs = U.linear_grad64(dy, x, w, pre, act)
    tied = among_nan(w.t().contiguous(), left, right).t()
    got = tss().linear_grad(among_nan(dy, left, right), x, tied, activation=act,
                            pre=None if act == "none" else among_nan(pre, right, left))
    for g, ref, err, what in zip(got, refs, errs, ("dx", "dw", "db")):
        U.within(g, ref, err, f"{what} {m}x{n}x{k} {act} {dt}")
    got = tss().linear_grad(dy, among_nan(x.t().contiguous(), left, right).t(), among_nan(w, left, right),
                            activation=act, pre=None if act == "none" else pre)
    for g, ref, err, what in zip(got, refs, errs, ("dx", "dw", "db")):
        U.within(g, ref, err, f"{what} {m}x{n}x{k} {act} {dt}, x by columns")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 13, 33), (20, 7, 35), (200, 35, 13), (300, 259, 131)])
def test_product_of_operands_among_nan(m, n, k, dt):
    x, w, b, r = rnd(5, m, k, dt=dt), rnd(6, n, k, dt=dt), rnd(7, n, dt=dt), rnd(8, m, n, dt=dt)
    ref, err, _ = U.linear64(x, w, b, "relu", r)
    for by_rows in (True, False):
        for left, right in ((0, 8), (1, 3)):
            put = (lambda t: among_nan(t, left, right)) if by_rows else (
                lambda t: among_nan(t.t().contiguous(), left, right).t())
            U.within(tss().linear(put(x), put(w), among_nan(b[None], left, right)[0], "relu", among_nan(r, left, right)),
                     ref, err, f"{m}x{n}x{k} {dt}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_autograd_of_tied_weights(dt):
    # the reconstruction h @ v of a tied autoencoder, v's rows of odd length: v.t() is the weight
    m, n, k = 8, 13, 48
    h, v, c = rnd(9, m, k, dt=dt), rnd(10, k, n, dt=dt, scale=0.2), rnd(11, m, n, dt=dt)
    refs, errs = U.linear_grad64(c, h, v.t(), None, "none")
    h.requires_grad_(True)
    v.requires_grad_(True)
    tss().linear(h, v.t()).backward(c)
    U.within(h.grad, refs[0], errs[0], "h")
    U.within(v.grad, refs[1].t(), errs[1].t(), "v")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("rows,k,n,d", [(5, 30, 40, 512), (40, 300, 9000, 24), (3, 4, 20_000, 1100), (7, 3, 5, 3)])
def test_bias_gradient_of_the_encoder_alone_reads_no_rows(rows, k, n, d, flat, dt):
    # x is not read without dweight, and weight not without dx: both null
    lib = tss()._lib
    g = torch.Generator().manual_seed(12)
    idx = torch.randint(0, rows * n, (rows * k,), generator=g) if flat else torch.randint(0, n, (rows, k), generator=g)
    idx[..., -1] = -1
    v, gv = rnd(13, *idx.shape, dt=dt), rnd(14, *idx.shape, dt=dt)
    idx = idx.cuda()
    db = torch.full((n,), 7.0, dtype=DT[dt], device="cuda")
    sel = ctypes.byref(lib.Selection(v.data_ptr(), idx.data_ptr(), rows, idx.numel() if flat else k, n, flat,
                                     tss().dtype_code(DT[dt])))
    size = ctypes.c_size_t()
    assert lib.lib.topk_decode_workspace_size(sel, d, ctypes.byref(size)) == 0
    ws = torch.empty(size.value, dtype=torch.uint8, device="cuda")
    assert lib.lib.topk_encode_grad(sel, gv.data_ptr(), None, 0, None, 0, d, None, 0, None, 0, db.data_ptr(),
                                    ws.data_ptr(), size.value, torch.cuda.current_stream().cuda_stream) == 0
    e, _, j = U.entries(idx, rows, n)
    c = torch.where(v.reshape(-1).cpu()[e] > 0, gv.reshape(-1).cpu()[e].double(), 0.0)
    ref, err = U.group64(c, j, torch.zeros_like(j), n, torch.ones(1, 1))
    U.within(db.cpu(), ref[:, 0], err[:, 0])
    # beside dx, and against the call that computes all three
    x, w = rnd(15, rows, d, dt=dt), rnd(16, n, d, dt=dt)
    dx, _, alone = tss().encode_grad(gv, v, idx, x, w, need=(1, 0, 1))
    want = tss().encode_grad(gv, v, idx, x, w)
    assert torch.equal(alone, want[2]) and torch.equal(db, want[2]) and torch.equal(dx, want[0])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("total", [5, 6000])
@pytest.mark.parametrize("d", [3, 64, 1030])
def test_values_have_no_gradient_where_there_are_no_latents(d, total, dt):
    # no latent: every entry is out of range, and gets 0, also when an (empty) dweight is wanted beside it
    lib = tss()._lib
    v, g = rnd(17, total, dt=dt), rnd(18, 4, d, dt=dt)
    idx = torch.arange(total, device="cuda")
    dv, db = torch.full((total,), 7.0, dtype=DT[dt], device="cuda"), torch.full((d,), 7.0, dtype=DT[dt], device="cuda")
    somewhere = torch.zeros(64, dtype=DT[dt], device="cuda")     # stands for the empty matrices; nothing is written there
    sel = ctypes.byref(lib.Selection(v.data_ptr(), idx.data_ptr(), 4, total, 0, 1, tss().dtype_code(DT[dt])))
    size = ctypes.c_size_t()
    assert lib.lib.topk_decode_workspace_size(sel, d, ctypes.byref(size)) == 0
    ws = torch.empty(size.value + 1, dtype=torch.uint8, device="cuda")
    assert lib.lib.topk_decode_grad(sel, somewhere.data_ptr(), d, d, g.data_ptr(), d, dv.data_ptr(), somewhere.data_ptr(),
                                    d, db.data_ptr(), ws.data_ptr(), size.value,
                                    torch.cuda.current_stream().cuda_stream) == 0
    assert not dv.any() and not somewhere.any()
    U.within(db, g.double().sum(0), 7 * U.U32 * g.double().abs().sum(0))


def gelu_tail_errors(z, dt):
    """Relative errors of the normal distribution function and of z times its density, left of 0.

    bf16: the function is fitted to 1.8e-4 of its value, the rest of its evaluation (a reciprocal, a polynomial of six
    steps, an exponential) adds less than 1e-5; f32: erfc's argument is off by 1.3 roundings, which erfc takes
    z^2 + 1 times, and erfc itself by at most 16.  The density: an exponent of z^2 / 2 off by at most 5 roundings
    (bf16) or 2 (f32), the exponential and three products."""
    z2 = z * z
    if dt == "bf16":
        return 2e-4, (2.5 * z2 + 16) * U.U32
    return (1.3 * (z2 + 1) + 16) * U.U32, (z2 + 16) * U.U32


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("few", [True, False])
def test_gelu_and_its_slope_far_left_of_zero(few, dt):
    # relative to the value: an absolute bound near 1 says nothing of values of 1e-6 and 1e-30
    z = torch.linspace(-12.5, -3, 4001, device="cuda").to(DT[dt])[:, None].contiguous()
    one = torch.ones(1, 1, dtype=DT[dt], device="cuda")
    z64 = z.double()
    tail, bell = 0.5 * torch.special.erfc(-z64 / math.sqrt(2)), torch.exp(-z64 * z64 / 2) / math.sqrt(2 * math.pi)
    e_tail, e_bell = gelu_tail_errors(z64, dt)
    y = torch.cat([tss().linear(p, one, activation="gelu") for p in z.split(16 if few else 4001)])
    U.within(y, z64 * tail, (z64 * tail).abs() * (e_tail + 2 * U.U32), "gelu")
    dx = tss().linear_grad(torch.ones_like(z), z, one, activation="gelu", pre=z, need=(1, 0, 0))[0]
    U.within(dx, tail + z64 * bell, tail * e_tail + (z64 * bell).abs() * e_bell + 2 * U.U32 * (z64 * bell).abs(), "slope")


def test_forward_mode_is_refused():
    # a result without a tangent would be read as one of zero, by these calls and by a backward inside a dual level
    import torch.autograd.forward_ad as fw
    T = tss()
    x, w, b = rnd(20, 5, 8), rnd(21, 6, 8), rnd(22, 6)
    v, i = T.encode(x, w, b, 7)
    wd, g, gv = rnd(23, 6, 4), rnd(24, 5, 4), rnd(25, 7)
    plain = T.linear(x, w, b)

    def calls(d):
        yield lambda: T.linear(d(x), w, b)
        yield lambda: T.linear(x, w, d(b))
        yield lambda: T.linear(x, w, b, residual=d(plain))
        yield lambda: T.linear_grad(d(plain), x, w)
        yield lambda: T.linear_grad(plain, x, d(w))
        yield lambda: T.encode(x, d(w), b, 7)
        yield lambda: T.encode_grad(d(gv), v, i, x, w)
        yield lambda: T.encode_grad(gv, v, i, d(x), w)
        yield lambda: T.decode(d(v), i, wd, rows=5)
        yield lambda: T.decode(v, i, wd, rows=5, bias=d(wd[0].contiguous()))
        yield lambda: T.decode_grad(g, v, i, d(wd))
        yield lambda: T.grad_norm([x, d(w)])
        yield lambda: T.clip_grad_norm(d(x.clone()), 1e-3)

    keep = x.clone()
    with fw.dual_level():
        for call in calls(lambda t: fw.make_dual(t, torch.ones_like(t))):
            with pytest.raises(RuntimeError, match="forward-mode"):
                call()
        for requires in (False, True):
            with pytest.raises(RuntimeError, match="forward-mode"):
                T.linear(fw.make_dual(x.clone().requires_grad_(requires), torch.ones_like(x)), w, b)
        leaf = x.clone().requires_grad_(True)
        y = T.linear(leaf, w, b, activation="gelu")
        with pytest.raises(RuntimeError, match="forward-mode"):
            torch.autograd.grad(y, leaf, fw.make_dual(torch.ones_like(y), torch.ones_like(y)))
        assert torch.equal(T.linear(x, w, b), plain)       # tensors without a tangent go on as ever
        for call in calls(lambda t: t):
            call()
    assert torch.equal(x, keep)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("m,n,k", [(1, 13, 7), (1, 1, 1), (1, 1, 65), (40, 1, 33), (200, 1, 131), (1, 131, 33), (1, 4099, 515),
                                   (2, 3, 5), (33, 2, 3)])
def test_gradients_of_one_line_with_nan_behind_it(m, n, k, act, dt):
    # one row of x or of W: a summed axis of one, whose line ends inside a word
    x, w, dy, pre = (rnd(1, m, k, dt=dt), rnd(2, n, k, dt=dt, scale=0.2), rnd(3, m, n, dt=dt), rnd(4, m, n, dt=dt))
    refs, errs = U.linear_grad64(dy, x, w, pre, act)
    for left in (0, 8):
        put = lambda t: among_nan(t, left, 24)   # noqa: E731
        got = tss().linear_grad(put(dy), put(x), put(w), activation=act, pre=None if act == "none" else put(pre))
        for g, ref, err, what in zip(got, refs, errs, ("dx", "dw", "db")):
            U.within(g, ref, err, f"{what} {m}x{n}x{k} {act} {dt}")
