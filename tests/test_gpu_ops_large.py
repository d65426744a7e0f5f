"""GPU: operators at strides, rows and entries near the ends of their ranges."""
import pytest
import torch

import ops_util as U
from top_selection_sample_amd import decode, decode_grad, linear, linear_grad

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("strided", ["x", "weight"])
def test_rows_of_a_tile_spread_over_more_than_2_31_bytes(strided):
    g = torch.Generator("cuda").manual_seed(3)
    big, few, k, ld = 512, 32768, 64, 5_000_000
    wide = torch.empty(big * ld, dtype=torch.bfloat16, device="cuda").as_strided((big, k), (ld, 1))
    wide.copy_(torch.randn(big, k, device="cuda", generator=g))
    other = torch.randn(few, k, device="cuda", generator=g).bfloat16()
    y = linear(wide, other) if strided == "x" else linear(other, wide).T
    ref = wide.double() @ other.double().T
    bound = (wide.double().abs() @ other.double().abs().T) * (k * 2.0 ** -24) + ref.abs() * 2.0 ** -8
    assert ((y.double() - ref).abs() <= bound).all()


def test_more_rows_than_one_grid_dimension_of_tiles_holds():
    """2^24 tiles of 64 rows and 2^30 rows to pack; each output is one product, rounded once."""
    m = (1 << 30) + 70
    x = torch.randn(m, 1, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    w = torch.tensor([[1.25]], device="cuda")
    y = linear(x, w)
    assert torch.equal(y, x * 1.25)


def test_decode_of_more_rows_than_one_grid_dimension_holds():
    rows, n, d = (1 << 24) + 5, 100, 8
    g = torch.Generator("cuda").manual_seed(5)
    values = torch.randn(rows, 1, device="cuda", generator=g)
    indices = torch.randint(0, n, (rows, 1), device="cuda", generator=g)
    weight = torch.randn(n, d, device="cuda", generator=g)
    assert torch.equal(decode(values, indices, weight), values * weight[indices[:, 0]])


def test_dots_of_more_entries_than_one_grid_dimension_holds():
    rows, k, n = (1 << 15) + 1, 1 << 14, 100
    g = torch.Generator("cuda").manual_seed(6)
    values = torch.ones(rows, k, device="cuda", dtype=torch.bfloat16)
    indices = torch.randint(0, n, (rows, k), device="cuda", generator=g)
    weight = torch.randint(-8, 8, (n, 1), device="cuda", generator=g).bfloat16()
    grad = torch.randint(-8, 8, (rows, 1), device="cuda", generator=g).bfloat16()
    dv = decode_grad(grad, values, indices, weight, (True, False, False))[0]
    for at in range(0, rows, 4096):   # products of small whole numbers are exact
        assert torch.equal(dv[at:at + 4096], grad[at:at + 4096] * weight[indices[at:at + 4096], 0])


def test_gradient_of_the_most_latents():
    n, d = (1 << 28) - 1, 1
    indices = torch.tensor([[0, 5, n - 1], [n - 1, n, -1]], device="cuda")
    values = torch.tensor([[1.0, 2.0, 3.0], [4.0, 5.0, 6.0]], device="cuda", dtype=torch.bfloat16)
    grad = torch.tensor([[2.0], [8.0]], device="cuda", dtype=torch.bfloat16)
    weight = torch.zeros(n, d, device="cuda", dtype=torch.bfloat16)
    dw = decode_grad(grad, values, indices, weight, (False, True, False))[1]
    at = torch.nonzero(dw[:, 0])[:, 0]
    assert at.tolist() == [0, 5, n - 1]
    assert dw[at, 0].tolist() == [2.0, 4.0, 6.0 + 32.0]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1001, 4099, 515), (1024, 4160, 512), (2100, 2200, 2048), (1090, 8200, 520), (4200, 4352, 1024)])
def test_tiles_behind_the_last_full_round(m, n, k, dt):
    # those are split along the summed axis and joined, the others are not
    g = torch.Generator().manual_seed(8)
    draw = lambda *shape, scale=1.0: (torch.randn(*shape, generator=g) * scale).to(DT[dt]).cuda()
    x, w, b, r = draw(m, k), draw(n, k, scale=k ** -0.5), draw(n), draw(m, n)
    want = U.linear64(x, w, b, "silu", r)
    xt, wt = x.t().contiguous().t(), w.t().contiguous().t()
    for xx, ww in ((x, w), (x, wt), (xt, w), (xt, wt)):
        U.within(linear(xx, ww, b, "silu", r), want[0], want[1], f"{m}x{n}x{k}")
    assert torch.equal(linear(x, w, b, "silu", r), linear(x, w, b, "silu", r))
    dy = draw(m, n)
    refs, errs = U.linear_grad64(dy, x, w, r, "gelu")
    for got, ref, err in zip(linear_grad(dy, x, w, activation="gelu", pre=r), refs, errs):
        U.within(got, ref, err, f"gradient {m}x{n}x{k}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 16, 4096), (16, 300, 8191), (3, 4097, 2049), (31, 65, 4095), (17, 40, 1025),
                                   (33, 64, 8192), (20, 7, 100_000), (129, 65, 20_001)])
def test_deep_products_of_few_rows(m, n, k, dt):
    g = torch.Generator().manual_seed(9)
    draw = lambda *shape, scale=1.0: (torch.randn(*shape, generator=g) * scale).to(DT[dt]).cuda()
    x, w, b, r = draw(m, k), draw(n, k, scale=k ** -0.5), draw(n), draw(m, n)
    want = U.linear64(x, w, b, "gelu", r)
    U.within(linear(x, w, b, "gelu", r), want[0], want[1], f"{m}x{n}x{k}")
    dy = draw(m, n)
    refs, errs = U.linear_grad64(dy, x, w, r, "relu")
    for got, ref, err in zip(linear_grad(dy, x, w, activation="relu", pre=r), refs, errs):
        U.within(got, ref, err, f"gradient {m}x{n}x{k}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(3067, 4686), (2100, 4103), (2500, 4161), (600, 1031), (70, 69), (130, 129)])
def test_last_columns_and_a_residual_in_place(m, n, dt):
    k = 64
    g = torch.Generator().manual_seed(10)
    draw = lambda *shape, scale=1.0: (torch.randn(*shape, generator=g) * scale).to(DT[dt]).cuda()
    x, w, b, r = draw(m, k), draw(n, k, scale=0.2), draw(n), draw(m, n)
    want = U.linear64(x, w, b, "silu", r)
    U.within(linear(x, w, b, "silu", r), want[0], want[1], f"{m}x{n}")
    import ctypes
    from top_selection_sample_amd import _lib, dtype_code
    y = r.clone()
    a = _lib.LinearArgs(x.data_ptr(), w.data_ptr(), b.data_ptr(), y.data_ptr(), y.data_ptr(), None, m, n, k, k, k, n, n, n,
                        dtype_code(DT[dt]), _lib.ACTIVATIONS["silu"], 0, 0)
    size = ctypes.c_size_t()
    assert _lib.lib.topk_linear_workspace_size(ctypes.byref(a), ctypes.byref(size)) == 0
    ws = torch.empty(size.value + 1, dtype=torch.uint8, device="cuda")
    assert _lib.lib.topk_linear(ctypes.byref(a), ws.data_ptr(), size.value, torch.cuda.current_stream().cuda_stream) == 0
    U.within(y, want[0], want[1], f"in place {m}x{n}")


def test_few_columns_of_more_rows_than_a_second_grid_dimension_holds():
    # 32 rows to a workgroup: more than 65536 of them
    m = (1 << 21) + 70
    g = torch.Generator("cuda").manual_seed(11)
    x = torch.randint(-8, 8, (m, 3), device="cuda", generator=g).bfloat16()
    w = torch.randint(-8, 8, (2, 3), device="cuda", generator=g).bfloat16()
    assert torch.equal(linear(x, w), (x.float()[:, None, :] * w.float()[None]).sum(2).bfloat16())


def test_tiles_beyond_one_grid_dimension():
    """2^22 + 2 tiles of 64 rows.  Aligned operands of more than 32 rows take the tiles, whatever
    the estimates for unaligned ones say; of one step and one column the smallest are cheapest."""
    m, k = (1 << 28) + 70, 8
    g = torch.Generator("cuda").manual_seed(12)
    x = torch.randint(-8, 8, (m, k), device="cuda", generator=g, dtype=torch.bfloat16)
    w = torch.randint(-8, 8, (1, k), device="cuda", generator=g, dtype=torch.bfloat16)
    assert x.data_ptr() % 16 == 0 and w.data_ptr() % 16 == 0
    y = linear(x, w)
    for at in range(0, m, 1 << 25):   # sums of small whole numbers are exact, and rounded once
        part = x[at:at + (1 << 25)]
        assert torch.equal(y[at:at + (1 << 25)], (part.float() * w.float()).sum(1, keepdim=True).bfloat16())


def test_copies_beyond_one_grid_dimension():
    """More than 2^30 16-byte pieces to copy, 256 to a workgroup, for rows of odd length that are
    too long for the kernel that reads them as they lie."""
    import ctypes
    from top_selection_sample_amd import _lib, dtype_code
    k, padded = 4097, 4104
    m = (1 << 30) // (padded // 8) + 38
    g = torch.Generator("cuda").manual_seed(13)
    x = torch.randint(-2, 3, (m, k), device="cuda", generator=g, dtype=torch.bfloat16)
    w = torch.randint(-2, 3, (1, k), device="cuda", generator=g, dtype=torch.bfloat16)
    a = _lib.LinearArgs(x.data_ptr(), w.data_ptr(), None, None, w.data_ptr(), None, m, 1, k, k, k, 0, 1, 0,
                        dtype_code(torch.bfloat16), 0, 0, 0)
    size = ctypes.c_size_t()
    assert _lib.lib.topk_linear_workspace_size(ctypes.byref(a), ctypes.byref(size)) == 0
    assert m * (padded // 8) > (1 << 30) and size.value >= m * padded * 2     # the copy is made
    y = linear(x, w)
    for at in range(0, m, 1 << 16):   # whole numbers below 2^24: exact in any order, and rounded once
        assert torch.equal(y[at:at + (1 << 16)], (x[at:at + (1 << 16)].float() @ w.float().t()).bfloat16())


def test_more_rows_by_columns_than_a_product_reads_in_place():
    # x stored by columns, 2^22 rows and more: read through a copy
    m, n, k = (1 << 22) + 5, 3, 8
    g = torch.Generator("cuda").manual_seed(14)
    x = torch.randint(-8, 8, (k, m), device="cuda", generator=g, dtype=torch.bfloat16).t()
    w = torch.randint(-8, 8, (n, k), device="cuda", generator=g, dtype=torch.bfloat16)
    assert torch.equal(linear(x, w), (x.float() @ w.float().t()).bfloat16())   # exact, and rounded once
    dy = torch.randint(-1, 2, (m, n), device="cuda", generator=g, dtype=torch.bfloat16)
    dx, dw, db = linear_grad(dy, x, w)
    assert torch.equal(dx, (dy.float() @ w.float()).bfloat16())
    # whole numbers below 2^24 on the way (random signs): exact in any order
    assert torch.equal(dw, (dy.double().t().contiguous() @ x.double()).bfloat16())
    assert torch.equal(db, dy.double().sum(0).bfloat16())


def test_rows_further_apart_than_2_31_elements():
    # two rows of a matrix too wide to be named by its stride: read through a copy
    ld, k, n = (1 << 31) + 24, 40, 5
    g = torch.Generator("cuda").manual_seed(15)
    x = torch.empty(2 * ld, dtype=torch.bfloat16, device="cuda").as_strided((2, k), (ld, 1))
    x.copy_(torch.randint(-8, 8, (2, k), device="cuda", generator=g))
    w = torch.randint(-8, 8, (n, k), device="cuda", generator=g, dtype=torch.bfloat16)
    want = (x.float() @ w.float().t()).bfloat16()
    assert torch.equal(linear(x, w), want) and torch.equal(linear(w, x), want.t())
    values, indices = torch.ones(1, 2, dtype=torch.bfloat16, device="cuda"), torch.tensor([[1, 0]], device="cuda")
    assert torch.equal(decode(values, indices, x), x.float().sum(0, keepdim=True).bfloat16())
