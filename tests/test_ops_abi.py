"""Refusals of the operators around the selection, without a GPU: every bad
call returns its status before anything is enqueued (the addresses here are
made up and never followed), and the Python functions raise."""
import ctypes
import math

import pytest

from top_selection_sample_amd import _lib

torch = pytest.importorskip("torch")
L = _lib.lib
OK, EINVAL, EDTYPE, EWORKSPACE = _lib.TOPK_OK, _lib.TOPK_EINVAL, _lib.TOPK_EDTYPE, _lib.TOPK_EWORKSPACE
A = 1 << 20   # an aligned address that is never followed


def linear_args(**kw):
    a = dict(x=A, w=A, bias=None, residual=None, y=A, pre=None, m=8, n=16, k=32, ldx=32, ldw=32, ldr=0, ldy=16, ldp=0,
             dtype=2, act=0, x_trans=0, w_trans=0)
    a.update(kw)
    return _lib.LinearArgs(**a)


def grad_args(**kw):
    a = dict(dy=A, pre=A, x=A, w=A, dx=A, dw=A, db=A, m=8, n=16, k=32, ldd=16, ldp=16, ldx=32, ldw=32, lddx=32, lddw=32,
             dtype=1, act=1, x_trans=0, w_trans=0)
    a.update(kw)
    return _lib.LinearGradArgs(**a)


def size_of(fn, a):
    out = ctypes.c_size_t()
    return fn(ctypes.byref(a), ctypes.byref(out)), out.value


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=0), EDTYPE), (dict(dtype=7), EDTYPE), (dict(act=4), EINVAL), (dict(act=-1), EINVAL),
    (dict(m=-1), EINVAL), (dict(n=1 << 31), EINVAL), (dict(k=-5), EINVAL), (dict(x=None), EINVAL), (dict(w=None), EINVAL),
    (dict(y=None), EINVAL), (dict(ldx=31), EINVAL), (dict(ldw=1), EINVAL), (dict(ldy=15), EINVAL), (dict(ldx=-32), EINVAL),
    (dict(x=A + 1), EINVAL), (dict(bias=A + 1), EINVAL), (dict(residual=A, ldr=3), EINVAL), (dict(pre=A, ldp=0), EINVAL),
    (dict(x_trans=1, ldx=7), EINVAL), (dict(w_trans=1, ldw=15), EINVAL), (dict(dtype=1, y=A + 2), EINVAL),
    (dict(ldy=1 << 31), EINVAL), (dict(k=1 << 22, ldx=1 << 22, ldw=1 << 22), EINVAL), (dict(n=1 << 22, ldy=1 << 22), EINVAL),
    (dict(x_trans=1, m=1 << 22, ldx=1 << 22), EINVAL), (dict(m=(1 << 31) - 1, n=1 << 12, ldy=1 << 12), EINVAL)])
def test_linear_refusals(kw, want):
    a = linear_args(**kw)
    assert size_of(L.topk_linear_workspace_size, a)[0] == want
    assert L.topk_linear(ctypes.byref(a), A, 1 << 40, None) == want


def test_linear_sizes_that_are_taken():
    for kw in (dict(), dict(m=0), dict(n=0), dict(k=0), dict(x_trans=1, ldx=8), dict(w_trans=1, ldw=16), dict(m=1, ldx=0, ldy=0),
               dict(dtype=1), dict(x=A + 2), dict(x=None, m=0), dict(residual=A, ldr=16), dict(pre=A, ldp=20)):
        assert size_of(L.topk_linear_workspace_size, linear_args(**kw))[0] == OK, kw
    assert L.topk_linear_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == EINVAL
    assert L.topk_linear_workspace_size(ctypes.byref(linear_args()), None) == EINVAL
    assert L.topk_linear(None, None, 0, None) == EINVAL


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=0), EDTYPE), (dict(act=9), EINVAL), (dict(dx=None, dw=None, db=None), EINVAL), (dict(dy=None), EINVAL),
    (dict(pre=None), EINVAL), (dict(ldp=15), EINVAL), (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(ldd=2), EINVAL),
    (dict(lddx=31), EINVAL), (dict(lddw=0), EINVAL), (dict(db=A + 2), EINVAL), (dict(m=-2), EINVAL), (dict(x_trans=1, ldx=7), EINVAL)])
def test_linear_grad_refusals(kw, want):
    a = grad_args(**kw)
    assert size_of(L.topk_linear_grad_workspace_size, a)[0] == want
    assert L.topk_linear_grad(ctypes.byref(a), A, 1 << 40, None) == want


def test_linear_grad_workspace():
    # dz and the column sums need scratch: a call with too little of it, or at a bad address, is refused
    a = grad_args(m=600)
    rc, need = size_of(L.topk_linear_grad_workspace_size, a)
    assert rc == OK and need > 0
    assert L.topk_linear_grad(ctypes.byref(a), A, need - 1, None) == EWORKSPACE
    assert L.topk_linear_grad(ctypes.byref(a), None, need, None) == EINVAL
    assert L.topk_linear_grad(ctypes.byref(a), A + 16, need, None) == EINVAL
    for kw in (dict(x=None, dw=None), dict(w=None, dx=None), dict(act=0, pre=None), dict(dx=None, db=None)):
        assert size_of(L.topk_linear_grad_workspace_size, grad_args(**kw))[0] == OK


def sel(**kw):
    a = dict(values=A, indices=A, rows=4, k=40, n=64, flat=1, dtype=1)
    a.update(kw)
    return _lib.Selection(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=0), EDTYPE), (dict(dtype=3), EDTYPE), (dict(rows=-1), EINVAL), (dict(k=-1), EINVAL), (dict(n=1 << 31), EINVAL),
    (dict(values=None), EINVAL), (dict(indices=None), EINVAL), (dict(indices=A + 4), EINVAL), (dict(values=A + 2), EINVAL),
    (dict(flat=0, rows=1 << 20, k=1 << 20), EINVAL), (dict(n=1 << 28), EINVAL), (dict(rows=1 << 28), EINVAL)])
def test_selection_refusals(kw, want):
    s = ctypes.byref(sel(**kw))
    assert L.topk_decode(s, A, 64, 64, None, A, 64, A, 1 << 40, None) == want
    assert L.topk_decode_grad(s, A, 64, 64, A, 64, A, A, 64, A, A, 1 << 40, None) == want
    assert L.topk_encode_grad(s, A, A, 64, A, 64, 64, A, 64, A, 64, A, A, 1 << 40, None) == want


def test_decode_refusals():
    s = ctypes.byref(sel())
    size = ctypes.c_size_t()
    assert L.topk_decode_workspace_size(s, 64, ctypes.byref(size)) == OK
    assert L.topk_decode_workspace_size(s, 64, None) == EINVAL
    assert L.topk_decode_workspace_size(s, -1, ctypes.byref(size)) == EINVAL
    assert L.topk_decode_workspace_size(s, 1 << 22, ctypes.byref(size)) == EINVAL
    assert L.topk_decode_workspace_size(None, 64, ctypes.byref(size)) == EINVAL
    big = 1 << 40
    for args in ((None, 64, 64, None, A, 64), (A, 63, 64, None, A, 64), (A, 64, -1, None, A, 64), (A, 64, 64, A + 1, A, 64),
                 (A, 64, 64, None, None, 64), (A, 64, 64, None, A, 60), (A + 2, 64, 64, None, A, 64)):
        assert L.topk_decode(s, *args, A, big, None) == EINVAL
    assert L.topk_decode_grad(s, A, 64, 64, None, 64, A, A, 64, A, A, big, None) == EINVAL
    assert L.topk_decode_grad(s, A, 64, 64, A, 64, None, None, 64, None, A, big, None) == EINVAL
    assert L.topk_decode_grad(s, None, 64, 64, A, 64, A, None, 64, None, A, big, None) == EINVAL
    assert L.topk_decode_grad(s, A, 64, 64, A, 64, None, A, 9, None, A, big, None) == EINVAL
    assert L.topk_decode_grad(s, A, 64, 64, A, 64, None, None, 0, A, None, 0, None) == EINVAL   # no workspace
    assert L.topk_decode_grad(s, A, 64, 64, A, 64, None, None, 0, A, A, 8, None) == EWORKSPACE
    assert L.topk_encode_grad(s, None, A, 64, A, 64, 64, A, 64, A, 64, A, A, big, None) == EINVAL
    assert L.topk_encode_grad(s, A, A, 64, A, 64, 64, None, 64, None, 64, None, A, big, None) == EINVAL
    assert L.topk_encode_grad(s, A, None, 64, A, 64, 64, A, 64, A, 64, A, A, big, None) == EINVAL
    assert L.topk_encode_grad(s, A, A, 64, None, 64, 64, A, 64, A, 64, A, A, big, None) == EINVAL


def test_norm_refusals():
    P, I, D = (ctypes.c_void_p * 2), (ctypes.c_int64 * 2), (ctypes.c_int32 * 2)
    ok = (P(A, A + 4096), I(100, 5), D(1, 2), 2)
    size = ctypes.c_size_t()
    assert L.topk_grad_norm_workspace_size(2, ok[1], ctypes.byref(size)) == OK and size.value > 0
    assert L.topk_grad_norm_workspace_size(2, ok[1], None) == EINVAL
    assert L.topk_grad_norm_workspace_size(2, I(-1, 3), ctypes.byref(size)) == EINVAL
    assert L.topk_grad_norm_workspace_size(-1, ok[1], ctypes.byref(size)) == EINVAL
    big = 1 << 40

    def both(args, want, norm=A, ws=A, have=big):
        assert L.topk_grad_norm(*args, norm, ws, have, None) == want
        assert L.topk_clip_grad_norm(*args, 1.0, 1e-6, norm, ws, have, None) == want

    both((P(A, A + 4096), I(100, 5), D(1, 0), 2), EDTYPE)
    both((P(A + 2, A + 4096), I(100, 5), D(1, 2), 2), EINVAL)
    both((P(None, A + 4096), I(100, 5), D(1, 2), 2), EINVAL)
    both((None, ok[1], ok[2], 2), EINVAL)
    both((ok[0], ok[1], None, 2), EINVAL)
    both(ok, EINVAL, norm=None)
    both(ok, EINVAL, norm=A + 2)
    both(ok, EINVAL, ws=None)
    both(ok, EINVAL, ws=A + 8)
    both(ok, EWORKSPACE, have=size.value - 1)
    for m, e in ((-1.0, 1e-6), (math.nan, 1e-6), (1.0, -1e-6), (1.0, math.nan)):
        assert L.topk_clip_grad_norm(*ok, m, e, A, A, big, None) == EINVAL
    # overlapping tensors cannot be scaled
    assert L.topk_clip_grad_norm(P(A, A + 396), I(100, 5), D(1, 2), 2, 1.0, 1e-6, A, A, big, None) == EINVAL
    assert L.topk_clip_grad_norm(P(A, A), I(100, 100), D(1, 1), 2, 1.0, 1e-6, A, A, big, None) == EINVAL


def test_python_refusals():
    import top_selection_sample_amd as tss
    x, w = torch.zeros(3, 4), torch.zeros(5, 4)
    for call in (lambda: tss.linear(x, w), lambda: tss.linear_grad(x, x, w), lambda: tss.encode(x, w, None, 2),
                 lambda: tss.decode(x[0], torch.zeros(4, dtype=torch.int64), w, rows=1),
                 lambda: tss.decode_grad(x, x[0], torch.zeros(4, dtype=torch.int64), w),
                 lambda: tss.encode_grad(x[0], x[0], torch.zeros(4, dtype=torch.int64), x, w),
                 lambda: tss.grad_norm([x]), lambda: tss.clip_grad_norm([x], 1.0)):
        with pytest.raises(ValueError):
            call()


def test_tensors_with_a_tangent_are_refused():
    import torch.autograd.forward_ad as fw
    from top_selection_sample_amd import _ops
    x, w = torch.zeros(3, 4), torch.zeros(5, 4)
    assert not _ops._wants_grad(x, None, w)
    with fw.dual_level():
        d = fw.make_dual(x, torch.ones(3, 4))
        assert not _ops._wants_grad(x, None, w)
        for call in (lambda: _ops._wants_grad(w, d), lambda: _ops._wants_grad(None, w.requires_grad_(True), d),
                     lambda: _ops._linear_grad_run(d, x, w, 0, None, (True, True, True)),
                     lambda: _ops._decode_grad_run(x, x, x, d, (True, True, True)),
                     lambda: _ops._encode_grad_run(d, x, x, x, w, (True, True, True)),
                     lambda: _ops._norm_run([x, d], None), lambda: _ops._norm_run(d, (1.0, 1e-6))):
            with pytest.raises(RuntimeError, match="forward-mode"):
                call()
        with fw._set_fwd_grad_enabled(False):
            assert not _ops._wants_grad(d)


def test_a_residual_in_place_has_the_strides_of_the_result():
    for kw, want in ((dict(residual=A, ldr=17), EINVAL), (dict(residual=A, ldr=16, ldy=20), EINVAL), (dict(residual=A, ldr=16), OK),
                     (dict(residual=A, ldr=20, ldy=20), OK), (dict(residual=A, ldr=99, m=1), OK), (dict(residual=A, ldr=9, m=0), OK),
                     (dict(residual=A, ldr=9, n=0), OK), (dict(residual=2 * A, ldr=17), OK)):
        assert size_of(L.topk_linear_workspace_size, linear_args(**kw))[0] == want, kw
        if want != OK:
            assert L.topk_linear(ctypes.byref(linear_args(**kw)), A, 1 << 40, None) == want
