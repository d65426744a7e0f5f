"""Refusals of the operators on a language model's selections, without a GPU:
every bad call returns its status before anything is enqueued (the addresses
here are made up and never followed), and the Python functions raise."""
import ctypes
import struct

import pytest

from top_selection_sample_amd import _lib

torch = pytest.importorskip("torch")
L = _lib.lib
OK, EINVAL, EDTYPE, EWORKSPACE = _lib.TOPK_OK, _lib.TOPK_EINVAL, _lib.TOPK_EDTYPE, _lib.TOPK_EWORKSPACE
A = 1 << 20   # an aligned address that is never followed
BIG = 1 << 50

FIELDS = {
    "dispatch": (_lib.DISPATCH_FORMAT, "x experts rows places offsets tokens k n_experts d ldx ldr dtype reserved",
                 dict(x=A, experts=A, rows=A, places=A, offsets=A, tokens=4, k=2, n_experts=8, d=16, ldx=16, ldr=16, dtype=1, reserved=0)),
    "combine": (_lib.COMBINE_FORMAT, "y places weights out tokens k n d ldy ldo dtype wdtype",
                dict(y=A, places=A, weights=A, out=A, tokens=4, k=2, n=8, d=16, ldy=16, ldo=16, dtype=2, wdtype=1)),
    "combine_grad": (_lib.COMBINE_GRAD_FORMAT, "grad y places weights dy dw tokens k n d ldg ldy lddy dtype wdtype",
                     dict(grad=A, y=A, places=A, weights=A, dy=A, dw=A, tokens=4, k=2, n=8, d=16, ldg=16, ldy=16, lddy=16, dtype=2, wdtype=2)),
    "attend": (_lib.ATTEND_FORMAT, "q k v lengths scores out b hq h n d sqb sqh skb skh skn svb svh svn ssb ssh sob soh scale dtype",
               dict(q=A, k=A, v=A, lengths=A, scores=A, out=A, b=2, hq=4, h=2, n=40, d=16, sqb=64, sqh=16, skb=1280, skh=640, skn=16,
                    svb=1280, svh=640, svn=16, ssb=80, ssh=40, sob=64, soh=16, scale=0.25, dtype=2)),
    "evict": (_lib.EVICT_FORMAT, "k v scores lengths ko vo so kept lo b h n d budget recent skb skh skn svb svh svn ssb ssh okb okh okn ovb ovh "
              "ovn osb osh dtype fill",
              dict(k=A, v=A, scores=A, lengths=A, ko=A, vo=A, so=A, kept=A, lo=A, b=2, h=2, n=40, d=16, budget=10, recent=4, skb=1280, skh=640,
                   skn=16, svb=1280, svh=640, svn=16, ssb=80, ssh=40, okb=320, okh=160, okn=16, ovb=320, ovh=160, ovn=16, osb=20, osh=10,
                   dtype=1, fill=1)),
    "sample": (_lib.SAMPLE_FORMAT, "z u tokens logprobs ts ks ps ms rows n ld top_k t p m dtype",
               dict(z=A, u=A, tokens=A, logprobs=A, ts=0, ks=0, ps=0, ms=0, rows=4, n=100, ld=100, top_k=5, t=1.0, p=0.9, m=0.0, dtype=1)),
}


def packed(name, **kw):
    fmt, names, base = FIELDS[name]
    v = {**base, **kw}
    return struct.pack(fmt, *(v[f] for f in names.split()))


def call(name, ws=A, size=BIG, **kw):
    a = packed(name, **kw)
    if name == "combine":
        return L.topk_combine(a, None)
    return getattr(L, "topk_" + name)(a, ws, size, None)


def need(name, **kw):
    out = ctypes.c_size_t()
    fmt, names, base = FIELDS[name]
    if name == "dispatch":
        v = {**base, **kw}
        return L.topk_dispatch_workspace_size(v["tokens"], v["k"], v["n_experts"], ctypes.byref(out)), out.value
    return getattr(L, f"topk_{name}_workspace_size")(packed(name, **kw), ctypes.byref(out)), out.value


BAD = [
    ("dispatch", dict(dtype=0), EDTYPE), ("dispatch", dict(tokens=-1), EINVAL), ("dispatch", dict(k=-1), EINVAL),
    ("dispatch", dict(tokens=1 << 20, k=1 << 12), EINVAL), ("dispatch", dict(n_experts=8193), EINVAL), ("dispatch", dict(n_experts=-1), EINVAL),
    ("dispatch", dict(d=1 << 22, ldx=1 << 22, ldr=1 << 22), EINVAL), ("dispatch", dict(ldx=15), EINVAL), ("dispatch", dict(ldr=15), EINVAL),
    ("dispatch", dict(x=0), EINVAL), ("dispatch", dict(rows=0), EINVAL), ("dispatch", dict(x=A + 2), EINVAL), ("dispatch", dict(experts=A + 4), EINVAL),
    ("dispatch", dict(places=0), EINVAL), ("dispatch", dict(offsets=0), EINVAL), ("dispatch", dict(offsets=0, tokens=0), EINVAL),
    ("combine", dict(dtype=0), EDTYPE), ("combine", dict(dtype=1, wdtype=2), EDTYPE), ("combine", dict(wdtype=0), EDTYPE),
    ("combine", dict(places=0), EINVAL), ("combine", dict(y=0), EINVAL), ("combine", dict(out=0), EINVAL), ("combine", dict(ldy=3), EINVAL),
    ("combine", dict(ldo=3), EINVAL), ("combine", dict(weights=A + 2), EINVAL), ("combine", dict(n=-1), EINVAL), ("combine", dict(d=-1), EINVAL),
    ("combine", dict(places=A + 2), EINVAL), ("combine", dict(n=1 << 31), EINVAL),
    ("combine_grad", dict(dtype=3), EDTYPE), ("combine_grad", dict(dy=0, dw=0), EINVAL), ("combine_grad", dict(grad=0), EINVAL),
    ("combine_grad", dict(y=0), EINVAL), ("combine_grad", dict(lddy=8), EINVAL), ("combine_grad", dict(ldg=8), EINVAL),
    ("combine_grad", dict(places=0), EINVAL), ("combine_grad", dict(dw=A + 1), EINVAL), ("combine_grad", dict(d=1 << 22), EINVAL),
    ("attend", dict(dtype=0), EDTYPE), ("attend", dict(d=257), EINVAL), ("attend", dict(d=-1), EINVAL), ("attend", dict(hq=5), EINVAL),
    ("attend", dict(h=0), EINVAL), ("attend", dict(n=-1), EINVAL), ("attend", dict(n=1 << 31), EINVAL), ("attend", dict(hq=2 * 4097), EINVAL),
    ("attend", dict(scale=float("nan")), EINVAL), ("attend", dict(scale=float("inf")), EINVAL), ("attend", dict(skn=-1), EINVAL),
    ("attend", dict(svb=(1 << 42) + 1), EINVAL), ("attend", dict(ssh=39), EINVAL), ("attend", dict(ssb=0), EINVAL), ("attend", dict(soh=15), EINVAL),
    ("attend", dict(sob=63), EINVAL), ("attend", dict(q=0), EINVAL), ("attend", dict(k=0), EINVAL), ("attend", dict(v=A + 1), EINVAL),
    ("attend", dict(out=0), EINVAL), ("attend", dict(scores=A + 2), EINVAL), ("attend", dict(lengths=A + 4), EINVAL), ("attend", dict(b=1 << 40), EINVAL),
    ("evict", dict(dtype=0), EDTYPE), ("evict", dict(budget=0), EINVAL), ("evict", dict(recent=11), EINVAL), ("evict", dict(recent=-1), EINVAL),
    ("evict", dict(okn=15), EINVAL), ("evict", dict(okh=159), EINVAL), ("evict", dict(ovb=0), EINVAL), ("evict", dict(osh=9), EINVAL),
    ("evict", dict(k=0), EINVAL), ("evict", dict(ko=0), EINVAL), ("evict", dict(so=0), EINVAL), ("evict", dict(kept=0), EINVAL),
    ("evict", dict(lo=0), EINVAL), ("evict", dict(lengths=A + 4), EINVAL), ("evict", dict(d=1 << 22), EINVAL), ("evict", dict(skb=-1), EINVAL),
    ("evict", dict(v=A + 2), EINVAL), ("evict", dict(scores=0), EINVAL),
    ("sample", dict(dtype=0), EDTYPE), ("sample", dict(n=0), EINVAL), ("sample", dict(n=(1 << 24) + 1, ld=1 << 25), EINVAL), ("sample", dict(rows=-1), EINVAL),
    ("sample", dict(ld=99), EINVAL), ("sample", dict(z=0), EINVAL), ("sample", dict(u=0), EINVAL), ("sample", dict(tokens=0), EINVAL),
    ("sample", dict(logprobs=A + 2), EINVAL), ("sample", dict(ts=A + 2), EINVAL), ("sample", dict(ks=A + 4), EINVAL), ("sample", dict(ps=A + 1), EINVAL),
    ("sample", dict(ms=A + 3), EINVAL),
]


@pytest.mark.parametrize("name,kw,want", BAD)
def test_refusals(name, kw, want):
    assert call(name, **kw) == want


@pytest.mark.parametrize("name", ["dispatch", "combine_grad", "attend", "sample"])
def test_workspace(name):
    kw = dict(tokens=5000) if name == "dispatch" else {}
    rc, size = need(name, **kw)
    assert rc == OK and size > 0
    assert call(name, size=size - 1, **kw) == EWORKSPACE
    assert call(name, ws=None, size=size, **kw) == EINVAL
    assert call(name, ws=A + 16, size=size, **kw) == EINVAL
    if name != "dispatch":
        assert getattr(L, f"topk_{name}_workspace_size")(None, ctypes.byref(ctypes.c_size_t())) == EINVAL
        assert getattr(L, f"topk_{name}_workspace_size")(packed(name), None) == EINVAL
    assert getattr(L, "topk_" + name)(None, None, 0, None) == EINVAL


def test_sizes_that_are_taken():
    assert need("dispatch", tokens=0) == (OK, 0)
    assert need("dispatch", tokens=0, n_experts=8192)[0] == OK
    assert need("dispatch", n_experts=0)[0] == OK
    assert need("dispatch", tokens=(1 << 31) - 1, k=1)[0] == OK
    assert need("evict", b=0)[0] == OK
    assert need("attend", scores=0, ssb=0, ssh=0)[0] == OK
    assert need("attend", b=1, ssb=0)[0] == OK                       # one sequence: its stride is not looked at
    assert need("attend", ssb=40, ssh=80)[0] == OK                   # heads outermost
    assert need("attend", skh=0, svn=0)[0] == OK                     # inputs may be expanded
    assert need("attend", n=0)[0] == OK
    assert need("evict", okb=160, okh=320)[0] == OK
    assert need("evict", okb=320, okn=32, okh=16)[0] == OK           # [b, n, h, d]
    assert need("sample", rows=0) == (OK, 0)
    assert need("combine_grad", weights=0, dw=0, y=0)[0] == OK
    assert L.topk_combine(None, None) == EINVAL
    assert L.topk_evict(None, None, 0, None) == EINVAL
    assert L.topk_dispatch_workspace_size(4, 2, 8, None) == EINVAL


def test_python_refusals_on_the_cpu():
    import top_selection_sample_amd as tss
    x, e = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64)
    q, k = torch.zeros(1, 2, 8), torch.zeros(1, 1, 4, 8)
    for f in (lambda: tss.dispatch(x, e, 4), lambda: tss.combine(x, e), lambda: tss.combine_grad(x, x, e), lambda: tss.attend(q, k, k),
              lambda: tss.evict(k, k, torch.zeros(1, 1, 4), 2), lambda: tss.sample(x, torch.zeros(4))):
        with pytest.raises(ValueError, match="GPU tensor"):
            f()
