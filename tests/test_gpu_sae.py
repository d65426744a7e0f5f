"""A BatchTopK sparse autoencoder's training step out of the operators: encode
(product, relu, flattened top-k), decode, loss, backward, clipping.  Gradients
against a 64-bit step with the same selection, and against differences of the
loss; eager, captured and replayed."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def tss():
    import top_selection_sample_amd
    return top_selection_sample_amd


def model(dt, rows=96, d=64, n=700):
    g = torch.Generator().manual_seed(11)
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(dt).cuda()  # noqa: E731
    x = r(rows, d)
    return x, [r(n, d, scale=d ** -0.5), r(n, scale=0.05), r(n, d, scale=d ** -0.5), r(d, scale=0.1)]


def step(x, params, k):
    T = tss()
    we, be, wd, bd = params
    v, idx = T.encode(x, we, be, k)
    out = T.decode(v, idx, wd, rows=x.shape[0], bias=bd)
    loss = (out.float() - x.float()).square().mean()
    return loss, v, idx


def step64(x, params, idx):
    we, be, wd, bd = params
    acts = torch.relu(x @ we.t() + be)
    keep = torch.zeros_like(acts).reshape(-1)
    keep[idx] = 1
    out = (acts * keep.reshape(acts.shape)) @ wd + bd
    return (out - x).square().mean()


@pytest.mark.parametrize("dt,tol", [(torch.float32, 2e-5), (torch.bfloat16, 2e-2)])
def test_training_step(dt, tol):
    # tol: float32 sums of at most 700 terms over a few steps; in bfloat16 each of the four roundings on the way
    # (values, reconstruction, its gradient, the gradients) is off by up to 2^-8 of its value
    T = tss()
    x, params = model(dt)
    for p in params:
        p.requires_grad_(True)
    loss, _, idx = step(x, params, 96 * 16)
    loss.backward()
    ref = [p.detach().double().requires_grad_(True) for p in params]
    want = step64(x.double(), ref, idx)
    want.backward()
    assert abs(float(loss) - float(want)) <= tol * float(want)
    for p, q in zip(params, ref):
        assert float((p.grad.double() - q.grad).norm()) <= tol * float(q.grad.norm())
    before = [p.grad.clone() for p in params]
    norm = T.clip_grad_norm([p.grad for p in params], 0.01)
    total = torch.cat([b.double().reshape(-1) for b in before]).norm()
    assert abs(float(norm) - float(total)) <= 1e-6 * float(total)
    after = torch.cat([p.grad.double().reshape(-1) for p in params]).norm()
    assert float(after) <= 0.01 * (1 + tol)


def test_gradients_against_differences_of_the_loss():
    x, params = model(torch.float32)
    for p in params:
        p.requires_grad_(True)
    loss, _, idx = step(x, params, 96 * 16)
    grads = torch.autograd.grad(loss, params)
    g = torch.Generator().manual_seed(12)
    for i, gr in enumerate(grads):
        way = torch.randn(*gr.shape, generator=g).double().cuda()
        ends = []
        for s in (1e-6, -1e-6):   # the selection stays the one that was made: its gradient is defined so
            at = [p.detach().double() for p in params]
            at[i] = at[i] + s * way
            ends.append(float(step64(x.double(), at, idx)))
        want = (ends[0] - ends[1]) / 2e-6
        scale = float((gr.double() * way).abs().sum())
        assert abs(float((gr.double() * way).sum()) - want) <= 1e-4 * scale


def test_captured_step_next_to_eager_ones():
    # the whole step with the gradients as explicit calls, captured once and replayed with new inputs
    # between eager steps, whose autograd graphs stay alive meanwhile
    T = tss()
    x, params = model(torch.float32)
    we, be, wd, bd = params
    rows, k = x.shape[0], 96 * 8
    alive = [p.clone().requires_grad_(True) for p in params]
    held = step(x.clone(), alive, k)[0]

    def explicit():
        acts = T.linear(x, we, be, activation="relu")
        v, i = T.topk(acts.reshape(1, -1), k, params=T.default_params(seed=5, use_seed=1), workspace=ws)
        v, i = v[0], i[0]
        out = T.decode(v, i, wd, rows=rows, bias=bd)
        g = (out - x) * (2.0 / out.numel())
        dv, dwd, dbd = T.decode_grad(g, v, i, wd)
        dx, dwe, dbe = T.encode_grad(dv, v, i, x, we)
        grads = [dwe, dbe, dwd, dbd]
        return T.clip_grad_norm(grads, 0.01), grads

    ws = T.Workspace()
    explicit()
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        norm, grads = explicit()
    for s in range(3):
        x.copy_(torch.randn(*x.shape, generator=torch.Generator().manual_seed(20 + s)))
        cg.replay()
        torch.cuda.synchronize()
        want_norm, want = explicit()
        torch.cuda.synchronize()
        assert float(norm) == float(want_norm)
        for a, b in zip(grads, want):
            assert torch.equal(a, b)
        eager = [p.clone().requires_grad_(True) for p in params]
        step(x, eager, k)[0].backward()
        T.clip_grad_norm([p.grad for p in eager], 0.01)
        for a, p in zip(grads, eager):
            assert float((a - p.grad).norm()) <= 1e-5 * float(a.norm())
    held.backward()


def test_autograd_is_refused_under_capture():
    # a captured backward next to a live eager graph of the same leaves would end the process
    T = tss()
    x, params = model(torch.float32)
    we, be, wd, bd = params
    leaf = we.clone().requires_grad_(True)
    eager = T.linear(x, leaf)
    v, i = T.encode(x, we, be, 32)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for call in (lambda: T.linear(x, leaf), lambda: T.encode(x, leaf, be, 32),
                     lambda: T.decode(v, i, leaf, rows=x.shape[0])):
            with pytest.raises(RuntimeError, match="capture"):
                call()
        with torch.no_grad():
            out = T.linear(x, leaf)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    eager.sum().backward()
