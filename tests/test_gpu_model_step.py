"""The operators on a language model's selections together, as they are used:
decoding steps with a cache that is cut, experts and a drawn token, eager and
as a replayed graph; and a training step through a router's selection."""
import pytest

import model_util as M
import ops_util as U

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def tss():
    import top_selection_sample_amd
    return top_selection_sample_amd


def rnd(seed, *shape, dt=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dt).cuda()


class Model:
    """One layer: attention over a cache, eight experts, a vocabulary of 1003."""

    def __init__(self, b, dt):
        self.b, self.hq, self.h, self.d, self.e, self.n = b, 8, 2, 32, 8, 96
        wide = self.hq * self.d
        self.wide = wide
        self.wq = rnd(1, wide, wide, dt=dt, scale=wide ** -0.5)
        self.wk, self.wv = (rnd(s, self.h * self.d, wide, dt=dt, scale=wide ** -0.5) for s in (2, 3))
        self.router = rnd(4, self.e, wide, dt=dt, scale=wide ** -0.5)
        self.up = rnd(5, self.e, 64, wide, dt=dt, scale=wide ** -0.5)
        self.down = rnd(6, self.e, wide, 64, dt=dt, scale=0.125)
        self.head = rnd(7, 1003, wide, dt=dt, scale=wide ** -0.5)
        self.words = rnd(8, 1003, wide, dt=dt)
        self.k = torch.zeros(b, self.h, self.n, self.d, dtype=dt, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.scores = torch.zeros(b, self.h, self.n, device="cuda")
        self.lengths = torch.zeros(b, dtype=torch.int64, device="cuda")
        self.token = torch.zeros(b, dtype=torch.int64, device="cuda")
        self.u = torch.zeros(b, device="cuda")
        self.nothing = torch.zeros(b, self.h, device="cuda")
        self.ws = tss().Workspace()

    def step(self):
        T = tss()
        x = self.words[self.token]
        at = torch.arange(self.b, device="cuda")
        self.k[at, :, self.lengths] = T.linear(x, self.wk).reshape(self.b, self.h, self.d)
        self.v[at, :, self.lengths] = T.linear(x, self.wv).reshape(self.b, self.h, self.d)
        self.scores[at, :, self.lengths] = self.nothing
        self.lengths.add_(1)
        q = T.linear(x, self.wq).reshape(self.b, self.hq, self.d)
        x = x + T.attend(q, self.k, self.v, self.lengths, self.scores).reshape(self.b, -1)
        value, expert = T.topk(T.linear(x, self.router), 2, workspace=self.ws)
        rows, places, offsets = T.dispatch(x, expert, self.e)
        # a step of few tokens takes every expert over all rows, and keeps its own
        of = (torch.arange(rows.shape[0], device="cuda")[:, None] >= offsets[1:]).sum(1)
        y = torch.zeros_like(rows)
        for e in range(self.e):
            y = torch.where((of == e)[:, None], T.linear(T.linear(rows, self.up[e], activation="silu"), self.down[e]), y)
        x = x + T.combine(y, places, torch.softmax(value.float(), 1))
        token, logprob = T.sample(T.linear(x, self.head), self.u, temperature=0.8, top_k=40, top_p=0.95)
        self.token.copy_(token)
        return x, expert, places, offsets, token, logprob

    def cut(self):
        k, v, s, kept, lengths = tss().evict(self.k, self.v, self.scores, 40, recent=8, lengths=self.lengths)
        self.k[:, :, :40], self.v[:, :, :40], self.scores[:, :, :40] = k, v, s
        self.lengths.copy_(lengths)
        return kept

    def state(self):
        return [t.clone() for t in (self.k, self.v, self.scores, self.lengths, self.token)]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_decoding(dt):
    with torch.no_grad():
        a, b = Model(5, dt), Model(5, dt)
        for m in (a, b):
            m.step()
            m.cut()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b.step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = b.step()
        a.step()
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x, y)
        drawn = set()
        for i in range(120):
            u = torch.rand(5, generator=torch.Generator().manual_seed(i)).cuda()
            a.u.copy_(u)
            b.u.copy_(u)
            before = [t.clone() for t in (a.k, a.v, a.scores, a.lengths)]
            got = a.step()
            graph.replay()
            torch.cuda.synchronize()
            for x, y in zip(got, held):
                assert torch.equal(x, y), i
            drawn.update(got[4].tolist())
            if i % 30 == 7:      # the weights that were added are those of a softmax: a group's heads add 1 each
                added = (a.scores.double() - before[2].double()).cpu()
                for r in range(5):
                    e = int(a.lengths[r])
                    added[r, :, e - 1] = a.scores[r, :, e - 1].cpu().double()
                    # 4 heads' probabilities, each entry's sum rounded at scores below 200
                    assert bool(((added[r, :, :e].sum(1) - 4).abs() <= 1e-4 + e * 200 * U.U32).all())
            if int(a.lengths.max()) == a.n:
                scores, lengths = a.scores.clone(), a.lengths.clone()
                kept = a.cut()
                assert torch.equal(kept.cpu(), M.evict64(scores, lengths, 40, 8)[0])
                assert torch.equal(kept, b.cut()) and int(a.lengths.max()) == 40
            for x, y in zip(a.state(), b.state()):
                assert torch.equal(x, y), i
        assert len(drawn) > 20


def test_training_through_experts():
    """x -> router -> two experts each -> weighted sum -> loss; gradients against torch in 64 bits."""
    T = tss()
    t, d, e = 300, 48, 6
    x0, w0, r0, target = rnd(1, t, d), rnd(2, e, d, d, scale=d ** -0.5), rnd(3, e, d, scale=d ** -0.5), rnd(4, t, d)
    x, w, r = (v.clone().requires_grad_() for v in (x0, w0, r0))
    logits = T.linear(x, r)
    expert = T.topk(logits.detach(), 2)[1]
    gate = torch.softmax(logits.gather(1, expert), 1)
    rows, places, offsets = T.dispatch(x, expert, e)
    at = offsets.tolist()
    y = torch.cat([T.linear(rows[at[i]:at[i + 1]], w[i], activation="silu") for i in range(e)])
    loss = (T.combine(y, places, gate) - target).square().mean()
    loss.backward()
    x64, w64, r64 = (v.cpu().double().requires_grad_() for v in (x0, w0, r0))
    pick = expert.cpu()
    gate64 = torch.softmax((x64 @ r64.t()).gather(1, pick), 1)
    every = torch.nn.functional.silu(torch.einsum("td,efd->tef", x64, w64))
    out = (every.gather(1, pick[..., None].expand(t, 2, d)) * gate64[..., None]).sum(1)
    want = (out - target.cpu().double()).square().mean()
    want.backward()
    # sums of at most t or e * d products in three layers, each step off by U32 of magnitudes that add up to a few times
    # the largest gradient: 1e-4 of it is thirty times what they give
    for got, ref in ((loss.detach()[None], want.detach()[None]), (x.grad, x64.grad), (w.grad, w64.grad), (r.grad, r64.grad)):
        assert float((got.cpu().double() - ref).abs().max()) <= 1e-4 * float(ref.abs().max())
