"""GPU: a block's operators on other streams, captured and replayed, and a run of them together
with the losses, the norms and the step around them."""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import (FusedAdamW, FusedDropout, FusedGroupNorm, FusedLayerNorm, FusedRouter,
                                               FusedTokenLoss)

pytestmark = pytest.mark.gpu


def _cases(tokens=700, experts=64, k=4, width=96):
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, z, dw = rand(tokens, width), rand(tokens, experts), rand(tokens, k)
    step = torch.tensor([4], dtype=torch.int32, device="cuda")
    drop, router = FusedDropout(0.3, 8), FusedRouter(tokens, experts, k, score="sigmoid", groups=8, top_groups=4)
    bias = 0.001 * torch.arange(experts, device="cuda")
    w, ids, slots, _ = router.route(z, bias)
    rows = rand(tokens * k, width)
    norm, t = FusedGroupNorm(width, 8, 7, activation="silu"), x.view(7, 100, width)
    _, mean, rstd = norm.forward(t)
    return [lambda **kw: [drop.forward(x, step, x, **kw)], lambda **kw: [drop.backward(x, step, **kw)],
            lambda **kw: router.route(z, bias, **kw), lambda **kw: [router.backward(dw, z, ids, **kw)],
            lambda **kw: [router.dispatch(x, slots, **kw)], lambda **kw: [router.combine(rows, slots, w, **kw)],
            lambda **kw: router.combine_backward(x, rows, slots, w, **kw), lambda **kw: norm.forward(t, **kw),
            lambda **kw: norm.backward(t, t, None, None, mean, rstd, **kw)]


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_do_not_share_memory_with_work_on_the_current_stream(raw):
    s = torch.cuda.Stream()
    for call in _cases():
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        blocks = [torch.empty_like(t) for t in want]
        at = {b.data_ptr() for b in blocks}
        torch.cuda._sleep(20_000_000)           # about 10 ms, far longer than the call
        for b in blocks:
            b.fill_(float("nan") if b.is_floating_point() else -7)
        del b, blocks
        got = call(stream=s.cuda_stream if raw else s)
        assert not at & {t.data_ptr() for t in got}
        s.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        current = torch.cuda.current_stream()
        for t in got:
            t.record_stream(current)


class Block:
    """Group norm over each sequence, routing, two experts' products a token, dropout and the residual, layer
    norm, a policy loss; and all the way back into the plan's grads."""

    def __init__(self, tokens=256, width=64, experts=8, k=2, vocab=500, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.tokens, self.width, self.experts, self.k = tokens, width, experts, k
        self.x, self.labels = rand(4, tokens // 4, width), torch.randint(0, vocab, (tokens,), device="cuda", generator=g)
        self.weights, self.adv = torch.full((tokens,), 1 / tokens, device="cuda"), rand(tokens)
        p = dict(gw=1 + 0.1 * rand(width), gb=0.1 * rand(width), gate=0.3 * rand(width, experts),
                 up=rand(experts, width, width) / 8, lw=1 + 0.1 * rand(width), lb=0.1 * rand(width), out=rand(width, vocab) / 8)
        self.p, self.g = p, {n: torch.zeros_like(t) for n, t in p.items()}
        zeros = lambda: [torch.zeros_like(t) for t in p.values()]  # noqa: E731
        self.opt = FusedAdamW(list(p.values()), list(self.g.values()), zeros(), zeros(), [0.0] * len(p))
        self.lr, self.steps = torch.tensor([1e-3], device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        self.bias = torch.zeros(experts, device="cuda")
        self.gn, self.ln = FusedGroupNorm(width, 8, 4, activation="silu"), FusedLayerNorm(width)
        self.router = FusedRouter(tokens, experts, k, score="sigmoid", groups=4, top_groups=3, group_score="top2", scale=1.5)
        self.drop, self.loss = FusedDropout(0.2, 17, 1), FusedTokenLoss(tokens)
        self.norm = torch.zeros(1, device="cuda")

    def step(self, update=True):
        p, g, flat = self.p, self.g, (self.tokens, self.width)
        h, mean, rstd = self.gn.forward(self.x, p["gw"], p["gb"])
        h = h.view(flat)
        z = h @ p["gate"]
        w, ids, slots, starts = self.router.route(z, self.bias)
        xs = self.router.dispatch(h, slots)
        of = torch.searchsorted(starts[1:], torch.arange(len(xs), dtype=torch.int32, device="cuda"), right=True)
        ys = torch.bmm(xs[:, None], p["up"][of])[:, 0]
        y = self.router.combine(ys, slots, w)
        r = self.drop.forward(y, self.steps, self.x.view(flat))
        n, lm, lr = self.ln.forward(r, p["lw"], p["lb"])
        logits = n @ p["out"]
        stats, _, dlogits = self.loss.policy(logits, self.labels, self.weights, self.adv)
        torch.mm(n.t(), dlogits, out=g["out"])
        dr, _, _ = self.ln.backward(dlogits @ p["out"].t(), r, p["lw"], lm, lr, dweight=g["lw"], dbias=g["lb"])
        dy = self.drop.backward(dr, self.steps)
        dys, dw = self.router.combine_backward(dy, ys, slots, w)
        g["up"].zero_().index_add_(0, of, xs[:, :, None] * dys[:, None])
        dxs = torch.bmm(dys[:, None], p["up"][of].transpose(1, 2))[:, 0]
        dz = self.router.backward(dw, z, ids)
        torch.mm(h.t(), dz, out=g["gate"])
        dh = self.router.combine(dxs, slots) + dz @ p["gate"].t()
        self.dx, _, _ = self.gn.backward(dh.view_as(self.x), self.x, p["gw"], p["gb"], mean, rstd, dweight=g["gw"], dbias=g["gb"])
        self.dx = self.dx + dr.view_as(self.x)
        if update:
            self.opt.grad_norm(self.norm)
            self.opt.step(self.lr, self.steps)
            self.router.balance(self.bias, starts, 0.01)
        return stats, ids, starts

    def plain(self, kept, ids):
        """The loss by torch in 64 bits with the same mask and the same experts, for its gradients."""
        leaf = {n: t.detach().double().requires_grad_() for n, t in self.p.items()}
        x = self.x.double().requires_grad_()
        f = torch.nn.functional
        h = f.silu(f.group_norm(x.transpose(1, 2), 8, leaf["gw"], leaf["gb"], 1e-5)).transpose(1, 2).reshape(self.tokens, -1)
        s = torch.sigmoid(h @ leaf["gate"]).gather(1, ids)
        w = 1.5 * s / s.sum(1, keepdim=True)
        y = (torch.einsum("tw,twkv->tkv", h, leaf["up"][ids].transpose(1, 2)) * w[:, :, None]).sum(1)
        r = x.view(self.tokens, -1) + torch.where(kept, y / (1 - float(np.float32(0.2))), 0.0)
        logits = f.layer_norm(r, (self.width,), leaf["lw"], leaf["lb"], 1e-5) @ leaf["out"]
        lp = f.log_softmax(logits, 1).gather(1, self.labels[:, None])[:, 0]
        # at the first step the ratio is 1, whose slope is that of exp at 0
        loss = -(self.weights.double() * self.adv.double() * torch.exp(lp - lp.detach())).sum()
        loss.backward()
        return loss, {n: t.grad for n, t in leaf.items()}, x.grad


def test_a_block_s_gradients_are_the_formula_s():
    """float32 through eleven operators: 1e-4 of each gradient's largest entry is a hundred times the sums' u sqrt(n)."""
    from oracle import dropout as DR
    torch.backends.cuda.matmul.allow_tf32 = False
    b = Block()
    stats, ids, starts = b.step(update=False)
    kept = torch.from_numpy(DR.keep((b.tokens, b.width), 0.2, 17, 0, 1)).cuda()
    assert (ids >= 0).all() and int(starts[-1]) == b.tokens * b.k
    loss, grads, dx = b.plain(kept, ids.long())
    assert abs(stats[0].item() - loss.item()) < 1e-5
    for name, want in grads.items():
        assert (b.g[name].double() - want).abs().max() <= 1e-4 * want.abs().max(), name
    assert (b.dx.double() - dx).abs().max() <= 1e-4 * dx.abs().max()


def test_a_captured_block_trains_as_an_eager_one():
    """Each replay reads the step counter, so that its mask is that step's."""
    eager, graphed = Block(), Block()
    for _ in range(2):
        eager.step()
        graphed.step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            graphed.step()
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(4):
        eager.step()
        g.replay()
        torch.cuda.synchronize()
        assert int(eager.steps) == int(graphed.steps)
        # the products of the experts' grads add by atomics: equal up to their order
        for n in eager.p:
            assert torch.allclose(eager.p[n], graphed.p[n], rtol=1e-3, atol=1e-4), n
    assert eager.loss.status() == 0 and graphed.ln.status() == 0


def test_captured_calls_give_the_bits_of_plain_ones():
    for call in _cases():
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                got = call()
        for _ in range(2):
            for t in got:
                t.fill_(-3)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got))


# the kernels that a group norm's sizes choose among: lanes, a CTA's part, a cluster, parts of samples
@pytest.mark.parametrize("shape,groups", [((900, 1, 256), 8), ((40, 6, 96), 4), ((6, 700, 320), 32), ((2, 60_000, 64), 4), ((9, 9000, 512), 8)])
def test_a_captured_group_norm_gives_the_bits_of_plain_calls(shape, groups):
    n, length, c = shape
    x, dy = torch.empty(shape, device="cuda", dtype=torch.bfloat16), torch.empty(shape, device="cuda", dtype=torch.bfloat16)
    w, b = torch.rand(c, device="cuda"), torch.rand(c, device="cuda")
    norm = FusedGroupNorm(c, groups, n, activation="silu")
    out = [torch.empty_like(x), torch.empty(n, groups, device="cuda"), torch.empty(n, groups, device="cuda"), torch.empty_like(x),
           torch.empty_like(w), torch.empty_like(w)]

    def run():
        norm.forward(x, w, b, y=out[0], mean=out[1], rstd=out[2])
        norm.backward(dy, x, w, b, out[1], out[2], dx=out[3], dweight=out[4], dbias=out[5])

    x.normal_(), dy.normal_()
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            run()
    for _ in range(3):
        x.normal_(), dy.normal_()
        run()
        want = [t.clone() for t in out]
        for t in out:
            t.fill_(-1.0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, out))
    assert norm.status() == 0


def test_two_plans_at_once_do_not_disturb_one_another():
    """Samples in parts wait for one another; on two streams each plan's have words of their own."""
    x = [torch.randn(3, 30_000, 96, device="cuda") for _ in range(2)]
    norms = [FusedGroupNorm(96, 4, 3) for _ in range(2)]
    routers = [FusedRouter(5000, 64, 4) for _ in range(2)]
    z = [torch.randn(5000, 64, device="cuda") for _ in range(2)]
    want = [[*norms[i].forward(x[i]), *routers[i].route(z[i])] for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i] = [*norms[i].forward(x[i], stream=s), *routers[i].route(z[i], stream=s)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert norms[0].status() == norms[1].status() == 0


def test_calls_after_a_plan_that_did_not_fit():
    from adamw_optimizer_step_tensor_gb300 import AdamWError, _capi
    for call in _cases():
        want = [t.clone() for t in call()]
        with pytest.raises(AdamWError) as e:
            FusedGroupNorm(1 << 16, 1 << 16, 1 << 24)          # 8 TB of means
        assert e.value.status == _capi.ENOMEM
        assert all(torch.equal(a, b) for a, b in zip(want, call()))


def test_routes_without_places():
    from adamw_optimizer_step_tensor_gb300 import _capi
    router, z = FusedRouter(3000, 64, 4), torch.randn(3000, 64, device="cuda")
    w, ids, _, _ = router.route(z)
    w2, ids2 = torch.zeros_like(w), torch.zeros_like(ids)
    _capi.adamw_route(router.plan, _capi.F32, 3000, z.data_ptr(), 64, None, w2.data_ptr(), ids2.data_ptr(), None, None,
                      torch.cuda.current_stream().cuda_stream)
    assert torch.equal(w, w2) and torch.equal(ids, ids2)
