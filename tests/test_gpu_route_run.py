"""The operators behind the router and the head together, as a mixture's layer and a decoding step use them, against the
same in float64; the layer's training step with its gradients against torch's."""
import numpy as np
import pytest
import torch

import streaming_sinkhorn_solver_amd as sk
from oracle import routed as oro
from scores_cases import DEV, U, close, f64

pytestmark = pytest.mark.gpu


def experts(rows, plan, up):
    """Each expert's product with its own rows; rows behind the last segment stay zero."""
    out = torch.zeros(rows.shape[0], up.shape[2], dtype=rows.dtype, device=rows.device)
    ends = plan.offsets.tolist()
    for e in range(up.shape[0]):
        out[ends[e]:ends[e + 1]] = rows[ends[e]:ends[e + 1]] @ up[e]
    return out


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan):
        ctx.plan = plan
        return sk.route_dispatch(x, plan, out=torch.zeros(plan.source.numel(), x.shape[1], dtype=x.dtype, device=x.device))

    @staticmethod
    def backward(ctx, d_rows):
        return sk.route_combine(d_rows, ctx.plan), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, plan):
        ctx.plan = plan
        ctx.save_for_backward(rows, weights)
        return sk.route_combine(rows, plan, weights)

    @staticmethod
    def backward(ctx, d_y):
        rows, weights = ctx.saved_tensors
        return *sk.route_combine_grad(rows, ctx.plan, weights, d_y, d_rows=torch.zeros_like(rows)), None


class Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, scores, k):
        r = sk.scores_route(scores, k)
        ctx.save_for_backward(scores, r.idx)
        ctx.mark_non_differentiable(r.idx)
        return r.weights, r.idx

    @staticmethod
    def backward(ctx, d_weights, _):
        scores, idx = ctx.saved_tensors
        return sk.scores_route_grad(scores, idx, d_weights.contiguous()), None


@pytest.mark.parametrize("n,k,m,d,h,align", [(1, 2, 4, 64, 32, 1), (130, 3, 8, 72, 40, 1), (257, 4, 16, 129, 65, 8)])
def test_layer_and_its_gradients(n, k, m, d, h, align):
    r = np.random.default_rng(n)
    x, router = r.normal(size=(n, d)), r.normal(size=(d, m)) / np.sqrt(d)
    up, dy = r.normal(size=(m, d, h)) / np.sqrt(d), r.normal(size=(n, h))
    g = lambda a: torch.from_numpy(a.astype(np.float32)).to(DEV)
    X, R, W = g(x).requires_grad_(), g(router).requires_grad_(), g(up).requires_grad_()
    scores = X @ R
    weights, idx = Route.apply(scores, k)
    plan = sk.route_sort(idx, m, align=align)
    rows = Dispatch.apply(X, plan)
    y = Combine.apply(experts(rows, plan, W), weights, plan)
    y.backward(g(dy))
    # the same densely in float64, for the choice that was made
    X2, R2, W2 = (t.detach().double().cpu().requires_grad_() for t in (X, R, W))
    s2 = X2 @ R2
    pick = idx.cpu().long()
    w2 = torch.softmax(s2.gather(1, pick), 1)
    each = torch.stack([X2 @ W2[e] for e in range(m)], 1)  # (n, m, h)
    y2 = (w2[:, :, None] * each.gather(1, pick[:, :, None].expand(n, k, h))).sum(1)
    y2.backward(g(dy).double().cpu())
    assert np.array_equal(f64(idx).astype(int), np.argsort(-f64(scores), axis=1, kind="stable")[:, :k])
    # float32 products of d, m or h terms of order 1 with one another: errors some u of the sum of the sizes
    for got, want, size in ((y, y2, d), (X.grad, X2.grad, d + h + m), (R.grad, R2.grad, n + h), (W.grad, W2.grad, n)):
        want = want.detach().numpy()
        close(got, want, 64 * U * size ** 0.5 * (1 + np.abs(want).max()) * np.ones_like(want), "layer")


def test_decoding_step():
    """Tokens through a mixture's layer, the head's scores, drafted tokens verified, log-probabilities of what is emitted."""
    n_rows, b, k, m, d, vocab = 5, 9, 2, 8, 96, 3001
    n = n_rows * b
    r = np.random.default_rng(3)
    g = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV)
    x, router, up, head = (g(r.normal(size=s) / np.sqrt(s[0] if len(s) < 3 else s[1]) * 2) for s in
                           ((n, d), (d, m), (m, d, d), (d, vocab)))
    route = sk.scores_route(x @ router, k, score_fn="sigmoid", bias=g(r.normal(size=m) * 0.1), counts=True)
    plan = sk.route_sort(route.idx, m, align=4)
    assert torch.equal(plan.counts, route.counts)
    rows = sk.route_dispatch(x, plan, out=torch.zeros(plan.source.numel(), d, device=DEV))
    y = sk.route_combine(experts(rows, plan, up), plan, route.weights, add=x)
    logits = y @ head
    draft = logits + 0.3 * torch.randn(n, vocab, device=DEV)
    tokens = torch.where(torch.arange(n, device=DEV) % n_rows < n_rows - 1, torch.distributions.Categorical(logits=draft).sample(), -1)
    starts = torch.arange(b + 1, device=DEV) * n_rows
    ua, us = torch.rand(n, device=DEV), torch.rand(b, device=DEV)
    v = sk.scores_verify(logits, tokens, starts, ua, us, draft=draft, eps=0.9)
    acc, nxt, emitted, _, _ = oro.verify(f64(logits), tokens.cpu().numpy(), starts.cpu().numpy(), f64(ua), f64(us), f64(draft), 0.9)
    assert np.array_equal(v.accepted.cpu().numpy(), acc) and np.array_equal(v.next.cpu().numpy(), nxt)
    assert np.array_equal(v.tokens.cpu().numpy(), emitted) and 0 < acc.sum() < n - b
    # what the head's operator says of the emitted tokens
    lp = sk.scores_logprobs(logits, v.tokens, eps=0.9)
    assert torch.equal(lp.logp == 0, v.tokens < 0)
    # both from float32 sums of 3001 terms: 6 ln m + 64 u and 3 ln m + 150 u of them, 4 u of what is taken from the maximum
    close(v.logp, f64(lp.logp), (9 * np.log(vocab) + 230) * U + 8 * U * np.abs(f64(lp.logp)), "logp")
    # the layer in float64
    plan_ref = oro.sort(route.idx.cpu().numpy(), m, 4)
    for got, want in zip(plan, plan_ref):
        assert np.array_equal(got.cpu().numpy(), want)
    each = np.stack([f64(x) @ f64(up[e]) for e in range(m)], 1)
    want = f64(x) + (f64(route.weights)[:, :, None] * np.take_along_axis(each, route.idx.cpu().numpy().astype(int)[:, :, None], 1)).sum(1)
    close(y, want, 64 * U * d ** 0.5 * np.abs(want).max() * np.ones_like(want), "layer")
