"""scores_solve against the float64 reference, and the three operators together."""
import threading

import numpy as np
import pytest
import torch

import streaming_sinkhorn_solver_amd as sk
from oracle import scores as osc
from scores_cases import DEV, U, close, matrix
from sk_inputs import random_problem

pytestmark = pytest.mark.gpu


def potential_error(s, f, g, a, b, eps, iters):
    """One half-step: t = c s + h carries 4 u of its largest size T (base 2), the log-sum-exp's sum 2 u + 3 u T ln2 per
    term and at most 200 additions in a row, its logarithm and the product with eps ln2 a few u of the potential.  A
    half-step moves two potentials no further apart (sup norm), so the errors of the 2 iters half-steps add."""
    fin = np.isfinite(s)
    size = np.abs(np.where(fin, s, 0.0)).max() + np.abs(f).max() + np.abs(g).max()
    logs = max(abs(np.log(a[a > 0]).min()), abs(np.log(b[b > 0]).min()))
    T = (size / eps + logs) * 1.4427
    half = eps * (12 * T + 250) * U + 6 * U * size
    return 2 * max(iters, 1) * half


def check(x, s, a, b, eps, iters, g_init=None):
    n, m = s.shape
    dev = lambda v: None if v is None else torch.from_numpy(v).to(DEV)  # noqa: E731
    f, g = sk.scores_solve(x, dev(a), dev(b), eps=eps, n_iters=iters, g_init=dev(g_init), check=False)
    fo, go = osc.solve(s, a, b, eps, iters, g_init)
    aa, bb = np.full(n, 1.0 / n) if a is None else a, np.full(m, 1.0 / m) if b is None else b
    tol = potential_error(np.where((aa > 0)[:, None], s, 0.0), fo[aa > 0], go, aa, bb, eps, iters)
    live = aa > 0
    close(f[torch.from_numpy(live).to(DEV)], fo[live], tol, "f")
    close(g, go, tol, "g")
    return f, g


SHAPES = [(1, 1), (1, 9), (50, 1), (7, 3), (33, 8), (200, 16), (100, 17), (65, 64), (300, 100), (1000, 128), (70, 200),
          (513, 256), (20, 300), (40, 512), (9, 1000), (300, 1024), (20000, 60)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,m", SHAPES)
def test_shapes(n, m, dtype):
    x, s = matrix(n, m, dtype, n + m, spread=1.0, pad=m % 3, offset=n % 2)
    r = np.random.default_rng(n)
    a, b = r.random(n).astype(np.float32) + np.float32(0.1), r.random(m).astype(np.float32) + np.float32(0.1)
    a, b = a / a.sum(), b / b.sum()
    check(x, s, None, None, 0.5, 6)
    check(x, s, a, b, 0.2, 3)
    check(x, s, a, None, 0.3, 1, r.normal(size=m).astype(np.float32))
    check(x, s, None, b, 0.3, 0, r.normal(size=m).astype(np.float32))
    check(x, s, None, None, 0.3, 0)


@pytest.mark.parametrize("m", [5, 40, 256, 700])
@pytest.mark.parametrize("n", [30, 3000])
def test_zero_weights_masks_and_far_columns(n, m):
    """Padding rows that hold NaN, experts without capacity, masked pairs, an empty row and an empty column, and a
    column so far below the others that its share underflows float32."""
    x, s = matrix(n, m, "f32", n * m, spread=1.0, mask=0.2)
    r = np.random.default_rng(m)
    a, b = r.random(n).astype(np.float32), np.ones(m, np.float32)
    a[2:5] = 0.0
    b[1] = 0.0
    a, b = a / a.sum(), b / b.sum()
    x[2:5], s[2:5] = float("nan"), np.nan
    x[7], s[7] = -float("inf"), -np.inf
    x[8:, 2], s[8:, 2] = -300.0, -300.0
    x[:2, 2], s[:2, 2] = -np.inf, -np.inf
    x[5:7, 2], s[5:7, 2] = -np.inf, -np.inf
    live = (np.arange(n) < 2) | (np.arange(n) >= 5)
    x[torch.from_numpy(live).to(DEV), 3], s[live, 3] = -np.inf, -np.inf
    for iters in (1, 2, 5):
        f, g = check(x, s, a, b, 0.5, iters)
        assert f[7] == 0 and g[3] == 0 and torch.isfinite(g).all()
        if m > 5:  # (at m = 5 the mask leaves some rows nothing but the far column)
            assert g[2] > 200


@pytest.mark.parametrize("n", [200, 5000])
@pytest.mark.parametrize("mass", [1.0, 2.0 ** 66])
def test_far_column_at_any_mass(n, mass):
    """A column whose shares lie around the smallest float32 exponential: one row's share is kept, the others' are flushed."""
    s = np.zeros((n, 3), np.float32)
    s[:, 1] = -87.6
    s[3, 1] = -86.0
    a, b = np.full(n, mass / n, np.float32), np.array([mass / 2, mass / 4, mass / 4], np.float32)
    for iters in (1, 3):
        check(torch.from_numpy(s).to(DEV), s.astype(np.float64), a, b, 1.0, iters)


def test_equals_the_point_cloud_solver():
    """The same costs through the library's own solver: C = |x - y|^2 as scores -C."""
    x, y, a, b = random_problem(300, 200, 3, 5)
    X, Y, A, B = (torch.from_numpy(v).to(DEV) for v in (x, y, a, b))
    c = ((x[:, None, :].astype(np.float64) - y[None, :, :]) ** 2).sum(-1)
    s = (-c).astype(np.float32)
    f, g = sk.scores_solve(torch.from_numpy(s).to(DEV), A, B, eps=0.1, n_iters=20)
    fp, gp, _ = sk.solve(X, Y, A, B, eps=0.1, n_iters=20)
    fo, go = osc.solve(s, a, b, 0.1, 20)
    live_a, live_b = a > 0, b > 0
    tol = potential_error(s.astype(np.float64), fo[live_a], go[live_b], a, b, 0.1, 20)
    close(f, fo, tol, "f")
    close(g, go, tol, "g")
    # the point-cloud solver's stated parity, 1e-4 of the largest cost
    assert np.abs(fp.cpu().numpy() - fo)[live_a].max() <= 1e-4 * c.max() and np.abs(gp.cpu().numpy() - go)[live_b].max() <= 1e-4 * c.max()


def test_warm_start_in_place_continues():
    x, s = matrix(500, 60, "f32", 3, spread=1.0)
    f, g = sk.scores_solve(x, eps=0.3, n_iters=12)
    f5, g5 = sk.scores_solve(x, eps=0.3, n_iters=5)
    f7, g7 = sk.scores_solve(x, eps=0.3, n_iters=7, g_init=g5, g=g5)
    assert g7.data_ptr() == g5.data_ptr() and torch.equal(g7, g) and torch.equal(f7, f)


def test_checks_weights_and_refuses():
    x = torch.zeros((4, 6), device=DEV)
    a, b = torch.full((4,), 0.25, device=DEV), torch.full((6,), 1 / 6, device=DEV)
    sk.scores_solve(x, a, b, eps=1.0, n_iters=1)
    for bad in (lambda: sk.scores_solve(x, 2 * a, b, eps=1.0, n_iters=1), lambda: sk.scores_solve(x, -a, b, eps=1.0, n_iters=1),
                lambda: sk.scores_solve(x, a[:3], b, eps=1.0, n_iters=1), lambda: sk.scores_solve(x, a.double(), b, eps=1.0, n_iters=1),
                lambda: sk.scores_solve(x, eps=0.0, n_iters=1), lambda: sk.scores_solve(x, eps=1.0, n_iters=-1),
                lambda: sk.scores_solve(x, eps=1.0, n_iters=1, g_init=a), lambda: sk.scores_solve(x, eps=1.0, n_iters=1, f=b),
                lambda: sk.scores_solve(x[:0], eps=1.0, n_iters=1),
                lambda: sk.scores_solve(torch.zeros((2, 1025), device=DEV), eps=1.0, n_iters=1)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sk.SinkhornError, match="WORKSPACE"):
        sk.scores_solve(x, eps=1.0, n_iters=1, ws=torch.empty(4, dtype=torch.uint8, device=DEV))


def loads(idx, m):
    return np.bincount(idx.reshape(-1), minlength=m)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,m,k", [(512, 16, 2), (4096, 64, 4)])
def test_balance_route_and_gradient_together(n, m, k, dtype):
    """A router's step: potentials of its scores, the choice under them, weights and their gradient."""
    r = np.random.default_rng(m)
    host = torch.from_numpy(r.normal(size=(n, m)) + 2.0 * r.normal(size=(1, m))).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    x, s = host.to(DEV), host.double().numpy()
    f, g = sk.scores_solve(x, eps=0.2, n_iters=30)
    plain = sk.scores_route(x, k, counts=True)
    even = sk.scores_route(x, k, bias=g, select_on="logit", counts=True)
    idx, w, cnt = osc.route(s, k, bias=g.cpu().numpy(), select_on="logit")
    assert np.array_equal(even.idx.cpu().numpy(), idx) and np.array_equal(even.counts.cpu().numpy(), cnt)
    assert even.counts.max() < plain.counts.max() / 2  # the popular experts' load falls
    # the plan of the potentials loads every expert alike
    plan = np.exp((f.double().cpu().numpy()[:, None] + g.double().cpu().numpy()[None, :] + s) / 0.2) / (n * m)
    assert np.abs(plan.sum(0) * m - 1).max() < 1e-3
    dw = torch.randn((n, k), device=DEV)
    grad = sk.scores_route_grad(x, even.idx, dw)
    want = osc.route_grad(s, idx, dw.cpu().numpy())
    assert np.abs(grad.double().cpu().numpy() - want).max() < (2.0 ** -8 if dtype == "bf16" else 1e-5) * np.abs(want).max()


def router_step(x, out, g, dw, logits, tgt, lp, ws_s, ws_l, grads, dl):
    sk.scores_solve(x, eps=0.25, n_iters=4, ws=ws_s, f=out["f"], g=g)
    r = sk.scores_route(x, 4, bias=g, select_on="logit", n_group=4, topk_group=2, group_top=2, counts=True, out=out["r"])
    sk.scores_route_grad(x, r.idx, dw, grad=grads[0])
    sk.scores_logprobs(logits, tgt, top=5, entropy=True, ws=ws_l, out=lp)
    sk.scores_logprobs_grad(logits, tgt, lp, d_logp=dl, d_entropy=dl, grad=grads[1])


def make_step(seed, n=700, m=64, v=20000):
    torch.manual_seed(seed)
    x, logits = torch.randn((n, m), device=DEV), torch.randn((40, v), device=DEV).to(torch.bfloat16)
    tgt = torch.randint(0, v, (40,), device=DEV)
    e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device=DEV)  # noqa: E731
    out = dict(f=e(n), r=sk.Routing(e(n, 4, dt=torch.int32), e(n, 4), e(m, dt=torch.int32)))
    lp = sk.Logprobs(e(40), e(40), e(40), e(40, 5, dt=torch.int32), e(40, 5), e(40, 2))
    args = (x, out, e(m), torch.randn((n, 4), device=DEV), logits, tgt, lp, sk.scores_solve_workspace(n, m, DEV),
            sk.scores_logprobs_workspace(torch.bfloat16, 40, v, 5, DEV), (torch.empty_like(x), torch.empty_like(logits)),
            torch.randn(40, device=DEV))
    return args, [out["f"], args[2], *out["r"], *lp, *args[9]]


def test_graph_replay_matches_eager():
    args, outs = make_step(1)
    router_step(*args)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        router_step(*args)
    for _ in range(4):
        for t in outs:
            t.fill_(-3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, want))
        # new scores at the captured addresses, then the old ones again
        keep = args[0].clone()
        args[0].mul_(0.5)
        graph.replay()
        eager, eager_outs = make_step(1)
        eager[0].copy_(args[0])
        router_step(*eager)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, eager_outs))
        args[0].copy_(keep)


def test_other_streams_and_two_threads():
    """Calls from two host threads on two streams of their own, with workspaces of their own, equal the calls alone."""
    cases = [make_step(s) for s in (2, 3)]
    want = []
    for args, outs in cases:
        router_step(*args)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.fill_(-3)
    torch.cuda.synchronize()
    errors = []

    def work(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(5):
                    router_step(*cases[k][0])
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for (_, outs), exp in zip(cases, want):
        assert all(torch.equal(p, q) for p, q in zip(outs, exp))


def test_results_repeat_bit_for_bit():
    args, outs = make_step(4, n=5000, m=256, v=131072)
    router_step(*args)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    for _ in range(3):
        router_step(*args)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, want))
