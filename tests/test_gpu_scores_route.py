"""scores_route and its gradient against the float64 reference."""
import numpy as np
import pytest
import torch

import streaming_sinkhorn_solver_amd as sk
from oracle import scores as osc
from scores_cases import DEV, U, close, half_step, matrix

pytestmark = pytest.mark.gpu


def weight_error(s, q):
    """q = exp of a difference (3 u of it and 2 u, |difference| <= the row's spread of finite scores, or |s| for the
    sigmoid), over a sum of at most 64 + 16 + 6 terms with the same errors, one division and one product."""
    fin = np.where(np.isfinite(s), s, 0.0)
    span = np.maximum(fin.max(1) - fin.min(1), np.abs(fin).max(1))
    span = np.minimum(span, 110.0)  # beyond that q is zero in float32
    return (6 * span[:, None] + 110) * U * np.abs(q) + 2.0 ** -126


def check(x, s, k, dtype, **how):
    d = dict(fn=how.pop("score_fn", "softmax"), **how)
    bias = d.pop("bias", None)
    gb = None if bias is None else torch.from_numpy(bias).to(DEV)
    r = sk.scores_route(x, k, score_fn=d["fn"], bias=gb, counts=True, **how_gpu(d))
    idx, w, cnt = osc.route(s, k, bias=bias, **d)
    assert np.array_equal(r.idx.cpu().numpy(), idx)
    assert np.array_equal(r.counts.cpu().numpy(), cnt)
    close(r.weights, w, weight_error(s, w), "weights")
    dw = np.random.default_rng(k).normal(size=w.shape).astype(np.float32)
    g = sk.scores_route_grad(x, r.idx, torch.from_numpy(dw).to(DEV), score_fn=d["fn"], renorm=d.get("renorm", True),
                             scale=d.get("scale", 1.0))
    check_grad(g, s, idx, dw, dtype, d)
    return r


def how_gpu(d):
    return {k: v for k, v in d.items() if k != "fn"}


def check_grad(g, s, idx, dw, dtype, d):
    """Each term q dq and the sum over the choice (at most 64 + 6 additions) carry the weight's error; one product
    with 1 - sigmoid; the row's own p times that sum; one rounding to the scores' type."""
    fn, renorm, scale = d["fn"], d.get("renorm", True), d.get("scale", 1.0)
    want = osc.route_grad(s, idx, dw, fn, renorm, scale)
    q = osc._weights(s, idx, fn, renorm)
    size = np.abs(q * dw * scale).sum(1, keepdims=True)
    rel = weight_error(s, np.ones((len(s), 1))) + 80 * U
    at = np.zeros_like(want)
    np.add.at(at, (np.arange(len(s))[:, None], idx), np.abs(q * dw * scale) + (q * size if renorm else 0.0))
    if fn == "softmax" and not renorm:
        at += osc._softmax(s) * size
    info = torch.finfo(g.dtype)
    close(g, want, 2 * rel * at + half_step(dtype) * np.abs(want) * (1 + 1e-3) + info.smallest_normal * info.eps / 2 + 2.0 ** -126,
          "grad")


# every width class (8, 16, 32, 64, 128, 256, 512, 1024 columns), full and ragged, one row to several workgroups
WIDTHS = [(1, 1), (3, 2), (70, 8), (33, 9), (100, 16), (65, 31), (40, 60), (257, 64), (50, 100), (33, 128), (20, 200),
          (130, 256), (9, 300), (6, 512), (5, 1000), (4, 1024)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,m", WIDTHS)
def test_widths(n, m, dtype):
    x, s = matrix(n, m, dtype, n + m, spread=1.5, pad=m % 3, offset=m % 2)
    bias = np.random.default_rng(m).normal(size=m).astype(np.float32) * np.float32(0.3)
    for k in sorted({1, min(m, 2), min(m, 8), min(m, 64)}):
        check(x, s, k, dtype, score_fn="softmax", renorm=False, scale=1.5)
        check(x, s, k, dtype, score_fn="sigmoid", renorm=True, bias=bias)
        check(x, s, k, dtype, score_fn="softmax", renorm=True, bias=bias, select_on="logit", scale=2.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,groups,topg", [(8, 2, 1), (8, 8, 3), (60, 4, 2), (64, 8, 4), (64, 64, 10), (126, 7, 3), (256, 8, 4),
                                           (256, 32, 5), (500, 5, 2), (1024, 16, 4)])
@pytest.mark.parametrize("fn", ["softmax", "sigmoid"])
def test_groups(m, groups, topg, fn, dtype):
    x, s = matrix(50, m, dtype, m + groups, spread=1.2)
    bias = np.random.default_rng(m).normal(size=m).astype(np.float32) * np.float32(0.1)
    k = min(8, topg * (m // groups))
    for gt in (1, 2) if m // groups > 1 else (1,):
        how = dict(score_fn=fn, n_group=groups, topk_group=topg, group_top=gt)
        check(x, s, k, dtype, **how)
        check(x, s, k, dtype, bias=bias, scale=2.5, **how)
        check(x, s, k, dtype, bias=bias, select_on="logit", renorm=False, **how)
        check(x, s, k, dtype, select_on="logit", **how)


@pytest.mark.parametrize("m", [8, 64, 256, 600])
@pytest.mark.parametrize("fn", ["softmax", "sigmoid"])
def test_ties_and_close_values(m, fn):
    """Equal scores, equal biases, and values apart by less than float32 tells."""
    x, s = matrix(200, m, "f32", m, ties=True)
    r = np.random.default_rng(m)
    k = min(m, 8)
    check(x, s, k, "f32", score_fn=fn)
    check(x, s, k, "f32", score_fn=fn, bias=np.zeros(m, np.float32))
    check(x, s, k, "f32", score_fn=fn, bias=r.integers(0, 2, m).astype(np.float32), select_on="logit")
    # scores that differ in the last bits: act rounds them together
    base = (1.0 + r.integers(0, 6, (200, m)) * 2.0 ** -23).astype(np.float32)
    x = torch.from_numpy(base).to(DEV)
    s = base.astype(np.float64)
    for how in (dict(), dict(bias=np.full(m, 0.25, np.float32)), dict(bias=np.full(m, 1000.0, np.float32), select_on="logit")):
        check(x, s, k, "f32", score_fn=fn, **how)
    # 16-bit scores, most of them equal to another, under a bias that is equal too or is not
    x, s = matrix(200, m, "bf16", m + 1, spread=1.0)
    check(x, s, k, "bf16", score_fn=fn, bias=np.zeros(m, np.float32))
    check(x, s, k, "bf16", score_fn=fn, bias=(r.integers(0, 2, m) * np.float32(2.0 ** -20)).astype(np.float32))
    x = torch.from_numpy(base).to(DEV)
    s = base.astype(np.float64)
    if m % 4 == 0:
        k = min(k, m // 2)  # half of the groups take part
        check(x, s, k, "f32", score_fn=fn, n_group=4, topk_group=2, group_top=2)
        check(x, s, k, "f32", score_fn=fn, n_group=4, topk_group=2, group_top=2, bias=np.full(m, 0.25, np.float32))


@pytest.mark.parametrize("fn", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_masks_and_extremes(dtype, renorm, fn):
    x, s = matrix(40, 64, dtype, 3, mask=0.9)
    x[5], s[5] = -float("inf"), -np.inf
    lowest = torch.finfo(x.dtype).min
    x[6], s[6] = lowest, lowest
    x[7, 1:], s[7, 1:] = lowest, lowest
    x[8] = -200.0 + torch.arange(64, device=DEV) % 8  # sigmoid below the float32 range
    x[9] = 200.0
    s[8:10] = x[8:10].double().cpu().numpy()
    check(x, s, 6, dtype, score_fn=fn, renorm=renorm)
    check(x, s, 6, dtype, score_fn=fn, renorm=renorm, n_group=8, topk_group=2)
    bias = np.zeros(64, np.float32)
    bias[:32] = -np.inf  # experts that are switched off
    check(x, s, 6, dtype, score_fn=fn, renorm=renorm, bias=bias, select_on="logit")


@pytest.mark.parametrize("fn", ["softmax", "sigmoid"])
def test_masks_with_a_bias(fn):
    """Masked experts decided by their bias alone, next to values that were rounded; exactly k experts left on."""
    r = np.random.default_rng(5)
    n, m, k = 300, 48, 6
    x, s = matrix(n, m, "f32", 17, spread=1.0, mask=0.7)
    bias = (r.integers(0, 3, m) * np.float32(0.25)).astype(np.float32)
    check(x, s, k, "f32", score_fn=fn, bias=bias)
    # an unmasked expert whose value equals a masked one's up to the last bits
    act = osc.route_values(s, fn, None, "score")
    for i in range(n):
        j = int(np.argmax(np.where(np.isfinite(s[i]), s[i], -np.inf)))
        bias[j % m] = np.float32(0.5 - act[i, j])
    check(x, s, k, "f32", score_fn=fn, bias=bias)
    off = np.full(m, -np.inf, np.float32)
    off[r.permutation(m)[:k]] = r.normal(size=k)
    check(x, s, k, "f32", score_fn=fn, bias=off)
    check(x, s, k, "f32", score_fn=fn, bias=off, select_on="logit")
    check(x, s, k, "f32", score_fn=fn, bias=off, n_group=4, topk_group=2, group_top=2)


def test_nan_and_infinity_leave_valid_choices():
    x, _ = matrix(64, 100, "f32", 9)
    x[3, 5] = float("nan")
    x[4, :] = float("nan")
    x[5, 7] = float("inf")
    for fn in ("softmax", "sigmoid"):
        for how in (dict(), dict(n_group=4, topk_group=2, group_top=2), dict(bias=torch.full((100,), float("nan"), device=DEV))):
            r = sk.scores_route(x, 9, score_fn=fn, counts=True, **how)
            idx = r.idx.cpu().numpy()
            assert idx.min() >= 0 and idx.max() < 100 and all(len(set(row)) == 9 for row in idx.tolist())
            assert int(r.counts.sum()) == 64 * 9
            assert torch.isfinite(r.weights[6:]).all()


def test_gradient_of_given_choices():
    """Dropped entries and an expert that stands twice."""
    x, s = matrix(30, 40, "f32", 11)
    r = np.random.default_rng(1)
    idx = r.integers(0, 40, (30, 5)).astype(np.int32)
    idx[::3, 2] = idx[::3, 4]
    dw = r.normal(size=(30, 5)).astype(np.float32)
    drop = idx.copy()
    drop[1::2, 1] = -1
    drop[4, :] = 40
    for fn in ("softmax", "sigmoid"):
        for renorm in (False, True):
            g = sk.scores_route_grad(x, torch.from_numpy(idx).to(DEV), torch.from_numpy(dw).to(DEV), score_fn=fn, renorm=renorm)
            check_grad(g, s, idx.astype(np.int64), dw, "f32", dict(fn=fn, renorm=renorm))
            g = sk.scores_route_grad(x, torch.from_numpy(drop).to(DEV), torch.from_numpy(dw).to(DEV), score_fn=fn, renorm=renorm)
            assert (g[4] == 0).all()
            for i in (1, 3, 8):  # rows one at a time: without the dropped entry
                keep = (drop[i] >= 0)
                check_grad(g[i:i + 1], s[i:i + 1], idx[i:i + 1, keep].astype(np.int64), dw[i:i + 1, keep], "f32",
                           dict(fn=fn, renorm=renorm))


@pytest.mark.parametrize("m", [8, 60, 256, 700])
def test_gradient_in_place_and_strided(m):
    x, _ = matrix(70, m, "bf16", m, pad=3, offset=1)
    r = sk.scores_route(x, 4, renorm=False)
    dw = torch.randn((70, 4), device=DEV)
    for fn, renorm in (("softmax", False), ("softmax", True), ("sigmoid", True)):
        want = sk.scores_route_grad(x, r.idx, dw, score_fn=fn, renorm=renorm)
        wide = torch.full((70, m + 2), 7.0, dtype=x.dtype, device=DEV)
        wide[:, 1:m + 1] = x
        sk.scores_route_grad(wide[:, 1:m + 1], r.idx, dw, score_fn=fn, renorm=renorm, grad=wide[:, 1:m + 1])
        assert torch.equal(wide[:, 1:m + 1], want) and (wide[:, 0] == 7).all() and (wide[:, -1] == 7).all()


def test_no_rows_and_many_rows():
    r = sk.scores_route(torch.empty((0, 9), device=DEV), 3, counts=True)
    assert r.idx.shape == (0, 3) and r.counts.tolist() == [0] * 9
    assert sk.scores_route_grad(torch.empty((0, 9), device=DEV), r.idx, r.weights).shape == (0, 9)
    n = 200_003
    x = torch.randn((n, 12), device=DEV)
    r = sk.scores_route(x, 2, counts=True)
    assert torch.equal(r.idx.long(), x.topk(2, dim=1).indices)
    assert torch.equal(r.counts.long(), torch.bincount(r.idx.long().reshape(-1), minlength=12))


@pytest.mark.parametrize("n,m,how", [(40_000, 64, dict(score_fn="sigmoid")),
                                     (17_001, 48, dict(score_fn="softmax", n_group=4, topk_group=2, group_top=2))])
def test_many_rows_in_doubt(n, m, how):
    """More rows than the second kernel's workgroups take at once, many of them with values a bit apart."""
    r = np.random.default_rng(n)
    base = (r.integers(-2, 3, (n, m)) + r.integers(0, 4, (n, m)) * 2.0 ** -22).astype(np.float32)
    check(torch.from_numpy(base).to(DEV), base.astype(np.float64), 6, "f32", bias=np.full(m, 0.125, np.float32), **how)


def test_refusals():
    x = torch.zeros((4, 8), device=DEV)
    r = sk.scores_route(x, 2)
    d = torch.ones((4, 2), device=DEV)
    for bad in (lambda: sk.scores_route(x, 0), lambda: sk.scores_route(x, 9), lambda: sk.scores_route(x, 3, n_group=3),
                lambda: sk.scores_route(x, 3, n_group=4, topk_group=1), lambda: sk.scores_route(x, 2, bias=d[:, 0]),
                lambda: sk.scores_route(x, 2, bias=torch.zeros(8, device=DEV).double()),
                lambda: sk.scores_route(x, 2, group_top=3), lambda: sk.scores_route(x, 2, scale=float("inf")),
                lambda: sk.scores_route(torch.zeros((2, 1025), device=DEV), 2),
                lambda: sk.scores_route(x, 3, out=r), lambda: sk.scores_route_grad(x, r.idx.long(), d),
                lambda: sk.scores_route_grad(x, r.idx, d[:, :1]), lambda: sk.scores_route_grad(x, r.idx[:3], d[:3]),
                lambda: sk.scores_route_grad(x, r.idx, d, grad=torch.zeros((4, 9), device=DEV))):
        with pytest.raises(ValueError):
            bad()
