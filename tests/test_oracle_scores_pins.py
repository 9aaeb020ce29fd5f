"""The float64 reference of the score-matrix operators against what it must
satisfy: finite differences, marginals, the point-cloud oracle at the same cost,
closed forms; and planted mistakes in it that these checks must notice."""
import numpy as np
import pytest

import oracle
from oracle import scores as osc

RNG = np.random.default_rng


def differences(fun, s, h=1e-6):
    """Central differences of a scalar function of a matrix."""
    g = np.zeros_like(s)
    for i in np.ndindex(*s.shape):
        if not np.isfinite(s[i]):
            continue
        up, dn = s.copy(), s.copy()
        up[i] += h
        dn[i] -= h
        g[i] = (fun(up) - fun(dn)) / (2 * h)
    return g


# central differences at h = 1e-6 of functions with values and third derivatives of order 1: truncation h^2 ~ 1e-12,
# cancellation 2^-52 / h ~ 2e-10 per unit of the value (about ten here)
DIFF_TOL = 1e-8


def test_solve_equals_point_cloud_oracle():
    r = RNG(1)
    x, y = r.normal(size=(9, 2)).astype(np.float32), r.normal(size=(7, 2)).astype(np.float32)
    a, b = r.random(9).astype(np.float32), r.random(7).astype(np.float32)
    a, b = a / a.sum(), b / b.sum()
    c = ((x[:, None, :].astype(np.float64) - y[None, :, :]) ** 2).sum(-1)
    f, g = osc.solve(-c, a, b, 0.3, 17)
    fo, go, _ = oracle.sinkhorn(x, y, a, b, 0.3, 17)
    assert np.abs(f - fo).max() < 1e-12 and np.abs(g - go).max() < 1e-12


def test_solve_marginals_and_warm_start():
    r = RNG(2)
    s = r.normal(size=(30, 5))
    s[3, 1] = s[8, 0] = -np.inf
    a, b = r.random(30), r.random(5)
    a[4] = 0.0
    a, b = a / a.sum(), b / b.sum()
    s[4, :] = np.nan  # padding
    f, g = osc.solve(s, a, b, 0.5, 400)
    plan = a[:, None] * b[None, :] * np.exp((f[:, None] + g[None, :] + np.where(np.isnan(s), 0, s)) / 0.5)
    assert np.abs(plan.sum(0) - b).max() < 1e-12 and np.abs(plan.sum(1) - a).max() < 1e-10
    f1, g1 = osc.solve(s, a, b, 0.5, 7, osc.solve(s, a, b, 0.5, 5)[1])
    f2, g2 = osc.solve(s, a, b, 0.5, 12)
    assert np.array_equal(f1, f2) and np.array_equal(g1, g2)


def test_solve_empty_rows_and_columns():
    s = np.array([[0.0, 1.0, -np.inf], [-np.inf] * 3, [0.5, -1.0, -np.inf]])
    f, g = osc.solve(s, None, None, 1.0, 3)
    assert f[1] == 0.0 and g[2] == 0.0 and np.isfinite(f).all() and np.isfinite(g).all()


@pytest.mark.parametrize("fn", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_grad_against_differences(fn, renorm):
    r = RNG(3)
    s, dw = r.normal(size=(4, 6)), r.normal(size=(4, 3))
    idx = osc.route(s, 3, fn)[0]
    idx[2] = [5, 1, 5]  # an index that stands twice

    def value(x):
        return float((1.7 * osc._weights(x, idx, fn, renorm) * dw).sum())

    assert np.abs(osc.route_grad(s, idx, dw, fn, renorm, 1.7) - differences(value, s)).max() < DIFF_TOL


def test_route_by_hand():
    s = np.log(np.array([[0.1, 0.4, 0.2, 0.3]]))
    idx, w, cnt = osc.route(s, 2, renorm=False)
    assert idx.tolist() == [[1, 3]] and np.allclose(w, [[0.4, 0.3]]) and cnt.tolist() == [0, 1, 0, 1]
    idx, w, _ = osc.route(s, 2, renorm=True, scale=2.0)
    assert np.allclose(w, [[8 / 7, 6 / 7]])
    # the bias takes part in the choice, not in the weights
    idx, w, _ = osc.route(s, 2, renorm=False, bias=np.array([0.35, 0, 0, 0]))
    assert idx.tolist() == [[0, 1]] and np.allclose(w, [[0.1, 0.4]])
    # groups {0, 1}, {2, 3}: the sum of two decides otherwise than the maximum
    s = np.log(np.array([[0.4, 0.05, 0.3, 0.25]]))
    assert osc.route(s, 2, n_group=2, topk_group=1, group_top=1)[0].tolist() == [[0, 1]]
    assert osc.route(s, 2, n_group=2, topk_group=1, group_top=2)[0].tolist() == [[2, 3]]
    # ties to the lower index; a masked expert is chosen last and weighs nothing
    s = np.array([[1.0, 1.0, -np.inf, 1.0]])
    idx, w, _ = osc.route(s, 4)
    assert idx.tolist() == [[0, 1, 3, 2]] and np.allclose(w, [[1 / 3, 1 / 3, 1 / 3, 0]])
    assert np.array_equal(osc.route(np.full((1, 3), -np.inf), 2)[1], [[0.0, 0.0]])


@pytest.mark.parametrize("eps", [1.0, 0.6])
def test_logprobs_grad_against_differences(eps):
    r = RNG(4)
    s = r.normal(size=(5, 7)) * 2
    s[1, 2] = s[3, 0] = -np.inf
    t = np.array([0, 3, -1, 6, 2])
    top = osc.logprobs(s, t, eps, 3)["top_idx"]
    top[4] = [2, 5, 2]  # a pick that is the target too, and twice
    d = dict(d_logp=r.normal(size=5), d_lse=r.normal(size=5), d_entropy=r.normal(size=5), d_top=r.normal(size=(5, 3)))

    def value(x):
        o = osc.logprobs(x, t, eps)
        lp = x / eps - o["lse"][:, None]
        return float((o["logp"] * d["d_logp"] + o["lse"] * d["d_lse"] + o["entropy"] * d["d_entropy"]).sum()
                     + (np.take_along_axis(lp, top, 1) * d["d_top"]).sum())

    g = osc.logprobs_grad(s, t, eps, top, **d)
    fin = np.isfinite(s)
    assert np.abs((g - differences(value, s))[fin]).max() < DIFF_TOL / eps ** 3
    assert np.abs(g[~fin]).max() == 0.0


def test_logprobs_closed_forms():
    s = np.zeros((1, 8))
    o = osc.logprobs(s, [3], 0.5, 8)
    assert np.allclose(o["logp"], -np.log(8)) and np.allclose(o["lse"], np.log(8)) and np.allclose(o["entropy"], np.log(8))
    assert o["top_idx"].tolist() == [list(range(8))]
    o = osc.logprobs(np.full((1, 4), -np.inf), [1], 1.0, 2)
    assert o["lse"][0] == -np.inf and o["logp"][0] == -np.inf and o["entropy"][0] == 0.0
    assert o["top_idx"].tolist() == [[0, 1]] and (o["top_logp"] == -np.inf).all()
    assert np.isnan(osc.logprobs(s, [8])["logp"][0]) and osc.logprobs(s, [-1])["logp"][0] == 0.0


@pytest.mark.parametrize("plant", ["no_pull", "no_entropy_mean", "no_temperature"])
def test_planted_mistakes_are_noticed(plant, monkeypatch):
    """A gradient with a term left out is off the differences by far more than their tolerance."""
    r = RNG(5)
    s, t, d = r.normal(size=(3, 5)), np.array([0, 1, 4]), r.normal(size=3)

    def value(x):
        o = osc.logprobs(x, t, 0.6)
        return float((o["logp"] * d + o["entropy"] * d).sum())

    g = osc.logprobs_grad(s, t, 0.6, d_logp=d, d_entropy=d)
    p = np.exp(s / 0.6 - osc.logprobs(s, t, 0.6)["lse"][:, None])
    wrong = {"no_pull": g + p * d[:, None] / 0.6,
             "no_entropy_mean": g + p * (osc.logprobs(s, t, 0.6)["entropy"] * d)[:, None] / 0.6,
             "no_temperature": g * 0.6}[plant]
    want = differences(value, s)
    assert np.abs(g - want).max() < DIFF_TOL / 0.6 ** 3
    assert np.abs(wrong - want).max() > 1e-3
