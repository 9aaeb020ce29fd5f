"""The order of scores_route where float32 cannot tell values apart by itself: far negative sigmoid scores, values
around the smallest normal number, sums beyond the largest."""
import numpy as np
import pytest
import torch

import streaming_sinkhorn_solver_amd as sk
from oracle import scores as osc
from scores_cases import DEV

pytestmark = pytest.mark.gpu

F = np.float32


def logit(p):
    return (np.log(p) - np.log1p(-p)).astype(F)


def same_choice(s, k, dtype=torch.float32, **how):
    """idx and counts are those of the float64 reference."""
    x = torch.from_numpy(s).to(dtype)
    d = dict(how)
    bias = d.pop("bias", None)
    r = sk.scores_route(x.to(DEV), k, bias=None if bias is None else torch.from_numpy(bias).to(DEV), counts=True, **d)
    idx, _, cnt = osc.route(x.double().numpy(), k, fn=d.pop("score_fn", "softmax"), bias=bias, **d)
    wrong = (r.idx.cpu().numpy() != idx).any(1)
    assert not wrong.any(), f"{wrong.sum()} of {len(wrong)} rows, the first {np.flatnonzero(wrong)[0]}"
    assert np.array_equal(r.counts.cpu().numpy(), cnt)


@pytest.mark.parametrize("low", [-5, -12, -23, -40, -60, -80, -87, -95])
@pytest.mark.parametrize("m", [2, 40, 300])
def test_far_negative_sigmoid_scores_under_a_bias_of_their_size(m, low):
    """Two columns whose act and bias add up to almost the same number, the others far below them: the relative error of
    a float32 sigmoid grows with the score."""
    r = np.random.default_rng(m - low)
    a = np.exp(low)
    b = (-a * np.array([0.3, 0.9])).astype(F)
    act = a * (1 + r.random((20000, 1))) - b
    s = np.full((20000, m), -np.inf, F)
    bias = np.full(m, -1.0, F)
    s[:, [0, m - 1]], bias[[0, m - 1]] = logit(act), b
    same_choice(s, 2, score_fn="sigmoid", bias=bias)


def test_two_far_negative_sigmoid_scores():
    """Float32 values 3.0e-16 apart, in the other order than the values themselves."""
    s = np.array([[-22.945890426635742, -22.961633682250977]], F)
    same_choice(s, 2, score_fn="sigmoid", bias=np.array([-9.749198670583326e-11, -9.579995824404719e-11], F))


@pytest.mark.parametrize("low", [-30, -87, -95])
def test_far_softmax_acts_under_a_bias_of_their_size(low):
    """The same for softmax, whose bound grows with the distance to the row's maximum; subnormal acts among them."""
    r = np.random.default_rng(-low)
    a = np.exp(low)
    b = (-a * np.array([0.0, 0.3, 0.9])).astype(F)
    s = np.log(a * (1 + r.random((20000, 1))) - b.astype(np.float64)).astype(F)
    s[:, 0] = 0.0
    same_choice(s, 3, score_fn="softmax", bias=b)


@pytest.mark.parametrize("lo,hi", [(-5, -2), (-16, -12), (-30, -25), (-60, -55), (-86, -84)])
@pytest.mark.parametrize("size", [2, 20])
def test_groups_of_far_negative_sigmoid_scores(size, lo, hi):
    """Two groups whose two largest values add up to almost the same sum."""
    r = np.random.default_rng(size - lo)
    x = r.uniform(lo, hi, (60000, 3)).astype(F)
    p = osc._sigmoid(x.astype(np.float64))
    rest = p[:, 0] + p[:, 1] - p[:, 2]
    x, rest = x[rest > np.exp(lo - 1.0)], rest[rest > np.exp(lo - 1.0)]
    s = np.full((len(x), 2 * size), -np.inf, F)
    s[:, 0], s[:, size - 1], s[:, size], s[:, -1] = x[:, 0], x[:, 1], x[:, 2], logit(rest)
    same_choice(s, 2, score_fn="sigmoid", n_group=2, topk_group=1, group_top=2)


@pytest.mark.parametrize("lo,hi", [(-88.2, -86.8), (-88.7, -87.4), (-89.5, -88.5), (-103.0, -99.0)])
@pytest.mark.parametrize("size", [2, 20])
def test_groups_of_sigmoids_below_the_smallest_normal_number(size, lo, hi):
    """Group sums of subnormal sigmoids, and of some whose exponential is infinite in float32."""
    r = np.random.default_rng(size)
    n, groups = 20000, 4
    s = np.full((n, groups, size), -np.inf, F)
    s[:, :, :2] = r.uniform(lo, hi, (n, groups, 2))
    same_choice(s.reshape(n, -1), 3, score_fn="sigmoid", n_group=groups, topk_group=2, group_top=2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [2, 16])
@pytest.mark.parametrize("with_bias", [False, True])
def test_group_sums_beyond_float32(with_bias, size, dtype):
    """Masks of -inf and of the type's lowest value side by side, and groups of numbers near the largest."""
    r = np.random.default_rng(size)
    n, groups = 500, 8
    big = torch.finfo(dtype).max
    s = r.choice(np.array([-np.inf, -big], F), (n, groups, size))
    dead = r.random((n, groups)) < 0.5
    s[dead] = -np.inf
    s[: n // 2, :, 0] = np.where(r.random((n // 2, groups)) < 0.2, F(1.0), s[: n // 2, :, 0])
    s[-100:] = big * r.choice(np.array([0.5, 0.625, 0.75, 0.875, 1.0]), (100, groups, size))
    bias = np.zeros(groups * size, F) if with_bias else None
    for topg in (1, 3):
        same_choice(s.reshape(n, -1).astype(F), 2, dtype, select_on="logit", bias=bias, n_group=groups, topk_group=topg, group_top=2)


@pytest.mark.parametrize("m,k", [(8, 8), (8, 3), (40, 12), (300, 20)])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_score_and_bias_beyond_float32(sign, m, k):
    """Scores and biases near the type's ends: their sum is finite, whatever float32 makes of it."""
    r = np.random.default_rng(m)
    big = np.finfo(F).max
    s = r.choice(np.array([-np.inf if sign < 0 else 1.0, sign * big, sign * 0.75 * big, 0.5], F), (400, m), p=[0.4, 0.3, 0.25, 0.05])
    bias = (sign * r.choice(np.array([0.0, 0.5, 0.75, 1.0]), m) * big).astype(F)
    same_choice(s, k, select_on="logit", bias=bias)
    if m % 4 == 0 and k <= m // 2:
        for gt in (1, 2):
            same_choice(s, k, select_on="logit", bias=bias, n_group=4, topk_group=2, group_top=gt)


@pytest.mark.parametrize("fn,step", [("sigmoid", 5.0), ("softmax", -800.0)])
@pytest.mark.parametrize("m", [8, 48, 300])
def test_saturated_acts_tie_under_a_bias_and_keep_the_scores_order_without_one(m, fn, step):
    """Sigmoids that are 1, or softmax acts that are 0, in float64 too."""
    s = (40.0 + step * (np.arange(m) % 6))[None, :].repeat(20, 0).astype(F)
    if fn == "softmax":
        s[:, m // 2] = 5000.0
    x, k = torch.from_numpy(s).to(DEV), min(m // 4, 6)
    for bias in (None, np.zeros(m, F), np.full(m, 0.25, F)):
        same_choice(s, k, score_fn=fn, bias=bias)
        same_choice(s, k, score_fn=fn, bias=bias, n_group=2, topk_group=1, group_top=2)
    none, zero = (sk.scores_route(x, k, score_fn=fn, bias=b).idx[0].tolist() for b in (None, torch.zeros(m, device=DEV)))
    assert none == np.argsort(-s[0], kind="stable")[:k].tolist()
    assert zero == (list(range(k)) if fn == "sigmoid" else [m // 2] + list(range(k - 1)))
