"""The float64 reference of token rows under a routing and of drafted tokens against what it must satisfy; and planted
mistakes that these checks must notice."""
import numpy as np
import pytest

from oracle import routed as oro

RNG = np.random.default_rng


def choices(n, k, m, seed, dropped=0.2):
    r = RNG(seed)
    idx = np.array([r.permutation(m)[:k] for _ in range(n)], np.int32).reshape(n, k)
    idx[r.random((n, k)) < dropped] = r.choice([-1, m, m + 7])
    return idx


def check_plan(idx, m, align, capacity, plan):
    slot, source, counts, offsets = plan
    n, k = idx.shape
    flat, place = idx.reshape(-1), slot.reshape(-1)
    assert (offsets % align == 0).all() and (np.diff(offsets) >= counts).all() and (np.diff(offsets) < counts + align).all()
    assert len(source) >= offsets[-1]
    for e in range(m):
        want = np.nonzero(flat == e)[0]
        want = want[:capacity] if capacity else want
        here = source[offsets[e]:offsets[e + 1]]
        assert counts[e] == len(want) and np.array_equal(here[:len(want)], want) and (here[len(want):] == -1).all()
        assert np.array_equal(place[want], offsets[e] + np.arange(len(want)))
    assert (source[offsets[-1]:] == -1).all() and (place >= 0).sum() == counts.sum()


@pytest.mark.parametrize("n,k,m,align,capacity", [(0, 2, 3, 1, 0), (1, 1, 1, 1, 0), (17, 3, 5, 1, 0), (40, 4, 9, 8, 0), (40, 4, 9, 4, 6),
                                                  (40, 2, 3, 16, 1)])
def test_sort(n, k, m, align, capacity):
    idx = choices(n, k, m, n + m)
    plan = oro.sort(idx, m, align, capacity)
    check_plan(idx, m, align, capacity, plan)
    if n > 1:  # the last of an expert first: not stable
        wrong = oro.sort(idx[::-1, ::-1], m, align, capacity)
        with pytest.raises(AssertionError):
            check_plan(idx, m, align, capacity, wrong)


def test_rows_there_and_back():
    r = RNG(3)
    n, k, m, d = 13, 3, 6, 5
    idx = choices(n, k, m, 5)
    slot, _, _, offsets = oro.sort(idx, m, 4)
    rows = oro.sort_rows(n, k, m, 4)
    x, g = r.normal(size=(n, d)), r.normal(size=(rows, d))
    w, dy = r.normal(size=(n, k)), r.normal(size=(n, d))
    behind = np.full((rows, d), 7.0)
    out = oro.dispatch(x, slot, offsets, w, behind)
    assert (out[offsets[-1]:] == 7.0).all()
    # <dispatch(x), g> = <x, combine(g)>, with the weights as without
    for ww in (None, w):
        left = (oro.dispatch(x, slot, offsets, ww, behind)[:offsets[-1]] * g[:offsets[-1]]).sum()
        assert abs(left - (x * oro.combine(g, slot, ww)).sum()) < 1e-12
    # the gradient by differences: the sum is linear in the rows and in the weights
    d_rows, d_w = oro.combine_grad(g, slot, offsets, w, dy, behind)
    h = 1e-3
    for i in range(n):
        for c in range(k):
            up, dn = w.copy(), w.copy()
            up[i, c] += h
            dn[i, c] -= h
            diff = ((oro.combine(g, slot, up) - oro.combine(g, slot, dn)) * dy).sum() / (2 * h)
            assert abs(diff - d_w[i, c]) < 1e-10  # cancellation: some 2^-52 * 30 / h
    for s in range(int(offsets[-1])):
        up, dn = g.copy(), g.copy()
        up[s, 2] += h
        dn[s, 2] -= h
        diff = ((oro.combine(up, slot, w) - oro.combine(dn, slot, w)) * dy).sum() / (2 * h)
        assert abs(diff - d_rows[s, 2]) < 1e-10


def emitted_by(p_scores, q_scores, eps, eps_draft, residual=True):
    """The distribution of a request's first token, the random numbers on a midpoint grid."""
    m, grid = len(p_scores), 400
    q = oro.distribution(q_scores, eps_draft)[0]
    u = (np.arange(grid) + 0.5) / grid
    got = np.zeros(m)
    for x in range(m):
        if q[x] == 0.0:
            continue
        for ua in u:
            acc, nxt, _, _, _ = oro.verify([p_scores], [x], [0, 1], [ua], [0.5], [q_scores], eps, eps_draft)
            if acc[0]:
                got[x] += q[x] / grid
                continue
            p = oro.distribution(p_scores, eps)[0]
            w = np.maximum(p - q, 0.0) if residual else p
            # the draw takes each column for its share of the grid
            got += q[x] / grid * w / w.sum()
            assert nxt[0] == oro.draw(np.maximum(p - q, 0.0), 0.5)
    return got


def test_what_is_emitted_is_distributed_as_the_target():
    r = RNG(9)
    ps, qs = r.normal(size=5), r.normal(size=5)
    ps[3] = -np.inf
    want = oro.distribution(ps, 0.8)[0]
    # each column's acceptance is taken at 400 points: off by at most half a point each
    assert np.abs(emitted_by(ps, qs, 0.8, 1.2) - want).max() < 5 * 0.5 / 400
    assert np.abs(emitted_by(ps, qs, 0.8, 1.2, residual=False) - want).max() > 5 * 0.5 / 400


def test_draw_takes_each_column_for_its_share():
    w = np.array([0.0, 0.25, 0.0, 0.5, 0.25, 0.0])
    assert [oro.draw(w, u) for u in (0.0, 0.2499, 0.25, 0.7499, 0.75, 0.9999, 1.0)] == [1, 1, 3, 3, 4, 4, 4]
    assert oro.draw(np.zeros(3), 0.5) == -1


def test_verify_edges():
    s = np.log(np.array([[0.5, 0.25, 0.25, 0.0], [0.1, 0.2, 0.3, 0.4]]) + 1e-300)
    s[0, 3] = -np.inf
    one = lambda tok, u, row=0, **how: oro.verify(s[row:row + 1], [tok], [0, 1], [u], [0.6], **how)
    assert one(0, 0.49)[0][0] == 1 and one(0, 0.51)[0][0] == 0  # certain proposals: taken with probability p
    assert one(0, 0.51)[1][0] == 2  # of 1 and 2, equally likely, by 0.6
    assert one(3, 0.0)[0][0] == 0 and one(3, 0.0)[3][0] == 0.0  # masked
    assert one(9, 0.0)[0][0] == 0 and one(-1, 0.0)[1][0] == 1  # not in the vocabulary; none drafted
    same = s[:1]
    assert one(1, 0.9999, draft=same)[0][0] == 1
    assert one(1, 1.0, draft=same)[1][0] == 1  # p - q leaves nothing: from p
    assert one(0, 0.0, eps=0.0)[0][0] == 1 and one(1, 0.0, eps=0.0)[1][0] == 0
    acc, nxt, tok, ratio, logp = oro.verify(np.repeat(s[1:], 5, 0), [3, 3, -1, 2, 3], [0, 3, 3, 5], [0.1] * 5, [0.95, 0.5, 0.05])
    assert acc.tolist() == [2, 0, 2] and nxt.tolist() == [3, -1, -1] and tok.tolist() == [3, 3, 3, 2, 3]
    assert np.allclose(logp, np.log([0.4, 0.4, 0.4, 0.3, 0.4])) and np.allclose(ratio, [0.4, 0.4, 0.0, 0.3, 0.4])
    bad = s.copy()
    bad[0, 2] = np.nan
    acc, nxt, tok, ratio, _ = oro.verify(bad, [0, 3], [0, 1, 2], [0.0, 0.0], [0.5, 0.5])
    assert acc.tolist() == [0, 1] and nxt.tolist() == [-1, -1] and np.isnan(ratio[0]) and ratio[1] == pytest.approx(0.4)
