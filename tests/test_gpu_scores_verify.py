"""scores_verify against the float64 reference."""
import numpy as np
import pytest
import torch

import streaming_sinkhorn_solver_amd as sk
from oracle import routed as oro
from scores_cases import DEV, DTYPES, U, close, matrix

pytestmark = pytest.mark.gpu


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def case(lengths, m, dtype, seed, draft=True, pad=0, offset=0, mask=0.0, spread=2.0, tail=0, head=0):
    """Requests of these numbers of rows, the last of each without a drafted token; head and tail: rows of no request.
    (target, draft, tokens, starts, u_accept, u_sample) on the GPU and as numpy."""
    r = np.random.default_rng(seed)
    starts = head + np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    n = int(starts[-1]) + tail
    s, ss = matrix(n, m, dtype, seed, spread, pad, offset, mask)
    q = qs = None
    if draft:
        near = np.where(np.isfinite(ss), ss, 0.0) + r.normal(size=(n, m)) * 0.5
        near[r.random((n, m)) < mask / 2] = -np.inf
        buf = torch.full((offset + n * (m + pad),), float("nan"), dtype=DTYPES[dtype])
        win = buf[offset:].view(n, m + pad)[:, :m]
        win.copy_(torch.from_numpy(near))
        q, qs = buf.to(DEV)[offset:].view(n, m + pad)[:, :m], win.double().numpy()
    tokens = np.full(n, -1, np.int64)
    for a, b in zip(starts[:-1], starts[1:]):
        for i in range(a, b - 1):
            p = oro.distribution(qs[i] if draft else ss[i], 1.0)[0]
            tokens[i] = r.choice(m, p=p / p.sum()) if p.sum() > 0 else r.integers(m)
    ua, us = r.random(n).astype(np.float32), r.random(len(lengths)).astype(np.float32)
    return (s, q, gpu(tokens), gpu(starts), gpu(ua), gpu(us)), (ss, qs, tokens, starts, ua, us)


def check(got, want, scores, eps):
    accepted, after, emitted, ratio, logp = want
    assert np.array_equal(got.accepted.cpu().numpy(), accepted)
    assert np.array_equal(got.next.cpu().numpy(), after)
    assert np.array_equal(got.tokens.cpu().numpy(), emitted)
    # p and q come from float32 sums: a term carries 3 u of its exponent and as much by the moves of the running maximum
    # (weighted mean at most ln m) and 2 u of the exponential; then at most 32 additions of a block, 4 u for each of a
    # thread's blocks (two of them at the least, one per 4096 scores at the most) and 20 u for lanes, waves and parts.
    # All else is float64: exponents off by some 2^-50 of the largest; one rounding to float32.
    m = scores.shape[1]
    one = (6 * np.log(m) + 60 + 4 * (m / 4096 + 2)) * U
    big = np.abs(np.where(np.isfinite(scores), scores, 0.0)).max(initial=1.0) / (eps or 1.0)
    noise = (big + 64) * 2.0 ** -48
    close(got.ratio, ratio, (2 * one + U) * np.abs(ratio) + noise + 2.0 ** -149, "ratio")
    close(got.logp, logp, one + U * np.abs(logp) + noise, "logp")


def run(data, ref, eps=1.0, eps_draft=1.0, **how):
    s, q, tokens, starts, ua, us = data
    got = sk.scores_verify(s, tokens, starts, ua, us, draft=q, eps=eps, eps_draft=eps_draft, **how)
    ss, qs, tokens, starts, ua, us = ref
    check(got, oro.verify(ss, tokens, starts, ua, us, qs, eps, eps_draft), ss, eps)
    return got


# one column; around a run of 16 bytes, a wave's row (512 runs), four chunks of the draw (512 entries at these sizes), a part of a cut row
COLUMNS = [1, 2, 5, 8, 33, 511, 2047, 2048, 2049, 4096, 4099, 8192, 8200, 50001, 131072]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m", COLUMNS)
@pytest.mark.parametrize("draft", [True, False])
def test_shapes(m, dtype, draft):
    lengths = [3, 1, 5] if m > 4000 else [4, 1, 7, 2, 1, 3, 9, 2]
    data, ref = case(lengths, m, dtype, m + draft, draft, pad=m % 3, offset=m % 2)
    run(data, ref)
    run(data, ref, eps=0.7, eps_draft=1.4)
    run(data, ref, eps=0.0)


@pytest.mark.parametrize("m", [7, 300, 5000, 40000])
@pytest.mark.parametrize("mask", [0.5, 0.99])
@pytest.mark.parametrize("draft", [True, False])
def test_masks(m, mask, draft):
    """Masked columns are neither taken nor drawn, also where they leave a row nothing."""
    data, ref = case([3, 2, 1, 4, 1, 2], m, "f32", m, draft, mask=mask)
    s, ss = data[0], ref[0]
    for i in (1, 5):  # an empty target row, with and without a drafted token
        s[i] = -float("inf")
        ss[i] = -np.inf
    if draft:
        data[1][7] = -float("inf")
        ref[1][7] = -np.inf
    run(data, ref)
    run(data, ref, eps=0.0)
    got = run(data, ref, eps=1.5)
    rows = got.tokens >= 0
    assert torch.isfinite(s[rows, got.tokens[rows]]).all()
    # the type's lowest value in place of -inf
    low = torch.finfo(torch.float32).min
    s.masked_fill_(s == -float("inf"), low)
    ss[ss == -np.inf] = low
    run(data, ref)
    run(data, ref, eps=0.0)


@pytest.mark.parametrize("lengths", [[1] * 200, [0, 3, 0, 0, 2, 0], [70, 1, 130], [2] * 70 + [0] * 70 + [1] * 70, [1]])
def test_requests(lengths):
    """Many, empty and long requests; rows before the first and behind the last are left as they are."""
    data, ref = case(lengths, 50, "bf16", len(lengths), True, head=2, tail=3)
    s, q, tokens, starts, ua, us = data
    ua *= 0.5  # most are taken
    ref[4][:] *= np.float32(0.5)
    ss, qs, t, st, a, u = ref
    n, b = len(t), len(u)
    for eps in (0.8, 0.0):
        out = sk.Verified(torch.full((b,), 77, dtype=torch.int32, device=DEV), torch.full((b,), 77, device=DEV),
                          torch.full((n,), 77, device=DEV), torch.full((n,), 77.0, device=DEV), torch.full((n,), 77.0, device=DEV))
        got = sk.scores_verify(s, tokens, starts, ua, us, draft=q, eps=eps, out=out)
        assert got.tokens.data_ptr() == out.tokens.data_ptr()
        fill = (np.full(n, 77), np.full(n, 77.0), np.full(n, 77.0))
        check(got, oro.verify(ss, t, st, a, u, qs, eps, 1.0, fill), ss, eps)
        # the emitted tokens over the drafted ones
        over = tokens.clone()
        over_got = sk.scores_verify(s, over, starts, ua, us, draft=q, eps=eps,
                                    out=out._replace(tokens=over, accepted=torch.empty_like(out.accepted)))
        assert torch.equal(over_got.tokens[2:n - 3], got.tokens[2:n - 3]) and torch.equal(over_got.accepted, got.accepted)


def test_padded_requests():
    """Requests of equal numbers of rows that end at their first row without a drafted token; or at none."""
    n_rows, m = 6, 333
    data, ref = case([n_rows] * 9, m, "f32", 5, True)
    s, q, tokens, starts, ua, us = data
    ss, qs, t, st, a, u = ref
    for r in range(9):
        if r < 7:
            t[r * n_rows + r % n_rows] = -1  # drafted tokens behind it take no part
    t[8 * n_rows + n_rows - 1] = 3  # the last has none without one
    a[8 * n_rows:] = 0.0
    data, ref = (s, q, gpu(t), starts, gpu(a), us), (ss, qs, t, st, a, u)
    got = run(data, ref)
    assert int(got.accepted[8]) == n_rows and int(got.next[8]) == -1
    run(data, ref, eps=0.0)
    # rows that no request looks at may hold anything
    for r in range(7):
        s[r * n_rows + r % n_rows + 1:(r + 1) * n_rows] = float("nan")
        q[r * n_rows + r % n_rows:(r + 1) * n_rows] = float("nan")
    again = sk.scores_verify(s, data[2], starts, data[4], us, draft=q)
    for x, y in zip(again, got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("m", [40, 9000])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_bad_scores(m, value):
    """A NaN or +inf score: its row takes and draws nothing, no other row is touched."""
    data, ref = case([2, 2, 2, 3, 1], m, "f32", m, True)
    s, q, ss, qs = data[0], data[1], ref[0], ref[1]
    for i, j in ((0, 0), (5, m - 1), (9, m // 2)):
        s[i, j] = value
        ss[i, j] = value
    q[2, 3] = value
    qs[2, 3] = value
    run(data, ref)
    ref[1][:] = np.where(np.isfinite(qs), qs, 0.0)  # greedy does not look at the draft's scores
    run(data, ref, eps=0.0)


def test_extreme_scores_and_temperatures():
    for dtype, big in (("f32", 1e38), ("bf16", 1e38), ("f16", 6e4)):
        data, ref = case([3, 2, 4, 1], 600, dtype, 3, True)
        s, q, ss, qs = data[0], data[1], ref[0], ref[1]
        s[1, 5], ss[1, 5] = big, float(torch.tensor(big, dtype=DTYPES[dtype]))
        s[4], ss[4] = -big, -float(torch.tensor(big, dtype=DTYPES[dtype]))
        q[2, 7], qs[2, 7] = -big, -float(torch.tensor(big, dtype=DTYPES[dtype]))
        run(data, ref)
        run(data, ref, eps=1e-3, eps_draft=1e-2)
        run(data, ref, eps=100.0, eps_draft=1e6)
    # each part of a row far above the ones before it, and the other way round
    m = 30000
    for sign in (1, -1):
        data, ref = case([2, 1], m, "f32", 8, False)
        ramp = np.linspace(0, 3000, m).astype(np.float32) * sign
        data[0][:] = gpu(np.tile(ramp, (3, 1)))
        ref[0][:] = ramp.astype(np.float64)
        run(data, ref)
        run(data, ref, eps=300.0)


def test_random_numbers_at_their_borders():
    """u = 0, the largest below 1, 1, and ones that a caller should not pass."""
    data, ref = case([2, 2, 2, 2], 64, "f32", 2, True, mask=0.3)
    s, q, tokens, starts, _, _ = data
    below = float(np.nextafter(np.float32(1), np.float32(0)))
    for ua in (0.0, below, 1.0):
        for us in (0.0, below, 1.0):
            a, u = np.full(8, ua, np.float32), np.full(4, us, np.float32)
            run((s, q, tokens, starts, gpu(a), gpu(u)), ref[:4] + (a, u))
    for odd in (float("nan"), -1.0, 2.0, float("inf"), -float("inf")):
        a, u = torch.full((8,), odd, device=DEV), torch.full((4,), odd, device=DEV)
        for draft in (q, None):
            got = sk.scores_verify(s, tokens, starts, a, u, draft=draft)
            rows = got.tokens >= 0
            assert (got.tokens < 64).all() and torch.isfinite(s[rows, got.tokens[rows]]).all()


@pytest.mark.parametrize("m", [300, 20000])
@pytest.mark.parametrize("draft", [True, False])
def test_decisions_next_to_the_border(m, draft):
    """u just below and just above p / q: float32 numbers around it, closer than float32 sums can tell."""
    lengths = [4] * 40
    data, ref = case(lengths, m, "f32", m, draft)
    s, q, tokens, starts, ua, us = data
    ss, qs, t, st, a, u = ref
    n = len(t)
    r = np.random.default_rng(7)
    for i in range(n):
        if t[i] < 0:
            continue
        p = oro.distribution(ss[i], 1.0)[0][t[i]]
        x = p / oro.distribution(qs[i], 1.0)[0][t[i]] if draft else p
        v = np.float32(min(x, 1.0))
        a[i] = np.nextafter(v, np.float32(r.integers(0, 2) * 2)) if r.random() < 0.7 else v
    run((s, q, tokens, starts, gpu(a), us), (ss, qs, t, st, a, u))


def test_tokens_of_no_column():
    data, ref = case([2, 2, 3], 20, "f32", 4, True)
    t = ref[2]
    t[0], t[2], t[5] = 20, 2 ** 62, 21
    for draft in (True, False):
        data2 = (data[0], data[1] if draft else None, gpu(t)) + data[3:]
        ref2 = (ref[0], ref[1] if draft else None) + ref[2:]
        got = run(data2, ref2)
        assert int(got.accepted[0]) == 0 and int(got.accepted[1]) == 0
        run(data2, ref2, eps=0.0)


def test_same_distribution_is_always_taken_and_p_is_kept():
    """p = q: every token is taken.  What is emitted over many draws is distributed as p."""
    data, ref = case([4] * 50, 500, "bf16", 6, True)
    s, _, tokens, starts, ua, us = data
    got = sk.scores_verify(s, tokens, starts, ua, us, draft=s)
    assert (got.accepted == 3).all() and (got.ratio.view(50, 4)[:, :3] == 1.0).all()
    m, b = 6, 60000
    r = np.random.default_rng(0)
    ps, qs = r.normal(size=m), r.normal(size=m)
    p, q = (oro.distribution(v.astype(np.float32), 1.0)[0] for v in (ps, qs))
    x = r.choice(m, size=b, p=q / q.sum())
    t = np.stack([x, np.full(b, -1)], 1).reshape(-1)
    got = sk.scores_verify(gpu(np.tile(ps.astype(np.float32), (2 * b, 1))), gpu(t), gpu(np.arange(b + 1) * 2), torch.rand(2 * b, device=DEV),
                           torch.rand(b, device=DEV), draft=gpu(np.tile(qs.astype(np.float32), (2 * b, 1))))
    share = np.bincount(got.tokens[::2].cpu().numpy(), minlength=m) / b
    assert np.abs(share - p).max() < 6 * 0.5 / np.sqrt(b)  # six standard deviations


def test_ties_of_greedy():
    for m in (16, 3000, 70000):
        s = torch.zeros(4, m, device=DEV)
        s[1, 7:] = 2.0
        s[2, m - 1] = 1.0
        s[3, 2] = s[3, m - 2] = 5.0
        tokens = torch.tensor([0, 7, m - 1, -1], device=DEV)
        got = sk.scores_verify(s, tokens, torch.tensor([0, 4], device=DEV), None, None, eps=0.0)
        assert got.accepted.tolist() == [3] and got.next.tolist() == [2] and got.tokens.tolist() == [0, 7, m - 1, 2]


def test_refusals():
    data, _ = case([2, 2], 30, "f32", 1, True)
    s, q, tokens, starts, ua, us = data
    call = lambda **how: sk.scores_verify(**{**dict(scores=s, tokens=tokens, starts=starts, u_accept=ua, u_sample=us, draft=q), **how})
    call()
    for bad in (dict(tokens=tokens.int()), dict(tokens=tokens[:3]), dict(tokens=None), dict(starts=starts.int()), dict(starts=starts[:0]),
                dict(starts=starts[None]), dict(u_accept=ua.double()), dict(u_accept=None), dict(u_sample=us[:1]), dict(u_sample=None),
                dict(draft=q.half()), dict(draft=q[:3]), dict(draft=q[:, :29]), dict(draft=q.cpu()), dict(eps=-1.0), dict(eps_draft=0.0),
                dict(eps=float("nan")), dict(ws=torch.empty(16, device=DEV)), dict(tokens=tokens.cpu())):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    with pytest.raises(sk.SinkhornError, match="SK_ERR_WORKSPACE"):
        call(ws=torch.empty(256, dtype=torch.uint8, device=DEV))


def test_no_rows_and_no_requests():
    empty = torch.empty(0, 12, device=DEV)
    none, zeros = torch.empty(0, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    for eps in (1.0, 0.0):
        got = sk.scores_verify(empty, zeros[:0], zeros, none, torch.rand(2, device=DEV), eps=eps)
        assert got.accepted.tolist() == [0, 0] and got.next.tolist() == [-1, -1] and got.tokens.numel() == 0
        got = sk.scores_verify(torch.zeros(2, 12, device=DEV), zeros[:2], zeros[:1], torch.rand(2, device=DEV), none, eps=eps)
        assert got.accepted.numel() == 0


def test_streams_graphs_and_determinism():
    m = 20000
    data, ref = case([4, 2, 6, 1, 5], m, "bf16", 11, True)
    s, q, tokens, starts, ua, us = data
    want = sk.scores_verify(s, tokens, starts, ua, us, draft=q)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        got = sk.scores_verify(s, tokens, starts, ua, us, draft=q)
    other.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    n, b = s.shape[0], 5
    for eps in (1.0, 0.0):
        ws = sk.scores_verify_workspace(s.dtype, n, m, b, DEV)
        out = sk.scores_verify(s, tokens, starts, ua, us, draft=q, eps=eps, ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sk.scores_verify(s, tokens, starts, ua, us, draft=q, eps=eps, ws=ws, out=out)
        for step in range(4):
            ua.copy_(torch.rand(n, device=DEV))
            us.copy_(torch.rand(b, device=DEV))
            s.copy_(torch.randn(n, m, device=DEV) * 2)
            ws.fill_(step * 37)  # what the workspace held does not matter
            graph.replay()
            torch.cuda.synchronize()
            eager = sk.scores_verify(s, tokens, starts, ua, us, draft=q, eps=eps)
            assert all(torch.equal(x, y) for x, y in zip(out, eager)), (eps, step)
