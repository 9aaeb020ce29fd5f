"""scores_verify where a request or a row lies at the border of what there is: starts outside the matrix, scores further
apart than float32 reaches, a residual that is next to nothing; and every layout of the draw's chunks."""
import numpy as np
import pytest
import torch

import streaming_sinkhorn_solver_amd as sk
from oracle import routed as oro
from scores_cases import DEV
from test_gpu_scores_verify import case, check, gpu, run

pytestmark = pytest.mark.gpu


# the first request's first row is row 0 of the matrix, the last one's last row is row n - 1; some are empty
@pytest.mark.parametrize("starts", [[-2, 3], [-5, -1, 2, 9], [-3, -3, 4], [-7, 0, 5], [-9, -4], [0, 3, 40], [2, 7, 12, 30], [-1, 60], [12, 15],
                                    [-2 ** 62, 4, 2 ** 62]])
@pytest.mark.parametrize("m", [50, 9000])
@pytest.mark.parametrize("draft", [True, False])
def test_starts_outside_the_matrix(starts, m, draft):
    n = 12
    data, ref = case([n], m, "f32", m + len(starts), draft)
    s, q, tokens, _, ua, _ = data
    ss, qs, t, _, a, _ = ref
    t[5] = t[8] = -1
    st = np.array(starts, np.int64)
    b = len(st) - 1
    u = np.random.default_rng(b).random(b).astype(np.float32)
    tokens, ua = gpu(t), ua * 0.5
    a = a * np.float32(0.5)
    for eps in (0.8, 0.0):
        want = oro.verify(ss, t, np.clip(st, 0, n), a, u, qs, eps, 1.0, (np.full(n, 77), np.full(n, 77.0), np.full(n, 77.0)))
        for byte in (0, 0x11, 0x3f, 0x7f, 0xff):  # what the workspace held does not matter
            ws = sk.scores_verify_workspace(s.dtype, n, m, b, DEV).fill_(byte)
            out = sk.Verified(*(torch.full((size,), 77, dtype=dtype, device=DEV) for size, dtype in
                                ((b, torch.int32), (b, torch.int64), (n, torch.int64), (n, torch.float32), (n, torch.float32))))
            check(sk.scores_verify(s, tokens, gpu(st), ua, gpu(u), draft=q, eps=eps, ws=ws, out=out), want, ss, eps)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [40, 3000, 20000])
def test_draft_rows_that_are_not_there(m, dtype):
    """Rows of the draft without a drafted token are not read: the matrix may end before the last request's last row."""
    data, ref = case([3, 2, 1, 4], m, dtype, m, True)
    s, q, tokens, starts, ua, us = data
    n, b = s.shape[0], 4
    want = sk.scores_verify(s, tokens, starts, ua, us, draft=q)
    short = torch.full((n - 1, m), float("nan"), dtype=q.dtype, device=DEV)
    rows = (tokens >= 0).nonzero()[:, 0]
    short[rows] = q[rows]
    out = [torch.empty_like(t) for t in want]
    ws = sk.scores_verify_workspace(s.dtype, n, m, b, DEV)
    code = sk.load_library().sk_scores_verify(
        s.data_ptr(), sk.DTYPES[s.dtype], n, m, s.stride(0), 1.0, short.data_ptr(), m, 1.0, tokens.data_ptr(), starts.data_ptr(), b,
        ua.data_ptr(), us.data_ptr(), *(t.data_ptr() for t in out), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert code == 0
    for got, ref_ in zip(out, want):
        assert torch.equal(got, ref_)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [2, 5, 600, 30000])
@pytest.mark.parametrize("draft", [True, False])
def test_scores_further_apart_than_float32_reaches(m, dtype, draft):
    """Differences of scores beyond the largest float32, at temperatures where they count."""
    data, ref = case([3, 2, 4, 1], m, dtype, m, draft)
    s, q, ss, qs = data[0], data[1], ref[0], ref[1]
    r = np.random.default_rng(m)
    for i in range(10):
        for win, held in ((s, ss), (q, qs)):
            if win is None:
                continue
            x = r.choice([-3e38, 3e38, -2e38, 1e38, 0.0], m)
            x[r.integers(m)] = -3e38 if i % 2 else 3e38  # (a thread's first scores far below or above the others)
            win[i] = gpu(x).to(win.dtype)
            held[i] = win[i].double().cpu().numpy()
    for eps in (1e38, 3e37, 5e36):
        run(data, ref, eps=eps, eps_draft=eps)
        run(data, ref, eps=eps, eps_draft=1.2e38)
    run(data, ref, eps=1.0, eps_draft=1e-30)


def next_to_proportional(m, seed, off):
    """A target's and a draft's row whose probabilities are alike but for one column in 512 that the target raises by some
    2^-28 each, and a drafted one that it lowers so far that the sums differ by `off` of what was added.  The draft's
    scores are 1.5 times as large, at 1.5 times the temperature, so float32 sums of the two differ by roundings."""
    r = np.random.default_rng(seed)
    base = np.round(r.normal(size=m) * 32) / 16
    top = base.max()
    first = np.arange(0, m, 512)
    up = first + r.integers(0, 1 << 30, len(first)) % np.minimum(512, m - first)
    base[up] = top - 16 - np.round(r.random(len(up)) * 16) / 16
    added = (np.exp(base[up] - top) * (np.e - 1)).sum()
    down = (up[0] + 1) % m
    base[down] = np.round(16 * (top + np.log(4 * added))) / 16
    s = base.astype(np.float32)
    s[up] += 1
    s[down] = np.float32(top + np.log(np.exp(base[down] - top) - added * (1 - off)))
    return s, (1.5 * base).astype(np.float32), down


@pytest.mark.parametrize("off", [0.5, 0.1, 0.02, 0.0, -0.1, -0.5, -2.0])
@pytest.mark.parametrize("m,b", [(20000, 4), (20000, 512), (700, 1200), (140000, 6)])
def test_residual_next_to_nothing(m, b, off):
    """The draw is that of the exact residual also where p and q are alike in nearly all of the row and what is left is 2^-21 or
    less.  An exponential is within 2^-38 of itself, and in a column where p and q are alike both carry the same error, so
    borders are within some 2^-17 of what is left; the random numbers keep 2^-13 away from every one."""
    kinds = 4
    rows = [next_to_proportional(m, 10 * k + m, off) for k in range(kinds)]
    r = np.random.default_rng(b)
    s, q, tokens = np.zeros((2 * b, m), np.float32), np.zeros((2 * b, m), np.float32), np.full(2 * b, -1, np.int64)
    us, want = np.zeros(b, np.float32), np.zeros(b, np.int64)
    for k, (target, draft, down) in enumerate(rows):
        w = np.maximum(oro.distribution(target, 1.0)[0] - oro.distribution(draft, 1.5)[0], 0.0)
        w /= w.sum()
        ends = np.cumsum(w)
        heavy = np.nonzero(w > 2.0 ** -11)[0]
        for i in range(k, b, kinds):
            j = int(r.choice(heavy))
            us[i] = ends[j] - w[j] * r.uniform(0.3, 0.7)
            if off > 0.0 and i < 2 * kinds and i % 2:  # (only the raised columns are left)
                j, us[i] = int(np.nonzero(w)[0][0]), 0.0
            s[2 * i], q[2 * i], tokens[2 * i], want[i] = target, draft, down, j
    got = sk.scores_verify(gpu(s), gpu(tokens), gpu(2 * np.arange(b + 1)), torch.full((2 * b,), 0.97, device=DEV), gpu(us),
                           draft=gpu(q), eps=1.0, eps_draft=1.5)
    assert (got.accepted == 0).all()
    assert np.array_equal(got.next.cpu().numpy(), want)


# A chunk of the draw is 512 entries where b m is 2^21 at most, 1024 up to 2^22, 2048 beyond.  Up to 256 chunks are added up
# by the threads at once, more in turns; with 1024 requests or more a request's chunks are one workgroup's.
LAYOUTS = [([4], 131072), ([4], 131073), ([3, 1], 151936), ([2], 201089), ([2], 262144), ([2], 600011),  # 512, 256 chunks and more
           ([2] * 60, 43008), ([2] * 60, 43007), ([2] * 50, 46081),                                       # 1024
           ([2] * 120, 40961), ([2] * 120, 40960), ([2, 1] * 9, 270337),                                  # 2048
           ([2] * 1100, 9001), ([1, 2] * 600, 513)]                                                       # a workgroup per request


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("lengths,m", LAYOUTS, ids=lambda v: f"{len(v)}x{v[0]}" if isinstance(v, list) else str(v))
def test_layouts_of_the_draw(lengths, m, draft, dtype):
    data, ref = case(lengths, m, dtype, m, draft)
    b, r = len(lengths), np.random.default_rng(m)
    below = np.nextafter(np.float32(1), np.float32(0))
    run(data, ref)
    # what is drawn at the ends and in the middle of the row, also where all drafted tokens but the last are taken
    for u in ((0.0, below, 0.5) if b < 4 else (np.where(r.random(b) < 0.5, 0.0, below),)):
        a, u = np.where(r.random(len(ref[4])) < 0.5, below, 0.0).astype(np.float32), np.broadcast_to(u, b).astype(np.float32)
        run(data[:4] + (gpu(a), gpu(u)), ref[:4] + (a, u))


@pytest.mark.parametrize("m,b", [(9001, 2), (9001, 1100), (131073, 3), (151936, 3), (50001, 64)])
def test_nothing_left_to_draw_from(m, b):
    """p = q and a drafted token that is refused all the same: the draw is from p; also in a row whose mass is at its ends."""
    data, ref = case([2] * b, m, "f32", b, True)
    s, ss = data[0], ref[0]
    s[:2, 1:m - 1] = -float("inf")
    ss[:2, 1:m - 1] = -np.inf
    a = np.ones(2 * b, np.float32)
    t = ref[2].copy()
    t[0] = 0
    got = run((s, s, gpu(t), data[3], gpu(a), data[5]), (ss, ss, t, ref[3], a, ref[5]))
    assert (got.accepted == 0).all() and (got.next >= 0).all()
