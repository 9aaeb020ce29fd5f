"""scores_logprobs and its gradient against the float64 reference."""
import numpy as np
import pytest
import torch

import streaming_sinkhorn_solver_amd as sk
from oracle import scores as osc
from scores_cases import DEV, U, close, entropy_error, half_step, log_sum_error, matrix, softmax_terms

pytestmark = pytest.mark.gpu


def targets_of(n, m, seed):
    r = np.random.default_rng(seed)
    t = r.integers(0, m, n)
    t[r.random(n) < 0.2] = -1
    return t


def check_forward(r, ref, s, t, eps, top):
    d, p, log_s, e1, e2 = softmax_terms(s, eps)
    err = log_sum_error(e1)
    close(r.lse, ref["lse"], 4 * U * np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0))
          + 4 * U * np.abs(np.where(np.isfinite(s.max(1)), s.max(1), 0.0)) / eps + err, "lse")
    if t is not None:
        close(r.logp, ref["logp"], err + 4 * U * np.abs(np.where(np.isfinite(ref["logp"]), ref["logp"], 0.0))
              + 4 * U * np.abs(log_s), "logp")
    if r.entropy is not None:
        close(r.entropy, ref["entropy"], entropy_error(log_s, e1, e2), "entropy")
    if top:
        assert np.array_equal(r.top_idx.cpu().numpy(), ref["top_idx"])
        close(r.top_logp, ref["top_logp"], err[:, None] + 4 * U * np.abs(log_s)[:, None]
              + 4 * U * np.abs(np.where(np.isfinite(ref["top_logp"]), ref["top_logp"], 0.0)), "top_logp")


def check_grad(grad, s, t, eps, dtype, fwd_idx, d):
    """p carries (3 |d| + 4) u, the sum's error and that of log S; the bracket's terms their own roundings and the
    entropy's error; the result is rounded once to the scores' type (below its normal range by half its smallest step)."""
    want = osc.logprobs_grad(s, t, eps, fwd_idx, **d)
    fd, p, log_s, e1, e2 = softmax_terms(s, eps)
    zero = np.zeros(len(s))
    dl = np.abs(d.get("d_logp", zero)) if t is not None else zero
    dt = np.abs(d["d_top"]).sum(1) if "d_top" in d else zero
    de, dlse = np.abs(d.get("d_entropy", zero)), np.abs(d.get("d_lse", zero))
    logs = np.abs(fd) + np.abs(log_s)[:, None]
    bracket = (dl + dt + dlse)[:, None] + de[:, None] * (logs + 2 * e1[:, None])
    rel = (3 * np.abs(fd) + 80) * U + log_sum_error(e1)[:, None] + 4 * U * np.abs(log_s)[:, None]
    tol = p * (bracket * rel + (de * entropy_error(log_s, e1, e2))[:, None]) / eps
    tol = tol + 70 * U * (dl + dt)[:, None] / eps * (np.abs(want) > 0)
    info = torch.finfo(grad.dtype)
    tol = tol + half_step(dtype) * np.abs(want) * (1 + 1e-3) + info.smallest_normal * info.eps / 2
    close(grad, want, tol, "grad")


# one row and one column; around every chunk size (128 and 512 vectors of a wave, 1024 and 4096 of a workgroup, with
# 4 or 8 scores each), rows that start and end inside 16 bytes, several chunks
SHAPES = [(1, 1, 0, 0), (5, 2, 1, 1), (3, 7, 0, 3), (40, 33, 2, 1), (9, 511, 3, 2), (9, 512, 0, 0), (6, 1025, 1, 5),
          (7, 2047, 6, 7), (5, 2049, 0, 0), (4, 4097, 7, 1), (3, 8193, 0, 0), (2, 16384, 0, 0), (3, 16391, 5, 3),
          (2, 32769, 0, 1), (2, 50001, 0, 0), (1, 131072, 0, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,m,pad,offset", SHAPES)
def test_forward_shapes(n, m, pad, offset, dtype):
    x, s = matrix(n, m, dtype, n + m, pad=pad, offset=offset)
    t = targets_of(n, m, m)
    for top in sorted({0, 1, min(m, 5), min(m, 64)}):
        r = sk.scores_logprobs(x, torch.from_numpy(t).to(DEV), eps=0.7, top=top, entropy=top != 1)
        assert (r.entropy is None) == (top == 1) and (r.top_idx is None) == (top == 0)
        check_forward(r, osc.logprobs(s, t, 0.7, top), s, t, 0.7, top)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,m,pad,offset", SHAPES)
def test_gradient_shapes(n, m, pad, offset, dtype):
    x, s = matrix(n, m, dtype, 3 * n + m, pad=pad, offset=offset)
    t = targets_of(n, m, m + 1)
    r = np.random.default_rng(n * m)
    top = min(m, 6)
    fwd = sk.scores_logprobs(x, torch.from_numpy(t).to(DEV), eps=1.3, top=top, entropy=True)
    d = {k: r.normal(size=(n, top) if k == "d_top" else n).astype(np.float32) for k in
         ("d_logp", "d_lse", "d_entropy", "d_top")}
    gpu = {k: torch.from_numpy(v).to(DEV) for k, v in d.items()}
    idx = fwd.top_idx.cpu().numpy()
    tg = torch.from_numpy(t).to(DEV)
    for keys in (("d_logp",), ("d_lse", "d_top"), ("d_logp", "d_lse", "d_entropy", "d_top")):
        grad = sk.scores_logprobs_grad(x, tg, fwd, eps=1.3, **{k: gpu[k] for k in keys})
        check_grad(grad, s, t, 1.3, dtype, idx, {k: d[k] for k in keys})
    # into a buffer of another alignment, and over the scores themselves: the same bits
    wide = torch.full((n, m + 5), 7.0, dtype=x.dtype, device=DEV)
    sk.scores_logprobs_grad(x, tg, fwd, eps=1.3, grad=wide[:, 3:m + 3], **gpu)
    assert torch.equal(wide[:, 3:m + 3], grad) and (wide[:, :3] == 7).all() and (wide[:, m + 3:] == 7).all()
    own = torch.full((offset + n * (m + pad),), 7.0, dtype=x.dtype, device=DEV)
    own = own[offset:].view(n, m + pad)
    own[:, :m] = x
    sk.scores_logprobs_grad(own[:, :m], tg, fwd, eps=1.3, grad=own[:, :m], **gpu)
    assert torch.equal(own[:, :m], grad) and (own[:, m:] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m", [40, 1000, 9000, 40000])
@pytest.mark.parametrize("mask", [0.5, 0.999])
def test_masks(m, dtype, mask):
    """Most of a row masked, whole rows masked, and the lowest finite value in place of a mask."""
    n, top = 6, min(m, 20)
    x, s = matrix(n, m, dtype, m, mask=mask, offset=1, pad=1)
    x[2], s[2] = -float("inf"), -np.inf
    lowest = torch.finfo(x.dtype).min
    x[3, 1:], s[3, 1:] = lowest, lowest
    x[4], s[4] = lowest, lowest
    t = np.array([0, m // 2, 3, 1, 5, m - 1])
    tg = torch.from_numpy(t).to(DEV)
    r = sk.scores_logprobs(x, tg, top=top, entropy=True)
    ref = osc.logprobs(s, t, 1.0, top)
    check_forward(r, ref, s, t, 1.0, top)
    rng = np.random.default_rng(m)
    d = dict(d_logp=rng.normal(size=n).astype(np.float32), d_entropy=rng.normal(size=n).astype(np.float32),
             d_lse=rng.normal(size=n).astype(np.float32))
    grad = sk.scores_logprobs_grad(x, tg, r, **{k: torch.from_numpy(v).to(DEV) for k, v in d.items()})
    check_grad(grad, s, t, 1.0, dtype, None, d)


@pytest.mark.parametrize("kind", ["equal", "rounded", "ascending", "descending", "one_class", "late"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [300, 3000, 30000, 70001])
def test_top_orders(m, dtype, kind):
    """Alternatives where the largest entries crowd: all equal, many ties, sorted rows, all in one class of lanes."""
    n, top = 3, 64
    x, s = matrix(n, m, dtype, m, ties=kind == "rounded")
    if kind != "rounded":
        j = np.arange(m)
        row = {"equal": np.zeros(m), "ascending": j / m, "descending": -j / m,
               "one_class": np.where(j % 512 < 8, 5.0 + (j * 7 % 1024) / 1024, 0.0),
               "late": np.where(j >= m - 70, 1.0, 0.0)}[kind]
        x[:] = torch.from_numpy(row).to(DEV)
        s = x.double().cpu().numpy()
    r = sk.scores_logprobs(x, top=top)
    check_forward(r, osc.logprobs(s, None, 1.0, top), s, None, 1.0, top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,lanes", [(1500, 20), (3000, 20), (9000, 40), (70001, 40)])
def test_more_crowded_entries_than_the_list_holds(m, lanes, dtype):
    """The largest entries all lie in the columns of a few threads, more of them than are kept: fewer classes than k."""
    n, top = 3, 64
    per = 8 if dtype == "bf16" else 4  # scores of 16 bytes
    r = np.random.default_rng(m)
    v = np.arange(m) // per % (64 if m <= 3000 else 256)
    x = torch.from_numpy(np.where(v < lanes, 10.0 + r.normal(size=(n, m)), r.normal(size=(n, m))).astype(np.float32)).to(DEV)
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    s = x.double().cpu().numpy()
    r = sk.scores_logprobs(x, top=top)
    check_forward(r, osc.logprobs(s, None, 1.0, top), s, None, 1.0, top)


@pytest.mark.parametrize("kind", ["equal", "two_values", "masked", "rounded"])
def test_ties_in_whole_rows(kind):
    """Enough rows that none is cut: more blocks reach the bound than the list of them holds."""
    n, m, top = 1030, 17003, 20
    x = torch.zeros((n, m), dtype=torch.bfloat16, device=DEV)
    torch.manual_seed(3)
    if kind == "two_values":
        x[torch.rand((n, m), device=DEV) < 0.3] = 1.0
    elif kind == "masked":
        x[torch.rand((n, m), device=DEV) < 0.9995] = -float("inf")
    elif kind == "rounded":
        x.copy_(torch.randn((n, m), device=DEV).round())
    r = sk.scores_logprobs(x, top=top)
    order = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(r.top_idx.long(), order)
    want = torch.log_softmax(x.double(), 1)
    lse = torch.logsumexp(x.double(), 1)
    # 400 half steps (150 additions, the terms' own errors, the logarithm) of values below 16
    assert (r.lse - lse).abs().max() < 400 * U * 16
    got = want.gather(1, order)
    fin = torch.isfinite(got)
    assert torch.equal(torch.isfinite(r.top_logp), fin) and (r.top_logp - got)[fin].abs().max() < 400 * U * 16


def test_nan_and_infinity_stay_in_their_rows():
    x, s = matrix(5, 5000, "f32", 1)
    x[1, 77] = float("nan")
    x[3, 4] = float("inf")
    x[4, :4990] = float("nan")
    t = torch.arange(5, device=DEV)
    r = sk.scores_logprobs(x, t, top=30, entropy=True)
    for v in (r.lse, r.logp, r.entropy, r.top_logp):
        assert torch.isnan(v[[1, 3, 4]]).all() and torch.isfinite(v[[0, 2]]).all()
    idx = r.top_idx.long()
    assert (idx >= 0).all() and (idx < 5000).all()
    assert all(len(set(row.tolist())) == 30 for row in idx) and idx[3, 0] == 4
    # the ten numbers of row 4 first, then its NaN by their columns
    assert sorted(idx[4, :10].tolist()) == list(range(4990, 5000)) and idx[4, 10:].tolist() == list(range(20))
    g = sk.scores_logprobs_grad(x, t, r, d_logp=torch.ones(5, device=DEV))
    assert torch.isfinite(g[[0, 2]]).all()


def test_targets_outside_the_row():
    x, s = matrix(4, 100, "f32", 2)
    t = torch.tensor([100, -1, -(1 << 40), 1 << 40], device=DEV)
    r = sk.scores_logprobs(x, t)
    assert torch.isnan(r.logp[[0, 3]]).all() and (r.logp[[1, 2]] == 0).all() and torch.isfinite(r.lse).all()
    g = sk.scores_logprobs_grad(x, t, r, d_logp=torch.ones(4, device=DEV))
    assert torch.isnan(g[[0, 3]]).all() and (g[[1, 2]] == 0).all()


def test_no_rows_and_many_rows():
    r = sk.scores_logprobs(torch.empty((0, 9), device=DEV), torch.empty(0, dtype=torch.int64, device=DEV), top=3, entropy=True)
    assert r.logp.shape == (0,) and r.top_idx.shape == (0, 3)
    g = sk.scores_logprobs_grad(torch.empty((0, 9), device=DEV), None, r, d_lse=torch.empty(0, device=DEV))
    assert g.shape == (0, 9)
    n = (1 << 20) + 77  # more rows than workgroups of a launch
    x = torch.randn((n, 5), device=DEV)
    t = torch.randint(0, 5, (n,), device=DEV)
    r = sk.scores_logprobs(x, t, top=2)
    want = torch.log_softmax(x.double(), 1)  # 200 half steps of log-probabilities below 8, of gradients below 2
    assert (r.logp - want.gather(1, t[:, None])[:, 0]).abs().max() < 200 * U * 8
    assert torch.equal(r.top_idx[:, 0].long(), x.argmax(1))
    g = sk.scores_logprobs_grad(x, t, r, d_logp=torch.ones(n, device=DEV))
    assert (g + want.exp() - torch.nn.functional.one_hot(t, 5)).abs().max() < 200 * U * 2


def test_offsets_beyond_32_bits():
    """Rows 2^32 and more elements away from the first."""
    n, m, ld = 3, 1000, (1 << 31) + 8
    buf = torch.zeros(2 * ld + m, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((n, m), (ld, 1))
    x.copy_(torch.randn((n, m), device=DEV))
    small = x.contiguous()
    t = torch.tensor([1, 999, 500], device=DEV)
    d = torch.ones(n, device=DEV)
    a, b = sk.scores_logprobs(x, t, top=4, entropy=True), sk.scores_logprobs(small, t, top=4, entropy=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    want = sk.scores_logprobs_grad(small, t, b, d_logp=d)
    assert torch.equal(sk.scores_logprobs_grad(x, t, a, d_logp=d, grad=x), want)


def test_refusals():
    x = torch.zeros((4, 8), device=DEV)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    r = sk.scores_logprobs(x, t)
    d = torch.ones(4, device=DEV)
    for bad in (lambda: sk.scores_logprobs(x, t.int()), lambda: sk.scores_logprobs(x, t[:3]),
                lambda: sk.scores_logprobs(x, t.cpu()), lambda: sk.scores_logprobs(x, t, top=9),
                lambda: sk.scores_logprobs(x, t, eps=0.0), lambda: sk.scores_logprobs(x, t, eps=float("nan")),
                lambda: sk.scores_logprobs(x, t, out=r._replace(lse=d[:3])),
                lambda: sk.scores_logprobs_grad(x, None, r, d_logp=d),
                lambda: sk.scores_logprobs_grad(x, t, r, d_entropy=d),
                lambda: sk.scores_logprobs_grad(x, t, r, d_top=d[:, None]),
                lambda: sk.scores_logprobs_grad(x, t, r, d_logp=d.double()),
                lambda: sk.scores_logprobs_grad(x, t, r, d_logp=d, grad=x.half()),
                lambda: sk.scores_logprobs_grad(x, t, r, d_logp=d, grad=x.t()),
                lambda: sk.scores_logprobs_grad(x[:, :7], t, r, d_logp=d, grad=x[:, 1:])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sk.SinkhornError, match="WORKSPACE"):  # as every entry point that takes one
        sk.scores_logprobs(x, t, ws=torch.empty(8, dtype=torch.uint8, device=DEV))


def test_scores_in_another_order_are_copied():
    x, s = matrix(30, 20, "f32", 5)
    a, b = sk.scores_logprobs(x.t(), top=3, entropy=True), sk.scores_logprobs(x.t().contiguous(), top=3, entropy=True)
    assert torch.equal(a.lse, b.lse) and torch.equal(a.top_idx, b.top_idx) and torch.equal(a.entropy, b.entropy)
    row = x[0].expand(7, 20)
    assert torch.equal(sk.scores_logprobs(row).lse, sk.scores_logprobs(row.contiguous()).lse)
