"""route_sort, route_dispatch, route_combine and route_combine_grad against the float64 reference."""
import numpy as np
import pytest
import torch

import streaming_sinkhorn_solver_amd as sk
from oracle import routed as oro
from scores_cases import DEV, DTYPES, U, close, f64, half_step

pytestmark = pytest.mark.gpu


def choices(n, k, m, seed, dropped=0.15, alike=False):
    """k distinct experts of every token (alike: all tokens the same), some of them replaced by none of them."""
    r = np.random.default_rng(seed)
    if alike:
        idx = np.tile(np.arange(k) % m, (n, 1))
    else:
        idx = np.argsort(r.random((n, m)), axis=1)[:, :k] if m <= 64 else r.integers(0, m, (n, k))
    idx = np.asarray(idx, np.int32).reshape(n, k)
    if dropped:
        idx[r.random((n, k)) < dropped] = r.choice(np.array([-1, m, 2 ** 31 - 1, -2 ** 31]).astype(np.int32))
    return idx


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def window(rows, d, dtype, values=None, pad=0, offset=0, fill=float("nan")):
    """A (rows, d) window of a shifted buffer with longer rows: (window, the whole buffer)."""
    buf = torch.full((offset + rows * (d + pad) + 8,), fill, dtype=DTYPES[dtype], device=DEV)
    win = buf[offset:offset + rows * (d + pad)].view(rows, d + pad)[:, :d]
    if values is not None:
        win.copy_(gpu(values))
    return win, buf


def random_window(rows, d, dtype, seed, pad=0, offset=0):
    win, _ = window(rows, d, dtype, np.random.default_rng(seed).normal(size=(rows, d)), pad, offset)
    return win, f64(win)


def untouched(buf, win, fill):
    """Everything of the buffer but the window still holds the fill."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    torch.as_strided(mask, win.shape, win.stride(), win.storage_offset()).fill_(False)
    return bool((buf[mask] == fill).all())


# around one wave, one workgroup's share, one launch (4096 choices) and the launches beyond it
SORTS = [(0, 2, 5), (1, 1, 1), (1, 8, 64), (5, 3, 3), (64, 1, 2), (63, 4, 7), (512, 8, 256), (513, 8, 256), (1000, 6, 60),
         (4099, 7, 1024), (3000, 64, 100), (8192, 8, 33)]


@pytest.mark.parametrize("align,capacity", [(1, 0), (16, 0), (1, 3), (8, 100), (5, 17)])
@pytest.mark.parametrize("n,k,m", SORTS)
def test_sort(n, k, m, align, capacity):
    idx = choices(n, k, m, n + m)
    plan = sk.route_sort(gpu(idx), m, align=align, capacity=capacity)
    want = oro.sort(idx, m, align, capacity)
    assert plan.align == align
    for got, ref in zip(plan, want):
        assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("n,k,m", [(700, 4, 9), (3000, 8, 1000)])
def test_sort_one_expert_or_none(n, k, m):
    for idx in (choices(n, 1, m, 1, 0.0, True), np.full((n, k), -1, np.int32), np.full((n, k), m - 1, np.int32)):
        plan = sk.route_sort(gpu(idx), m, align=4)
        for got, ref in zip(plan, oro.sort(idx, m, 4)):
            assert np.array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("m", [300, 1000])
def test_sort_many_choices(m):
    """69 workgroups: more than add up one another's counts among 1000 experts, not among 300."""
    n, k = 140001, 8
    idx = choices(n, k, m, 4, 0.1)
    plan = sk.route_sort(gpu(idx), m, align=16)
    flat = idx.reshape(-1).astype(np.int64)
    flat = np.where((flat >= 0) & (flat < m), flat, m)
    order = np.argsort(flat, kind="stable")
    counts = np.bincount(flat, minlength=m + 1)[:m]
    offsets = np.concatenate([[0], np.cumsum((counts + 15) // 16 * 16)])
    assert np.array_equal(plan.counts.cpu().numpy(), counts) and np.array_equal(plan.offsets.cpu().numpy(), offsets)
    source = np.full(plan.source.numel(), -1)
    order = order[:counts.sum()]
    at = offsets[flat[order]] + np.arange(len(order)) - (np.cumsum(counts) - counts)[flat[order]]
    source[at] = order
    slot = np.full(n * k, -1)
    slot[order] = at
    assert np.array_equal(plan.source.cpu().numpy(), source) and np.array_equal(plan.slot.cpu().numpy().reshape(-1), slot)


def test_sort_buffers_and_strides():
    idx = choices(77, 6, 11, 8)
    wide = torch.full((77, 13), 5, dtype=torch.int32, device=DEV)
    wide[:, 1:13:2] = gpu(idx)
    first = sk.route_sort(gpu(idx), 11, align=2)
    rows = sk.route_sort_rows(77, 6, 11, 2)
    out = sk.RoutePlan(torch.full((77, 6), 9, dtype=torch.int32, device=DEV), torch.full((rows + 50,), 9, dtype=torch.int32, device=DEV),
                       torch.full((11,), 9, dtype=torch.int32, device=DEV), torch.full((12,), 9, dtype=torch.int32, device=DEV))
    ws = sk.route_sort_workspace(77, 6, 11, DEV)
    second = sk.route_sort(wide[:, 1:13:2], 11, align=2, ws=ws, out=out)
    assert second.slot.data_ptr() == out.slot.data_ptr() and second.align == 2
    for a, b in zip(first[:4], second[:4]):
        assert torch.equal(a, b[:a.shape[0]])
    assert (second.source[rows:] == -1).all()
    with pytest.raises(ValueError, match="out.source"):
        sk.route_sort(gpu(idx), 11, align=2, out=out._replace(source=out.source[:rows - 1]))
    with pytest.raises(ValueError, match="out.slot"):
        sk.route_sort(gpu(idx), 11, out=out._replace(slot=out.slot[:, :5]))
    with pytest.raises(ValueError, match="ws"):
        sk.route_sort(gpu(idx), 11, ws=torch.empty(256, device=DEV))


def product_tol(want, dtype):
    """One float32 product, one rounding to the type (below its normal range by half its smallest step)."""
    info = torch.finfo(DTYPES[dtype])
    return (U + half_step(dtype) * (1 + 1e-3)) * np.abs(want) + info.smallest_normal * info.eps / 2 + 2.0 ** -126


def sum_tol(want, size, terms, dtype):
    """`terms` float32 additions of products, each off by u of the largest partial sum (at most `size`)."""
    err = (terms + 1) * U * size
    return err + product_tol(np.abs(want) + err, dtype)


# one element to rows longer than a workgroup's 256 runs, whole runs of 16 bytes and not
WIDTHS = [1, 3, 7, 8, 9, 31, 64, 100, 128, 129, 255, 512, 1027, 2048, 2056, 4100]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", WIDTHS)
def test_rows(d, dtype):
    n, k, m, align = 37, 3, 5, 4
    idx = choices(n, k, m, d)
    plan = sk.route_sort(gpu(idx), m, align=align)
    slot, _, _, offsets = oro.sort(idx, m, align)
    rows = plan.source.numel()
    r = np.random.default_rng(d)
    w = r.normal(size=(n, k)).astype(np.float32)
    pad, offset = d % 3, d % 2
    x, xs = random_window(n, d, dtype, 1, pad, offset)
    g, gs = random_window(rows, d, dtype, 2, 2 - pad, 1 - offset)
    for weights in (None, w):
        gw = None if weights is None else gpu(weights)
        out, buf = window(rows, d, dtype, None, pad, 1, 7.0)
        assert sk.route_dispatch(x, plan, gw, out=out) is out
        want = oro.dispatch(xs, slot, offsets, weights, np.full((rows, d), 7.0))
        close(out, want, 0.0 if weights is None else product_tol(want, dtype), "dispatch")
        assert untouched(buf, out, 7.0) and (out[offsets[-1]:] == 7.0).all()
        for add, adds in ((None, None), (x, xs)):
            y, buf = window(n, d, dtype, None, 1, offset, 7.0)
            assert sk.route_combine(g, plan, gw, add=add, out=y) is y
            want = oro.combine(gs, slot, weights, adds)
            size = oro.combine(np.abs(gs), slot, None if weights is None else np.abs(weights), None if adds is None else np.abs(adds))
            close(y, want, sum_tol(want, size, k + 1, dtype), "combine")
            assert untouched(buf, y, 7.0)
        d_rows, buf = window(rows, d, dtype, None, 1, offset, 7.0)
        _, d_w = sk.route_combine_grad(g, plan, gw, x, d_rows=d_rows)
        want, want_w = oro.combine_grad(gs, slot, offsets, weights, xs, np.full((rows, d), 7.0))
        close(d_rows, want, 0.0 if weights is None else product_tol(want, dtype), "d_rows")
        assert untouched(buf, d_rows, 7.0)
        _, size = oro.combine_grad(np.abs(gs), slot, offsets, weights, np.abs(xs), np.zeros((rows, d)))
        # 8 to 256 lanes, as many as the row's runs where they are fewer (128 count as 64): a lane adds d / 16 elements at most but for
        # rows of fewer than 20, then the lanes are added
        close(d_w, want_w, (d / 16 + 20) * U * size, "d_weights")


@pytest.mark.parametrize("n,d", [(1, 8195), (3, 16384), (129, 4100), (512, 4096), (513, 4096), (600, 4099)])
def test_long_rows(n, d):
    """Rows that a workgroup does not take at once: shared out among several (up to 512 tokens), or taken in turns."""
    k, m = 2, 3
    idx = choices(n, k, m, n)
    plan = sk.route_sort(gpu(idx), m, align=2)
    slot, _, _, offsets = oro.sort(idx, m, 2)
    rows = plan.source.numel()
    w = np.random.default_rng(n).normal(size=(n, k)).astype(np.float32)
    x, xs = random_window(n, d, "bf16", 1, 1, 1)
    g, gs = random_window(rows, d, "bf16", 2)
    out = sk.route_dispatch(x, plan, gpu(w), out=torch.full((rows, d), 7.0, dtype=torch.bfloat16, device=DEV))
    want = oro.dispatch(xs, slot, offsets, w, np.full((rows, d), 7.0))
    close(out, want, product_tol(want, "bf16"), "dispatch")
    want = oro.combine(gs, slot, w, xs)
    close(sk.route_combine(g, plan, gpu(w), add=x), want, sum_tol(want, oro.combine(np.abs(gs), slot, np.abs(w), np.abs(xs)), k + 1, "bf16"), "combine")
    over = x.clone(memory_format=torch.contiguous_format)
    sk.route_combine(g, plan, gpu(w), add=over, out=over)
    assert torch.equal(over, sk.route_combine(g, plan, gpu(w), add=x))


@pytest.mark.parametrize("k", [1, 2, 7, 8, 9, 16, 17, 64])
@pytest.mark.parametrize("d", [8, 200, 2048])
def test_many_choices_of_a_token(k, d):
    """Eight of a token's rows are in flight at a time."""
    n, m = 9, 64
    idx = choices(n, k, m, k, 0.3)
    plan = sk.route_sort(gpu(idx), m)
    slot, _, _, offsets = oro.sort(idx, m)
    rows = plan.source.numel()
    w = np.random.default_rng(k).normal(size=(n, k)).astype(np.float32)
    w[slot < 0] = np.nan  # a dropped choice's weight is not looked at
    g, gs = random_window(rows, d, "bf16", 3)
    x, xs = random_window(n, d, "bf16", 4)
    y = sk.route_combine(g, plan, gpu(w))
    want = oro.combine(gs, slot, w)
    close(y, want, sum_tol(want, oro.combine(np.abs(gs), slot, np.abs(w)), k + 1, "bf16"), "combine")
    rest = torch.full((rows, d), 3.0, dtype=torch.bfloat16, device=DEV)
    d_rows, d_w = sk.route_combine_grad(g, plan, gpu(w), x, d_rows=rest)
    want, want_w = oro.combine_grad(gs, slot, offsets, w, xs, np.full((rows, d), 3.0))
    close(d_rows, want, product_tol(want, "bf16"), "d_rows")
    _, size = oro.combine_grad(np.abs(gs), slot, offsets, w, np.abs(xs), np.zeros((rows, d)))
    close(d_w, want_w, (d / 16 + 20) * U * size, "d_weights")
    rest = torch.full((rows, d), 3.0, dtype=torch.bfloat16, device=DEV)
    want = oro.dispatch(xs, slot, offsets, w, np.full((rows, d), 3.0))
    close(sk.route_dispatch(x, plan, gpu(w), out=rest), want, product_tol(want, "bf16"), "dispatch")


@pytest.mark.parametrize("d", [5, 136, 1500])
def test_in_place_and_halves(d):
    n, k, m, align = 21, 4, 6, 8
    idx = choices(n, k, m, d)
    plan = sk.route_sort(gpu(idx), m, align=align)
    rows = plan.source.numel()
    g, _ = random_window(rows, d, "f16", 1)
    x, _ = random_window(n, d, "f16", 2)
    w = torch.randn(n, k, device=DEV)
    a, b = sk.route_combine_grad(g, plan, w, x, d_rows=g.clone())
    only, none = sk.route_combine_grad(g, plan, w, x, weights_grad=False, d_rows=g.clone())
    assert none is None and torch.equal(only, a)
    none, only = sk.route_combine_grad(g, plan, w, x, rows_grad=False)
    assert none is None and torch.equal(only, b)
    # the rows' gradient over the rows, the sum over what is added
    over = g.clone()
    got, got_w = sk.route_combine_grad(over, plan, w, x, d_rows=over)
    assert got is over and torch.equal(over, a) and torch.equal(got_w, b)
    y = sk.route_combine(g, plan, w, add=x)
    over = x.clone()
    assert sk.route_combine(g, plan, w, add=over, out=over) is over and torch.equal(over, y)
    # a weighted dispatch's gradients
    rows_x = sk.route_dispatch(x, plan, w)
    end = int(plan.offsets[-1])
    _, d_w = sk.route_combine_grad(g, plan, None, x, rows_grad=False)
    assert torch.equal(d_w, b) and torch.equal(rows_x[:end], a[:end])


def test_nothing_kept_and_no_tokens():
    plan = sk.route_sort(torch.full((6, 2), -1, dtype=torch.int32, device=DEV), 4, align=2)
    x = torch.randn(6, 40, device=DEV)
    rest = torch.full((plan.source.numel(), 40), 2.0, device=DEV)
    assert (sk.route_dispatch(x, plan, out=rest) == 2.0).all()
    assert (sk.route_combine(rest, plan) == 0.0).all() and torch.equal(sk.route_combine(rest, plan, add=x), x)
    d_rows, d_w = sk.route_combine_grad(rest, plan, None, x, d_rows=rest.clone())
    assert (d_rows == 2.0).all() and (d_w == 0.0).all()
    plan = sk.route_sort(torch.empty((0, 2), dtype=torch.int32, device=DEV), 4)
    assert plan.source.numel() == 0 and (plan.offsets == 0).all() and (plan.counts == 0).all()
    none = x[:0]
    assert sk.route_dispatch(none, plan).shape == (0, 40) and sk.route_combine(none, plan).shape == (0, 40)
    d_rows, d_w = sk.route_combine_grad(none, plan, None, none)
    assert d_rows.shape == (0, 40) and d_w.shape == (0, 2)


def test_special_values():
    """Infinities and NaN go where they belong; slots outside the rows are dropped."""
    plan = sk.route_sort(torch.tensor([[0, 1], [1, 2], [2, 0]], dtype=torch.int32, device=DEV), 3)
    x = torch.tensor([[1.0, float("inf")], [float("nan"), 2.0], [3.0, -4.0]], device=DEV)
    rows = sk.route_dispatch(x, plan)
    assert torch.equal(torch.isnan(rows).nonzero(), torch.tensor([[3, 0], [4, 0]], device=DEV))  # the rows are tokens 0 2, 0 1, 1 2
    w = torch.tensor([[0.0, 1.0], [1.0, 1.0], [0.5, 0.5]], device=DEV)
    y = sk.route_combine(rows, plan, w)
    assert torch.isnan(y[0, 1]) and torch.isnan(y[1, 0]) and y[1, 1] == 4.0 and torch.equal(y[2], x[2])  # 0 * inf is NaN
    wrong = plan._replace(slot=torch.tensor([[0, 6], [-5, 2 ** 31 - 1], [1, 5]], dtype=torch.int32, device=DEV))
    clean = torch.arange(12, dtype=torch.float32, device=DEV).view(6, 2)
    assert torch.equal(sk.route_combine(clean, wrong), torch.stack([clean[0], 0 * clean[0], clean[1] + clean[5]]))
    got = sk.route_dispatch(clean[:3], wrong, out=torch.zeros(6, 2, device=DEV))
    assert torch.equal(got[[0, 1, 5]], clean[[0, 2, 2]]) and (got[2:5] == 0).all()


def test_offsets_beyond_32_bits():
    """2.2e9 elements: addresses past 2^31 elements and 2^32 bytes."""
    n, d = 270001, 8192
    x = torch.empty((n, d), dtype=torch.bfloat16, device=DEV)
    x.copy_(torch.arange(n, device=DEV)[:, None] % 251)
    plan = sk.route_sort((torch.arange(n, device=DEV, dtype=torch.int32) * 7 % 5)[:, None].contiguous(), 5)
    rows = sk.route_dispatch(x, plan)
    back = sk.route_combine(rows, plan)
    assert torch.equal(back, x)
    last = plan.source[-3:].long()
    assert torch.equal(rows[-3:, ::1000], x[last][:, ::1000])
    del back
    over, d_w = sk.route_combine_grad(rows, plan, None, x, d_rows=rows)
    assert torch.equal(over[-3:, ::1000], x[last][:, ::1000])
    i = n - 2
    want = d * float((i % 251) ** 2)
    assert abs(float(d_w[i, 0]) - want) <= (d / 16 + 20) * U * want


def test_adjoint_and_differences():
    """<dispatch(x), g> = <x, combine(g)>, and combine's gradients by differences of the library's own sums."""
    n, k, m, d = 50, 3, 7, 96
    idx = choices(n, k, m, 2)
    plan = sk.route_sort(gpu(idx), m)
    rows, kept = plan.source.numel(), int(plan.offsets[-1])
    r = torch.Generator(device=DEV).manual_seed(5)
    x, g = (torch.randn(s, d, device=DEV, generator=r) for s in (n, rows))
    g[kept:] = 0
    w, dy = torch.randn(n, k, device=DEV, generator=r), torch.randn(n, d, device=DEV, generator=r)
    left = (sk.route_dispatch(x, plan, out=torch.zeros(rows, d, device=DEV)).double() * g.double()).sum()
    right = (x.double() * sk.route_combine(g, plan).double()).sum()
    # combine rounds each sum of at most 3 terms three times
    assert abs(float(left - right)) <= 3 * U * float((x.abs().double() * sk.route_combine(g.abs(), plan).double()).sum())
    d_rows, d_w = sk.route_combine_grad(g, plan, w, dy)

    def loss(rows_, w_):
        return float((sk.route_combine(rows_, plan, w_).double() * dy.double()).sum())

    # the sum is linear in w and in the rows, so a difference of step 1 (exact in float32 up to rounding) is the derivative
    size = float((sk.route_combine(g.abs(), plan, w.abs() + 1.0).double() * dy.abs().double()).sum())
    for i, c in ((0, 0), (13, 2), (49, 1)):
        e = torch.zeros_like(w)
        e[i, c] = 0.5
        diff = loss(g, w + e) - loss(g, w - e)
        assert abs(diff - float(d_w[i, c])) <= 16 * U * size
    for s in (0, kept // 2, kept - 1):
        e = torch.zeros_like(g)
        e[s, 5] = 0.5
        diff = loss(g + e, w) - loss(g - e, w)
        assert abs(diff - float(d_rows[s, 5])) <= 16 * U * (size + float(w.abs().max() * dy.abs().max()))


def test_refusals():
    idx = gpu(choices(10, 2, 4, 1, 0.0))
    plan = sk.route_sort(idx, 4)
    x, rows, w = torch.randn(10, 16, device=DEV), torch.randn(20, 16, device=DEV), torch.ones(10, 2, device=DEV)
    for call in (lambda: sk.route_dispatch(x[:9], plan), lambda: sk.route_dispatch(x, plan, w[:9]), lambda: sk.route_dispatch(x, plan, w.half()),
                 lambda: sk.route_dispatch(x, plan, out=rows.half()), lambda: sk.route_dispatch(x, plan, out=rows[:19]),
                 lambda: sk.route_combine(rows[:19], plan), lambda: sk.route_combine(rows, plan, add=x.half()),
                 lambda: sk.route_combine(rows, plan, add=x[:, :8]), lambda: sk.route_combine(rows, plan, out=x.t()),
                 lambda: sk.route_combine_grad(rows, plan, w, x.bfloat16()), lambda: sk.route_combine_grad(rows, plan, w, x[:5]),
                 lambda: sk.route_combine_grad(rows, plan, w, x, rows_grad=False, weights_grad=False),
                 lambda: sk.route_combine_grad(rows, plan, w, x, d_weights=w.double()),
                 lambda: sk.route_dispatch(x, plan._replace(slot=plan.slot.long())),
                 lambda: sk.route_dispatch(x, plan._replace(slot=plan.slot.cpu())),
                 lambda: sk.route_dispatch(x, plan._replace(align=2, offsets=plan.offsets[:3])),
                 lambda: sk.route_combine(rows, plan, out=rows[:10]), lambda: sk.route_dispatch(rows[:10], plan, out=rows)):
        with pytest.raises(ValueError):
            call()


def test_streams_and_graphs():
    """Another stream, and a graph of the whole way replayed with eager work between."""
    n, k, m, d = 300, 4, 16, 520
    x = torch.randn(n, d, device=DEV).bfloat16()
    w = torch.rand(n, k, device=DEV)
    idx = gpu(choices(n, k, m, 3))
    dy = torch.randn(n, d, device=DEV).bfloat16()
    rows = sk.route_sort_rows(n, k, m, 8)

    def way(plan, bufs):
        plan = sk.route_sort(idx, m, align=8, ws=bufs["ws"], out=plan)
        sk.route_dispatch(x, plan, out=bufs["rows"])
        sk.route_combine(bufs["rows"], plan, w, out=bufs["y"])
        sk.route_combine_grad(bufs["rows"], plan, w, dy, d_rows=bufs["d_rows"], d_weights=bufs["d_w"])
        sk.route_combine(bufs["d_rows"], plan, out=bufs["d_x"])
        return plan

    def buffers():
        return {"ws": sk.route_sort_workspace(n, k, m, DEV), "rows": torch.zeros(rows, d, device=DEV).bfloat16(),
                "y": torch.empty_like(x), "d_rows": torch.zeros(rows, d, device=DEV).bfloat16(), "d_w": torch.empty_like(w),
                "d_x": torch.empty_like(x)}

    def outputs(plan, bufs):
        return [t.clone() for t in plan[:4]] + [bufs[c].clone() for c in ("rows", "y", "d_rows", "d_w", "d_x")]

    def same(a, b):
        return all(torch.equal(p, q) for p, q in zip(a, b))

    eager = buffers()
    want = outputs(way(None, eager), eager)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        bufs = buffers()
        got = outputs(way(None, bufs), bufs)
    other.synchronize()
    assert same(want, got)
    bufs = buffers()
    plan = way(None, bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        way(plan, bufs)
    for step in range(4):
        idx.copy_(gpu(choices(n, k, m, 10 + step)))
        x.copy_(torch.randn(n, d, device=DEV))
        for c in ("rows", "d_rows"):
            bufs[c].zero_()
            eager[c].zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = outputs(plan, bufs)
        assert same(outputs(way(None, eager), eager), got), step
