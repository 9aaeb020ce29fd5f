"""The routed rows' sort at every number of pairs of a thread, and their buffers: windows of one buffer, outputs that
change apart from one another."""
import numpy as np
import pytest
import torch

import streaming_sinkhorn_solver_amd as sk
from scores_cases import DEV, DTYPES

pytestmark = pytest.mark.gpu


# the pairs of a thread are 1, 2, 4, 8 or 16, by the pairs that one workgroup (up to 4096) or the most of them would leave
@pytest.mark.parametrize("align,capacity", [(1, 0), (16, 0), (4, 90)])
@pytest.mark.parametrize("n,k,m", [(2047, 1, 1000), (4095, 1, 70), (99, 41, 1000), (9091, 11, 1000), (28571, 7, 1000), (400001, 1, 1000), (524287, 1, 1000),
                                   (157143, 7, 1000), (74899, 7, 60), (131071, 8, 60), (350003, 6, 60), (65535, 9, 512)])
def test_sort_pairs_of_a_thread(n, k, m, align, capacity):
    """Several workgroups, the last with fewer pairs, for every number of pairs of a thread."""
    r = np.random.default_rng(n)
    idx = r.integers(-m // 8, m + m // 8, (n, k)).astype(np.int32)  # (a fifth is none of the experts)
    plan = sk.route_sort(torch.from_numpy(idx).to(DEV), m, align=align, capacity=capacity)
    flat = idx.reshape(-1).astype(np.int64)
    flat = np.where((flat >= 0) & (flat < m), flat, m)
    order = np.argsort(flat, kind="stable")
    every = np.bincount(flat, minlength=m + 1)
    rank = np.arange(n * k) - (np.cumsum(every) - every)[flat[order]]
    kept = (flat[order] < m) & ((rank < capacity) if capacity else True)
    counts = np.minimum(every[:m], capacity) if capacity else every[:m]
    offsets = np.concatenate([[0], np.cumsum(-(-counts // align) * align)])
    slot, source = np.full(n * k, -1), np.full(plan.source.numel(), -1)
    slot[order[kept]] = offsets[flat[order[kept]]] + rank[kept]
    source[slot[order[kept]]] = order[kept]
    for got, want in zip(plan, (slot.reshape(n, k), source, counts, offsets)):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,gap", [(64, 0), (101, 3), (2048, 0), (2050, 6)])
def test_windows_of_one_buffer(d, gap, dtype):
    """Inputs and outputs side by side in the rows of one buffer have no element in common."""
    n, k, m = 24, 1, 5
    r = torch.Generator(device=DEV).manual_seed(d)
    idx = torch.randint(0, m, (n, k), device=DEV, dtype=torch.int32, generator=r)
    plan = sk.route_sort(idx, m)
    w = torch.rand(n, k, device=DEV, generator=r)

    def pair(seed):
        """Two (n, d) windows of a wide buffer: one with values, the other of sevens; and a check of all the rest."""
        wide = torch.full((n, 2 * d + gap), 7.0, dtype=DTYPES[dtype], device=DEV)
        a, b = wide[:, :d], wide[:, d + gap:]
        a.copy_(torch.randn(n, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)))
        return a, b, lambda was: torch.equal(a, was) and bool((wide[:, d:d + gap] == 7.0).all())

    for swap in (False, True):
        for call in (lambda x, out: sk.route_dispatch(x, plan, w, out=out), lambda x, out: sk.route_combine(x, plan, w, out=out),
                     lambda x, out: sk.route_combine(x.contiguous(), plan, w, add=x, out=out),
                     lambda x, out: sk.route_combine_grad(x.contiguous(), plan, w, x, d_rows=out)[0],
                     lambda x, out: sk.route_combine_grad(x, plan, w, x.contiguous(), d_rows=out)[0]):
            a, b, same = pair(3)
            if swap:  # the window with values behind the other
                values = a.clone()
                b.copy_(values)
                a.fill_(7.0)
                got, want = call(b, a), call(values, torch.empty_like(values))
                assert torch.equal(got, want) and torch.equal(b, values)
            else:
                was = a.clone()
                got, want = call(a, b), call(was, torch.empty_like(was))
                assert torch.equal(got, want) and same(was)


@pytest.mark.parametrize("d", [5, 40, 200, 700, 5000])
@pytest.mark.parametrize("n,k", [(1, 2), (333, 19), (4000, 3)])
def test_outputs_in_place_of_small_inputs(n, k, d):
    """The slots over the choices, the weights' gradient over the weights."""
    m, n = 30, min(n, 400) if d > 700 else n
    r = torch.Generator(device=DEV).manual_seed(n + d)
    idx = torch.randint(-2, m + 2, (n, k), device=DEV, dtype=torch.int32, generator=r)
    plan = sk.route_sort(idx, m, align=4)
    over = idx.clone()
    got = sk.route_sort(over, m, align=4, out=plan._replace(slot=over, source=plan.source.clone()))
    assert got.slot.data_ptr() == over.data_ptr() and all(torch.equal(a, b) for a, b in zip(got[:4], plan[:4]))
    x = torch.randn(n, d, device=DEV, generator=r).bfloat16()
    rows = torch.randn(plan.source.numel(), d, device=DEV, generator=r).bfloat16()
    w = torch.randn(n, k, device=DEV, generator=r)
    want, want_w = sk.route_combine_grad(rows, plan, w, x, d_rows=rows.clone())
    out = rows.clone()
    got_w = sk.route_combine_grad(rows, plan, w, x, d_rows=out, d_weights=w)[1]
    assert got_w is w and torch.equal(w, want_w) and torch.equal(out, want)
    with pytest.raises(ValueError, match="SK_ERR_OVERLAP"):
        sk.route_combine_grad(rows, plan, w, x, d_weights=rows.view(-1)[:2 * n * k].view(torch.float32).view(n, k))


def test_outputs_change_apart():
    """An output that is changed in place is no change of another: what autograd has saved of a plan stays valid."""
    plan = sk.route_sort(torch.randint(0, 4, (10, 2), dtype=torch.int32, device=DEV), 4)
    s = torch.randn(3, 40, device=DEV)
    v = sk.scores_verify(s, torch.tensor([1, 2, -1], device=DEV), torch.tensor([0, 3], device=DEV), torch.rand(3, device=DEV),
                         torch.rand(1, device=DEV))
    for outs in (plan[:4], v):
        for t in outs:
            before, values = [o._version for o in outs], [o.clone() for o in outs]
            t.add_(1)
            for o, b, x in zip(outs, before, values):
                assert (o._version != b) == (o is t) and torch.equal(o, x + 1 if o is t else x)

    class Way(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, plan):
            ctx.save_for_backward(plan.slot, plan.source)
            return sk.route_dispatch(x, plan)

        @staticmethod
        def backward(ctx, d_rows):
            slot, source = ctx.saved_tensors
            return sk.route_combine(d_rows, sk.RoutePlan(slot, source, None, None)), None

    x = torch.randn(10, 8, device=DEV, requires_grad=True)
    plan = sk.route_sort(torch.randint(0, 4, (10, 2), dtype=torch.int32, device=DEV), 4)
    y = Way.apply(x, plan)
    plan.counts.add_(plan.counts.clone())  # (a sum over training steps)
    y.backward(torch.ones_like(y))
    assert (x.grad == 2.0).all()
