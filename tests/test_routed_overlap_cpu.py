"""Outputs of the token-row entry points and of sk_scores_verify that overlap an input are refused before anything is
enqueued: checked without a GPU, at addresses that are never touched."""
import ctypes

import pytest

import streaming_sinkhorn_solver_amd as sk
from test_routed_boundary_cpu import OVERLAP, lib  # noqa: F401  (the fixture)

MB = 1 << 20


def addr(place, off=0):
    """An address in one of several places far from one another."""
    return ctypes.c_void_p(MB * (1 + 16 * place) + off)


SORT = dict(idx=0, slot=1, source=2, counts=3, offsets=4)
SORT_BYTES = dict(idx=80, slot=80, source=80, counts=48, offsets=52)


@pytest.mark.parametrize("out", ["slot", "source", "counts", "offsets"])
def test_sort(lib, out):  # noqa: F811
    def call(**at):
        a = {name: addr(place) for name, place in SORT.items()}
        a.update(at)
        return lib.sk_route_sort(a["idx"], 10, 2, 12, 1, 0, a["slot"], a["source"], 20, a["counts"], a["offsets"], addr(9), 256, None)

    for off in (4, SORT_BYTES["idx"] - 4) + (() if out == "slot" else (0,)):  # (slot may be idx)
        assert call(**{out: addr(0, off)}) == OVERLAP, off
        assert call(idx=addr(SORT[out], SORT_BYTES[out] - 4)) == OVERLAP


INPUTS = dict(slot=80, weights=80, counts=16, offsets=20)


def plan_at(name, where):
    """The plan's addresses with one of them elsewhere; counts and offsets are given together."""
    a = {k: addr(10 + i) for i, k in enumerate(INPUTS)}
    a[name] = where
    return a["slot"], a["weights"], a["counts"], a["offsets"]


@pytest.mark.parametrize("name", list(INPUTS))
def test_rows(lib, name):  # noqa: F811
    for off in (0, 4, 20 * 48 - 4, 4 - INPUTS[name]):
        slot, weights, counts, offsets = plan_at(name, addr(1, off))
        assert lib.sk_route_dispatch(addr(0), 0, 10, 12, 12, slot, 2, weights, counts, offsets, 4, addr(1), 20, 12, None) == OVERLAP
        assert lib.sk_route_combine_grad(addr(0), 0, 20, 12, 12, slot, 10, 2, weights, counts, offsets, 4, addr(2), 12, addr(1), 12,
                                         None, None) == OVERLAP
        if name in ("slot", "weights") and off < 10 * 48:
            assert lib.sk_route_combine(addr(0), 0, 20, 12, 12, slot, 10, 2, weights, None, 12, addr(1), 12, None) == OVERLAP


def test_gradient_of_the_weights(lib):  # noqa: F811
    def call(dw, **at):
        a = {k: addr(10 + i) for i, k in enumerate(INPUTS)}
        a.update(at)
        return lib.sk_route_combine_grad(addr(0), 0, 20, 12, 12, a["slot"], 10, 2, a["weights"], a["counts"], a["offsets"], 4, addr(2), 12,
                                         None, 12, dw, None)

    assert call(addr(0)) == OVERLAP and call(addr(0, 20 * 48 - 4)) == OVERLAP  # the rows
    assert call(addr(2, 100)) == OVERLAP and call(addr(2, -76)) == OVERLAP     # d_y
    for name in INPUTS:
        assert call(addr(5), **{name: addr(5, 4)}) == OVERLAP and call(addr(5), **{name: addr(5, -4)}) == OVERLAP


VERIFY = dict(s=0, tok=2, starts=3, ua=4, us=5)
VERIFY_BYTES = dict(s=(9 * 14 + 12) * 4, tok=80, starts=32, ua=40, us=12)
VERIFY_OUT = dict(acc=12, nxt=24, out=80, ratio=40, logp=40)


@pytest.mark.parametrize("out", list(VERIFY_OUT))
@pytest.mark.parametrize("name", list(VERIFY))
def test_verify(lib, name, out):  # noqa: F811
    """10 rows of 12 scores (row stride 14), 3 requests."""
    a = {k: addr(place) for k, place in VERIFY.items()}
    o = {k: addr(10 + i) for i, k in enumerate(VERIFY_OUT)}
    nb = lib.sk_scores_verify_workspace_bytes(0, 10, 12, 3)
    for off in (0, VERIFY_BYTES[name] - 8, 8 - VERIFY_OUT[out]):
        if (name, out, off) == ("tok", "out", 0):  # (these may be one)
            continue
        o[out] = addr(VERIFY[name], off)
        assert lib.sk_scores_verify(a["s"], 0, 10, 12, 14, 0.5, None, 12, 1.0, a["tok"], a["starts"], 3, a["ua"], a["us"], o["acc"], o["nxt"],
                                    o["out"], o["ratio"], o["logp"], addr(30), nb, None) == OVERLAP, off
