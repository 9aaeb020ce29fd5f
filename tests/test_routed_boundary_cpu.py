"""Refusals of the token-row entry points and of sk_scores_verify, checked without a GPU: every bad argument returns its
status (or raises) before anything is enqueued."""
import ctypes
import os

import pytest
import torch

import streaming_sinkhorn_solver_amd as sk
from oracle import routed as oro
from streaming_sinkhorn_solver_amd import build as skbuild

P = ctypes.c_void_p(0x100000)  # never dereferenced: validation returns first
F32, BF16, F16 = 0, 1, 2
OK, NULL, SHAPE, EPS, WS, DTYPE, ROUTE, OVERLAP = 0, 1, 2, 4, 11, 18, 19, 20
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sk.LIB_PATH):
        skbuild.build()
    return sk.load_library()


def addr(off):
    return ctypes.c_void_p(0x100000 + off)


def test_sort_rows(lib):
    for args in ((0, 1, 1, 1, 0), (1, 8, 64, 1, 0), (10, 3, 5, 16, 0), (10, 3, 5, 16, 7), (10, 3, 100, 4, 1), (1000, 4, 7, 1, 13)):
        assert lib.sk_route_sort_rows(*args) == oro.sort_rows(*args)
    for args in ((-1, 1, 1, 1, 0), (BIG, 1, 1, 1, 0), (1, 0, 1, 1, 0), (1, 65, 100, 1, 0), (1, 1, 0, 1, 0), (1, 1, 1025, 1, 0),
                 (1, 1, 1, 0, 0), (1, 1, 1, 1, -1), (1 << 30, 2, 8, 1, 0), (1 << 20, 1, 1024, 1 << 30, 0)):
        assert lib.sk_route_sort_rows(*args) == -1, args
    assert lib.sk_route_sort_workspace_bytes(1, 1, 1) == 256
    for args in ((-1, 1, 1), (1, 0, 1), (1, 1, 1025), (1 << 30, 2, 8)):
        assert lib.sk_route_sort_workspace_bytes(*args) == 0
    assert lib.sk_route_sort_workspace_bytes(1 << 20, 8, 256) < (1 << 20) * 8  # far below the choices


def test_sort_refusals(lib):
    def call(idx=P, n=10, k=2, m=12, align=1, cap=0, slot=P, source=P, rows=20, counts=P, offsets=P, ws=P, nb=None):
        need = lib.sk_route_sort_workspace_bytes(n, k, m)
        return lib.sk_route_sort(idx, n, k, m, align, cap, slot, source, rows, counts, offsets, ws, need if nb is None else nb,
                                 None)

    assert call(idx=None) == NULL and call(slot=None) == NULL and call(source=None) == NULL
    assert call(counts=None) == NULL and call(offsets=None) == NULL
    assert call(n=-1) == SHAPE and call(n=BIG) == SHAPE and call(m=0) == SHAPE and call(m=1025) == SHAPE
    assert call(rows=19) == SHAPE and call(rows=BIG) == SHAPE and call(align=2, rows=29) == SHAPE
    assert call(n=1 << 30, rows=1 << 31) == SHAPE
    assert call(k=0) == ROUTE and call(k=65) == ROUTE and call(align=0) == ROUTE and call(cap=-1) == ROUTE
    assert call(ws=None) == WS and call(ws=addr(64)) == WS and call(nb=255) == WS
    assert call(n=100000, rows=200000, nb=256) == WS


def test_dispatch_refusals(lib):
    def call(x=P, dt=F32, n=10, d=12, ld=12, slot=P, k=2, counts=None, offsets=None, m=4, out=addr(1 << 20), rows=20, ldo=12):
        return lib.sk_route_dispatch(x, dt, n, d, ld, slot, k, None, counts, offsets, m, out, rows, ldo, None)

    assert call(x=None) == NULL and call(slot=None) == NULL and call(out=None) == NULL
    assert call(counts=P) == NULL and call(offsets=P) == NULL and call(counts=P, offsets=P, m=0) == SHAPE
    assert call(counts=P, offsets=P, m=1025) == SHAPE
    assert call(n=-1) == SHAPE and call(d=0) == SHAPE and call(ld=11) == SHAPE and call(ldo=11) == SHAPE and call(rows=-1) == SHAPE
    assert call(rows=BIG) == SHAPE and call(n=BIG) == SHAPE and call(ld=1 << 60) == SHAPE
    assert call(dt=5) == DTYPE and call(x=addr(2)) == DTYPE and call(out=addr((1 << 20) + 1), dt=BF16) == DTYPE
    assert call(k=0) == ROUTE and call(k=65) == ROUTE
    assert call(out=P) == OVERLAP and call(out=addr(10 * 12 * 4 - 4)) == OVERLAP and call(x=addr((1 << 20) + 20 * 48 - 4)) == OVERLAP
    assert call(n=0, x=None, slot=None) == OK and call(rows=0, out=None) == OK


def test_combine_refusals(lib):
    def call(rows=P, dt=F32, nr=20, d=12, ldr=12, slot=P, n=10, k=2, add=None, lda=12, y=addr(1 << 20), ldy=12):
        return lib.sk_route_combine(rows, dt, nr, d, ldr, slot, n, k, None, add, lda, y, ldy, None)

    assert call(rows=None) == NULL and call(slot=None) == NULL and call(y=None) == NULL
    assert call(n=-1) == SHAPE and call(d=0) == SHAPE and call(ldr=11) == SHAPE and call(ldy=11) == SHAPE
    assert call(add=P, lda=3) == SHAPE and call(nr=-1) == SHAPE
    assert call(dt=-1) == DTYPE and call(rows=addr(2)) == DTYPE and call(add=addr(2)) == DTYPE and call(y=addr((1 << 20) + 2)) == DTYPE
    assert call(k=0) == ROUTE and call(k=65) == ROUTE
    assert call(y=P) == OVERLAP and call(y=addr(20 * 48 - 4)) == OVERLAP
    assert call(add=addr((1 << 20) + 4)) == OVERLAP and call(add=addr(1 << 20), lda=13) == OVERLAP
    assert call(n=0, slot=None, y=None) == OK

    def grad(rows=P, dt=F32, nr=20, d=12, ldr=12, slot=P, n=10, k=2, counts=None, offsets=None, m=4, dy=addr(1 << 21), ldy=12,
             dr=addr(1 << 20), ldd=12, dw=P):
        return lib.sk_route_combine_grad(rows, dt, nr, d, ldr, slot, n, k, None, counts, offsets, m, dy, ldy, dr, ldd, dw, None)

    assert grad(rows=None) == NULL and grad(slot=None) == NULL and grad(dy=None) == NULL and grad(dr=None, dw=None) == NULL
    assert grad(counts=P) == NULL and grad(counts=P, offsets=P, m=0) == SHAPE
    assert grad(n=-1) == SHAPE and grad(d=0) == SHAPE and grad(ldr=11) == SHAPE and grad(ldy=11) == SHAPE and grad(ldd=11) == SHAPE
    assert grad(dt=3) == DTYPE and grad(dr=addr((1 << 20) + 2)) == DTYPE and grad(dy=addr(2)) == DTYPE
    assert grad(k=0) == ROUTE and grad(k=65) == ROUTE
    assert grad(dr=addr(4)) == OVERLAP and grad(dr=P, ldd=13) == OVERLAP and grad(dr=addr(1 << 21)) == OVERLAP
    assert grad(n=0, rows=None, slot=None, dy=None, nr=0) == OK


def test_verify_refusals(lib):
    def wb(dt=F32, n=10, m=12, b=3):
        return lib.sk_scores_verify_workspace_bytes(dt, n, m, b)

    def call(s=P, dt=F32, n=10, m=12, ld=12, eps=1.0, q=None, ldq=12, eq=1.0, tok=P, starts=P, b=3, ua=P, us=P, acc=P, nxt=P,
             out=P, ratio=P, logp=P, ws=P, nb=None):
        return lib.sk_scores_verify(s, dt, n, m, ld, eps, q, ldq, eq, tok, starts, b, ua, us, acc, nxt, out, ratio, logp, ws,
                                    wb() if nb is None else nb, None)

    for name in ("s", "tok", "starts", "ua", "us", "acc", "nxt", "out", "ratio", "logp"):
        assert call(**{name: None}) == NULL, name
    assert call(n=-1) == SHAPE and call(m=0) == SHAPE and call(ld=11) == SHAPE and call(b=-1) == SHAPE and call(b=BIG) == SHAPE
    assert call(m=(1 << 30) + 1, ld=1 << 31, nb=1 << 50) == SHAPE and call(q=P, ldq=11) == SHAPE
    assert call(dt=3) == DTYPE and call(s=addr(2)) == DTYPE and call(q=addr(2)) == DTYPE
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(eps=eps) == EPS and call(q=P, eq=eps) == EPS
    assert call(q=P, eq=0.0) == EPS
    assert call(ws=None) == WS and call(ws=addr(8)) == WS and call(nb=wb() - 1) == WS
    assert call(b=0, tok=None, starts=None) == OK
    assert wb(dt=3) == 0 and wb(n=-1) == 0 and wb(m=0) == 0 and wb(b=-1) == 0 and wb(m=(1 << 30) + 1) == 0
    assert wb(dt=BF16, n=512, m=131072, b=64) < 512 * 131072 // 64  # far below the scores


def test_python_refusals_need_no_gpu():
    x, idx = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    plan = sk.RoutePlan(idx, torch.zeros(8, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(TypeError):
        sk.route_sort([[1]], 3)
    with pytest.raises(ValueError, match="int32"):
        sk.route_sort(idx.long(), 3)
    with pytest.raises(ValueError, match="GPU"):
        sk.route_sort(idx, 3)
    for bad in (dict(k=0), dict(m=0), dict(align=0), dict(capacity=-1), dict(n=1 << 31)):
        with pytest.raises(ValueError, match="invalid"):
            sk.route_sort_rows(**{**dict(n=4, k=2, m=3, align=1, capacity=0), **bad})
    with pytest.raises(ValueError, match="invalid"):
        sk.route_sort_workspace(4, 2, 2000, "cpu")
    for call in (lambda t: sk.route_dispatch(t, plan), lambda t: sk.route_combine(t, plan),
                 lambda t: sk.route_combine_grad(t, plan, None, t)):
        with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
            call(x.double())
        with pytest.raises(ValueError, match="GPU"):
            call(x)
        with pytest.raises(ValueError, match="d\\)"):
            call(x[0])
    with pytest.raises(TypeError):
        sk.scores_verify([[1.0]], None, None, None, None)
    with pytest.raises(ValueError, match="GPU"):
        sk.scores_verify(x, None, None, None, None)
    with pytest.raises(ValueError, match="invalid"):
        sk.scores_verify_workspace(torch.float64, 4, 8, 1, "cpu")
    with pytest.raises(ValueError, match="invalid"):
        sk.scores_verify_workspace(torch.float32, 4, 0, 1, "cpu")
