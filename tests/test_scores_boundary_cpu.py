"""Refusals of the score-matrix entry points, checked without a GPU: every bad
argument returns its status (or raises) before anything is enqueued."""
import ctypes
import os

import pytest
import torch

import streaming_sinkhorn_solver_amd as sk
from streaming_sinkhorn_solver_amd import build as skbuild

P = ctypes.c_void_p(0x100000)  # never dereferenced: validation returns first
F32, BF16, F16 = 0, 1, 2
OK, NULL, SHAPE, EPS, ITERS, WS, DTYPE, ROUTE, OVERLAP = 0, 1, 2, 4, 5, 11, 18, 19, 20


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sk.LIB_PATH):
        skbuild.build()
    return sk.load_library()


def addr(off):
    return ctypes.c_void_p(0x100000 + off)


def test_status_strings(lib):
    for code in (DTYPE, ROUTE, OVERLAP):
        assert lib.sk_status_string(code) != b"unknown status"
        assert sk._STATUS_NAMES[code].startswith("SK_ERR_")


def test_solve_refusals(lib):
    wb = lib.sk_scores_solve_workspace_bytes(10, 12)
    assert wb > 0

    def call(s=P, dt=F32, n=10, m=12, ld=12, eps=0.1, it=3, f=P, g=P, ws=P, nb=wb):
        return lib.sk_scores_solve(s, dt, n, m, ld, None, None, eps, it, None, f, g, ws, nb, None)

    assert call(s=None) == NULL and call(f=None) == NULL and call(g=None) == NULL
    assert call(n=0) == SHAPE and call(n=-1) == SHAPE and call(n=1 << 31) == SHAPE
    assert call(m=0) == SHAPE and call(m=1025, ld=1025) == SHAPE and call(ld=11) == SHAPE
    assert call(ld=1 << 60) == SHAPE
    assert call(dt=3) == DTYPE and call(dt=-1) == DTYPE and call(s=addr(2)) == DTYPE and call(s=addr(1), dt=BF16) == DTYPE
    for eps in (0.0, -1.0, float("nan"), float("inf"), 1e-39):
        assert call(eps=eps) == EPS
    assert call(it=-1) == ITERS
    assert call(ws=None) == WS and call(ws=addr(16)) == WS and call(nb=wb - 1) == WS
    for n, m in ((0, 4), (4, 0), (-1, 4), (4, 1025), (1 << 31, 4)):
        assert lib.sk_scores_solve_workspace_bytes(n, m) == 0
    # the workspace does not grow with n beyond a bound
    assert lib.sk_scores_solve_workspace_bytes(1 << 30, 1024) <= 4 << 20


def test_route_refusals(lib):
    def call(s=P, dt=F32, n=10, m=12, ld=12, fn=0, on=0, ng=1, tg=1, gt=1, k=2, rn=1, scale=1.0, idx=P, w=P):
        return lib.sk_scores_route(s, dt, n, m, ld, fn, None, on, ng, tg, gt, k, rn, scale, idx, w, None, None)

    assert call(s=None) == NULL and call(idx=None) == NULL and call(w=None) == NULL
    assert call(n=-1) == SHAPE and call(m=0) == SHAPE and call(m=1025, ld=1025) == SHAPE and call(ld=11) == SHAPE
    assert call(dt=7) == DTYPE and call(s=addr(2)) == DTYPE
    for bad in (dict(fn=2), dict(fn=-1), dict(on=2), dict(ng=0), dict(ng=5), dict(ng=13), dict(ng=4, tg=5), dict(ng=4, tg=0),
                dict(gt=0), dict(gt=3), dict(ng=12, tg=4, gt=2), dict(k=0), dict(k=13), dict(ng=4, tg=2, k=7), dict(rn=2),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(m=130, ld=130, ng=65)):
        assert call(**bad) == ROUTE, bad
    assert call(m=100, ld=100, k=65) == ROUTE
    assert call(s=None, n=0, idx=None, w=None) == OK  # nothing to route

    def grad(s=P, n=10, m=12, ld=12, fn=0, k=2, rn=0, idx=P, dw=P, g=addr(1 << 16), ldg=12, dt=F32):
        return lib.sk_scores_route_grad(s, dt, n, m, ld, fn, idx, dw, k, rn, 1.0, g, ldg, None)

    assert grad(s=None) == NULL and grad(idx=None) == NULL and grad(dw=None) == NULL and grad(g=None) == NULL
    assert grad(fn=3) == ROUTE and grad(k=0) == ROUTE and grad(k=13) == ROUTE and grad(rn=-1) == ROUTE
    assert grad(ldg=11) == SHAPE and grad(g=addr((1 << 16) + 2)) == DTYPE
    assert grad(g=addr(4)) == OVERLAP  # shifted by one score
    assert grad(g=P, ldg=13, ld=12) == OVERLAP  # the same place with another stride
    assert grad(g=addr(40), ld=24, ldg=24) == OVERLAP  # windows of one buffer that share columns
    assert grad(n=0, s=None, idx=None, dw=None, g=None) == OK


def test_logprobs_refusals(lib):
    def wb(dt=F32, n=10, m=12, top=0):
        return lib.sk_scores_logprobs_workspace_bytes(dt, n, m, top)

    def call(s=P, dt=F32, n=10, m=12, ld=12, eps=1.0, t=P, top=0, logp=P, lse=P, ti=P, tl=P, st=P, ws=P, nb=None):
        return lib.sk_scores_logprobs(s, dt, n, m, ld, eps, t, top, logp, lse, None, ti, tl, st, ws,
                                      wb() if nb is None else nb, None)

    assert call(s=None) == NULL and call(logp=None) == NULL and call(lse=None) == NULL and call(st=None) == NULL
    assert call(top=2, ti=None) == NULL and call(top=2, tl=None) == NULL
    assert call(n=-1) == SHAPE and call(m=0) == SHAPE and call(ld=3) == SHAPE and call(top=13) == SHAPE
    assert call(top=-1) == SHAPE and call(m=200, ld=200, top=65) == SHAPE
    assert call(m=(1 << 20) + 1, ld=1 << 21, top=1, nb=1 << 40) == SHAPE
    assert call(dt=9) == DTYPE and call(s=addr(1), dt=F16) == DTYPE
    assert call(eps=0.0) == EPS and call(eps=float("nan")) == EPS and call(eps=1e-39) == EPS
    assert call(ws=None) == WS and call(ws=addr(8)) == WS and call(nb=wb() - 1) == WS
    assert call(n=0, s=None, logp=None, lse=None, st=None) == OK
    assert wb(dt=4) == 0 and wb(n=-1) == 0 and wb(m=0) == 0 and wb(top=13) == 0 and wb(m=1 << 21, top=1) == 0
    assert wb(n=64, m=131072, top=20, dt=BF16) < 64 * 131072 // 4  # far below the scores

    def grad(s=P, n=10, m=12, ld=12, eps=1.0, t=P, st=P, ent=P, top=0, ti=P, dl=P, de=None, dt_=None, g=addr(1 << 16),
             ldg=12, dt=F32):
        return lib.sk_scores_logprobs_grad(s, dt, n, m, ld, eps, t, st, ent, top, ti, dl, None, de, dt_, g, ldg, None)

    assert grad(s=None) == NULL and grad(st=None) == NULL and grad(t=None) == NULL and grad(g=None) == NULL
    assert grad(de=P, ent=None) == NULL and grad(top=2, dt_=P, ti=None) == NULL
    assert grad(eps=-1.0) == EPS and grad(top=65, m=100, ld=100, ldg=100) == SHAPE and grad(ldg=5) == SHAPE
    assert grad(g=addr(8)) == OVERLAP and grad(g=addr(2 + (1 << 16))) == DTYPE
    assert grad(n=0, s=None, st=None, t=None, g=None) == OK


def test_python_refusals_need_no_gpu():
    s = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        sk.scores_route([[1.0]], 1)
    for call in (lambda x: sk.scores_solve(x, eps=1.0, n_iters=1), lambda x: sk.scores_route(x, 2),
                 lambda x: sk.scores_logprobs(x)):
        with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
            call(s.double())
        with pytest.raises(ValueError, match=r"\(n, m\)"):
            call(s[0])
        with pytest.raises(ValueError, match="GPU"):
            call(s)
    with pytest.raises(ValueError, match="score_fn"):
        sk.scores_route(s, 2, score_fn="relu")
    with pytest.raises(ValueError, match="select_on"):
        sk.scores_route(s, 2, select_on="bias")
    with pytest.raises(ValueError, match="score_fn"):
        sk.scores_route_grad(s, None, None, score_fn="relu")
    with pytest.raises(ValueError, match="invalid"):
        sk.scores_logprobs_workspace(torch.float32, 4, 8, 9, "cpu")
    with pytest.raises(ValueError, match="invalid"):
        sk.scores_logprobs_workspace(torch.float64, 4, 8, 0, "cpu")
    with pytest.raises(ValueError, match="invalid"):
        sk.scores_solve_workspace(4, 2000, "cpu")
