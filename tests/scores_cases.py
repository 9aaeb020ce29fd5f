"""Inputs and error bounds shared by the GPU tests of the score-matrix operators.

The bounds count float32 roundings of the computation as the library documents it
(differences from the row's maximum, one multiplication by log2e / eps, hardware
exp2 and log2 of one unit in the last place), with u = 2^-24 the half step.
"""
import numpy as np
import torch

U = 2.0 ** -24
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda:0"


def matrix(n, m, dtype, seed, spread=2.5, pad=0, offset=0, mask=0.0, ties=False):
    """(scores on the GPU: a window of a wider, shifted buffer, its float64 numpy copy)."""
    r = np.random.default_rng(seed)
    x = r.normal(size=(n, m)) * spread
    if ties:
        x = np.round(x)
    if mask:
        x[r.random((n, m)) < mask] = -np.inf
    ld = m + pad
    buf = torch.full((offset + n * ld,), float("nan"), dtype=DTYPES[dtype])
    win = buf[offset:].view(n, ld)[:, :m]
    win.copy_(torch.from_numpy(x))
    dev = buf.to(DEV)[offset:].view(n, ld)[:, :m]
    return dev, win.double().numpy()


def half_step(dtype):
    return torch.finfo(DTYPES[dtype]).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, tol, what):
    """Elementwise |got - want| <= tol, with infinities and NaN in the same places."""
    got, want, tol = np.broadcast_arrays(f64(got) if isinstance(got, torch.Tensor) else got, want, tol)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), what
    ok = ~(inf | np.isnan(want))
    err = np.abs(got[ok] - want[ok])
    worst = float((err / np.maximum(tol[ok], 1e-300)).max()) if err.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound (error {err.max():.3g})"


def softmax_terms(s, eps):
    """d = (s - max)/eps, p, log sum, E|d|, E d^2 of each row (float64; an empty row: p = 0)."""
    top = s.max(1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        d = np.where(np.isfinite(s), (s - np.where(np.isfinite(top), top, 0.0)) / eps, -np.inf)
        e = np.exp(d)
        tot = e.sum(1, keepdims=True)
        p = np.where(tot > 0, e / tot, 0.0)
        log_s = np.where(tot > 0, np.log(np.where(tot > 0, tot, 1.0)), 0.0)[:, 0]
    fd = np.where(np.isfinite(d), d, 0.0)
    return fd, p, log_s, (p * np.abs(fd)).sum(1), (p * fd ** 2).sum(1)


def log_sum_error(e1):
    """log S: every term carries 3 u |d| (subtraction, factor, product) and 2 u (exp2); at most 128 + 16 additions in
    a row (a lane's entries, lanes, waves, chunks), one multiplication per joined chunk, and the logarithm."""
    return (3 * e1 + 2 + 150) * U


def entropy_error(log_s, e1, e2):
    """H = log S - X / S: X's terms e d carry the errors of e and of d, and its sum's additions are relative to E|d|."""
    return log_sum_error(e1) + (3 * e2 + 5 * e1 + 150 * e1 + 150 * e1 + 4 * e1 + 2 * np.abs(log_s)) * U
