"""Dense float64 reference of the operators on a given score matrix.

Plain numpy from the definitions, with no running maximum, no base 2 and no
float32: Sinkhorn potentials with the cost -scores, routing to experts, token
log-probabilities, and the gradients of the last two.  Test infrastructure.
"""
from __future__ import annotations

import numpy as np


def _lse(z, axis):
    """log-sum-exp; -inf where nothing is left."""
    top = np.max(z, axis=axis, keepdims=True)
    top = np.where(np.isfinite(top), top, 0.0)
    with np.errstate(divide="ignore"):
        return np.squeeze(top, axis) + np.log(np.sum(np.exp(z - top), axis=axis))


def _log(w):
    with np.errstate(divide="ignore"):
        return np.log(np.asarray(w, np.float64))


def solve(scores, a, b, eps, n_iters, g_init=None):
    """Alternating half-steps f_i = -eps LSE_j[(g_j + s_ij)/eps + log b_j] and its transpose; potential 0 for a row or
    column that nothing is left of."""
    s = np.asarray(scores, np.float64)
    n, m = s.shape
    la = _log(np.full(n, 1.0 / n) if a is None else a)
    lb = _log(np.full(m, 1.0 / m) if b is None else b)
    s = np.where(la[:, None] == -np.inf, np.where(np.isfinite(s), s, 0.0), s)  # padding may hold anything
    f, g = np.zeros(n), np.zeros(m) if g_init is None else np.asarray(g_init, np.float64).copy()
    for _ in range(n_iters):
        x = _lse((g[None, :] + s) / eps + lb[None, :], 1)
        f = np.where(x == -np.inf, 0.0, -eps * np.where(x == -np.inf, 0.0, x))
        x = _lse((f[:, None] + s) / eps + la[:, None], 0)
        g = np.where(x == -np.inf, 0.0, -eps * np.where(x == -np.inf, 0.0, x))
    return f, g


def _log_softmax(z):
    """log softmax of each row, from differences to its largest entry (rows of large numbers lose nothing); -inf in an
    empty row."""
    top = np.max(z, axis=1, keepdims=True)
    top = np.where(top == -np.inf, 0.0, top)
    x = _lse(z - top, 1)
    return z - top - np.where(x == -np.inf, 0.0, x)[:, None]


def _softmax(s):
    return np.exp(_log_softmax(s))


def _sigmoid(s):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-s))


def _order(v, k):
    """Columns of the k largest of each row, descending, ties to the lower column; a NaN ranks as -inf."""
    return np.argsort(-np.where(np.isnan(v), -np.inf, v), axis=1, kind="stable")[:, :k]


def route_values(scores, fn, bias, select_on):
    """The values that decide the choice."""
    s = np.asarray(scores, np.float64)
    v = s if select_on == "logit" else _softmax(s) if fn == "softmax" else _sigmoid(s)
    return v if bias is None else v + np.asarray(bias, np.float64)


def route(scores, k, fn="softmax", bias=None, select_on="score", n_group=1, topk_group=1, group_top=1, renorm=True,
          scale=1.0):
    """(idx, weights, counts)."""
    s = np.asarray(scores, np.float64)
    n, m = s.shape
    # softmax and sigmoid rise with the score: where they alone decide, the scores decide (v is for the groups' sums)
    alone = bias is None and (n_group == 1 or group_top == 1)
    v = s if alone else route_values(s, fn, bias, select_on)
    if n_group > 1:
        per = v.reshape(n, n_group, m // n_group)
        score = np.sort(per, axis=2)[:, :, -group_top:].sum(axis=2)
        keep = np.zeros((n, n_group), bool)
        np.put_along_axis(keep, _order(score, topk_group), True, axis=1)
        if bias is None:
            v = s
        # columns of the other groups rank behind everything, masked ones included
        rank = np.empty((n, m), np.int64)
        np.put_along_axis(rank, _order(v, m), np.arange(m)[None, :].repeat(n, 0), axis=1)
        rank = rank + np.where(np.repeat(keep, m // n_group, axis=1), 0, m)
        idx = np.argsort(rank, axis=1, kind="stable")[:, :k]
    else:
        idx = _order(v, k)
    return idx, scale * _weights(s, idx, fn, renorm), np.bincount(idx.reshape(-1), minlength=m)


def _log_act(s, idx, fn):
    if fn == "sigmoid":
        return -np.logaddexp(0.0, -np.take_along_axis(s, idx, 1))
    return np.take_along_axis(_log_softmax(s), idx, 1)


def _weights(s, idx, fn, renorm):
    la = _log_act(s, idx, fn)
    return _softmax(la) if renorm else np.exp(la)


def route_grad(scores, idx, dw, fn="softmax", renorm=True, scale=1.0):
    """Gradient of the weights in the scores at the choice idx: the Jacobian of log weights, entry by entry."""
    s = np.asarray(scores, np.float64)
    n, m = s.shape
    q = _weights(s, idx, fn, renorm)
    part = q * np.asarray(dw, np.float64) * scale  # gradient in log q
    if renorm:
        part = part - q * part.sum(axis=1, keepdims=True)  # ... in log act
    out = np.zeros((n, m))
    if fn == "sigmoid":
        part = part * _sigmoid(-np.take_along_axis(s, idx, 1))
    for r in range(idx.shape[1]):
        out[np.arange(n), idx[:, r]] += part[:, r]
    if fn == "softmax" and not renorm:
        out -= _softmax(s) * part.sum(axis=1, keepdims=True)
    return out


def logprobs(scores, targets, eps=1.0, top=0):
    """dict(logp, lse, entropy, top_idx, top_logp)."""
    s = np.asarray(scores, np.float64)
    n, m = s.shape
    lse = _lse(s / eps, 1)
    lp = _log_softmax(s / eps)
    p = np.exp(lp)
    out = dict(lse=lse, entropy=-np.sum(np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0), axis=1))
    if targets is not None:
        t = np.asarray(targets)
        inside = np.clip(t, 0, m - 1)
        out["logp"] = np.where(t < 0, 0.0, np.where(t >= m, np.nan, lp[np.arange(n), inside]))
    if top:
        out["top_idx"] = _order(s, top)
        out["top_logp"] = np.take_along_axis(lp, out["top_idx"], 1)
    return out


def logprobs_grad(scores, targets, eps=1.0, top_idx=None, d_logp=None, d_lse=None, d_entropy=None, d_top=None):
    s = np.asarray(scores, np.float64)
    n, m = s.shape
    rows = np.arange(n)
    r = logprobs(s, None, eps)
    lp = _log_softmax(s / eps)
    p = np.exp(lp)
    out = np.zeros((n, m))
    if d_lse is not None:
        out += p * np.asarray(d_lse, np.float64)[:, None]
    if d_logp is not None:
        g = np.where(np.asarray(targets) < 0, 0.0, np.asarray(d_logp, np.float64))
        out -= p * g[:, None]
        out[rows, np.maximum(targets, 0)] += g
    if d_top is not None:
        for k in range(top_idx.shape[1]):
            g = np.asarray(d_top, np.float64)[:, k]
            out -= p * g[:, None]
            out[rows, top_idx[:, k]] += g
    if d_entropy is not None:
        plp = np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0)
        out -= (plp + p * r["entropy"][:, None]) * np.asarray(d_entropy, np.float64)[:, None]
    return out / eps
