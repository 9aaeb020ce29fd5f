"""Float64 reference of token rows under a routing and of the verification of drafted tokens.

Plain numpy, pair by pair and row by row from the definitions.  Test infrastructure.
"""
from __future__ import annotations

import numpy as np

from .scores import _log_softmax


def sort_rows(n, k, m, align=1, capacity=0):
    """The most rows that n tokens' sorted choices take."""
    rows = n * k + min(n * k, m) * (align - 1)
    return min(rows, m * -(-capacity // align) * align) if capacity else rows


def sort(idx, m, align=1, capacity=0, rows=None):
    """(slot, source, counts, offsets) of choices idx (n, k): each expert's in order, segments rounded up to align."""
    n, k = idx.shape
    flat = [int(e) for e in np.asarray(idx).reshape(-1)]
    mine = [[] for _ in range(m)]
    for t, e in enumerate(flat):
        if 0 <= e < m and not (capacity and len(mine[e]) >= capacity):
            mine[e].append(t)
    source = np.full(sort_rows(n, k, m, align, capacity) if rows is None else rows, -1, np.int32)
    slot = np.full(n * k, -1, np.int32)
    offsets = [0]
    for pairs in mine:
        for r, t in enumerate(pairs):
            slot[t] = offsets[-1] + r
            source[offsets[-1] + r] = t
        offsets.append(offsets[-1] + -(-len(pairs) // align) * align)
    return slot.reshape(n, k), source, np.array([len(p) for p in mine], np.int32), np.array(offsets, np.int32)


def dispatch(x, slot, offsets, weights, out):
    """out with x's rows at their slots, zeros in the rest of the segments, unchanged from offsets[-1] on."""
    out = np.array(out, np.float64)
    out[:offsets[-1]] = 0.0
    for i, r in zip(*np.nonzero(slot >= 0)):
        out[slot[i, r]] = np.asarray(x[i], np.float64) * (1.0 if weights is None else float(weights[i, r]))
    return out


def combine(rows, slot, weights=None, add=None):
    """y_i = add_i + sum over r of weights_ir rows[slot_ir]."""
    y = np.zeros((slot.shape[0], rows.shape[1])) if add is None else np.array(add, np.float64)
    for i, r in zip(*np.nonzero(slot >= 0)):
        y[i] += np.asarray(rows[slot[i, r]], np.float64) * (1.0 if weights is None else float(weights[i, r]))
    return y


def combine_grad(rows, slot, offsets, weights, d_y, out):
    """(d_rows, d_weights)."""
    d_weights = np.zeros(slot.shape)
    for i, r in zip(*np.nonzero(slot >= 0)):
        d_weights[i, r] = np.dot(np.asarray(rows[slot[i, r]], np.float64), np.asarray(d_y[i], np.float64))
    return dispatch(d_y, slot, offsets, weights, out), d_weights


def distribution(scores, eps):
    """(probabilities, log-probabilities) of one row; eps 0: one at the first largest score; an empty row: zeros."""
    s = np.asarray(scores, np.float64)
    eps = float(np.float32(eps))  # as it is handed over
    if eps == 0.0:
        p = np.zeros_like(s)
        if np.any(s > -np.inf):
            p[np.argmax(s)] = 1.0
        with np.errstate(divide="ignore"):
            return p, np.log(p)
    z = _log_softmax(s[None, :] / eps)[0]
    return np.exp(z), z


def draw(weights, u):
    """The first column whose cumulative weight exceeds u of the whole; -1 where there is none."""
    total = np.cumsum(weights)
    if not total[-1] > 0.0:
        return -1
    over = np.nonzero(total > u * total[-1])[0]
    return int(over[0]) if len(over) else int(np.nonzero(weights > 0)[0][-1])


def verify(scores, tokens, starts, u_accept, u_sample, draft=None, eps=1.0, eps_draft=1.0, fill=None):
    """(accepted, next, tokens, ratio, logp); fill: the (tokens, ratio, logp) of rows of no request."""
    s = np.asarray(scores, np.float64)
    n, m = s.shape
    b = len(starts) - 1
    accepted, after = np.zeros(b, np.int32), np.full(b, -1, np.int64)
    emitted, ratio, logp = (np.array(f) for f in fill) if fill else (np.full(n, -1, np.int64), np.zeros(n), np.zeros(n))
    for r in range(b):
        stopped = ended = False
        for i in range(int(starts[r]), int(starts[r + 1])):
            emitted[i], ratio[i], logp[i] = -1, 0.0, 0.0
            if ended:
                continue
            bad = np.any(np.isnan(s[i]) | (s[i] == np.inf))
            p, lp = distribution(s[i], eps) if not bad else (np.zeros(m), np.full(m, -np.inf))
            t = int(tokens[i])
            q = np.zeros(m)
            if t >= 0:
                if draft is not None and eps > 0.0:
                    d = np.asarray(draft[i], np.float64)
                    wrong = np.any(np.isnan(d) | (d == np.inf))
                    bad = bad or wrong
                    q = distribution(d, eps_draft)[0] if not wrong else q
                elif t < m:
                    q[t] = 1.0
                pt, qt = (p[t], q[t]) if t < m else (0.0, 1.0)
                ratio[i] = np.nan if bad else 0.0 if pt == 0.0 else 1.0 if pt >= qt else pt / qt
                taken = ratio[i] > 0.0 and (eps == 0.0 or float(u_accept[i]) * qt < pt)
            ended = t < 0
            if stopped:
                continue
            if t >= 0 and taken:
                accepted[r] += 1
                emitted[i], logp[i] = t, lp[t]
                continue
            stopped = True
            if bad:
                continue
            w = np.maximum(p - q, 0.0)
            after[r] = draw(w if w.sum() > 0.0 else p, 0.0 if eps == 0.0 else float(u_sample[r]))
            if after[r] >= 0:
                emitted[i], logp[i] = after[r], lp[after[r]]
    return accepted, after, emitted, ratio, logp
