"""Plain binary64 implementations of the operators on logit rows: shaping,
top logits and the distillation loss with its gradient.  One row at a time,
written from the definitions; inputs are the binary32 / bf16 values as
float64, ids and masks are whole numbers.  Test infrastructure only."""
from __future__ import annotations

import numpy as np

ST_OK = 0
ST_ROW_NAN, ST_ROW_POSINF, ST_ROW_ZERO_MASS, ST_BAD_TOPK = 1, 2, 3, 9
ST_Q_BAD_LEN, ST_Q_BAD_ID, ST_Q_UNSORTED, ST_Q_NONFINITE = 10, 11, 12, 13
ST_BAD_HISTORY, ST_BAD_PENALTY, ST_BAD_BIAS, ST_BAD_MASK = 19, 20, 21, 22


def shape_row(x, prompt=(), made=(), rep=1.0, freq=0.0, pres=0.0, temp=1.0, bias=(), allowed=None):
    """Shaped logits of one row and, per logit, the sum of the magnitudes
    that its value is built from (what rounding errors are relative to).
    prompt, made: token ids; bias: (id, value) pairs; allowed: bool [V]."""
    x = np.asarray(x, np.float64)
    z = x.copy()
    mag = np.abs(x)
    count = {}
    for t in made:
        count[int(t)] = count.get(int(t), 0) + 1
    for t in set(int(t) for t in prompt) | set(count):
        with np.errstate(invalid="ignore", over="ignore"):
            z[t] = z[t] / rep if z[t] > 0 else z[t] * rep
            mag[t] = abs(z[t])
            c = count.get(t, 0)
            if c:
                z[t] = z[t] - freq * c - pres
                mag[t] += abs(freq) * c + abs(pres)
    for t, b in bias:
        z[int(t)] += b
        mag[int(t)] += abs(b)
    z /= temp
    mag = mag / temp
    if allowed is not None:
        z = np.where(allowed, z, -np.inf)
        mag = np.where(allowed, mag, 0.0)
    return z, mag


def row_status(x):
    x = np.asarray(x, np.float64)
    if np.isnan(x).any():
        return ST_ROW_NAN
    if (x == np.inf).any():
        return ST_ROW_POSINF
    if (x == -np.inf).all():
        return ST_ROW_ZERO_MASS
    return ST_OK


def logsumexp(u):
    m = u.max()
    return m + np.log(np.exp(u - m).sum())


def top_row(x, k, temp=1.0):
    """(status, ids ascending, logits, lse) of one row."""
    x = np.asarray(x, np.float64)
    st = row_status(x)
    if st != ST_OK:
        return st, np.zeros(0, np.int64), np.zeros(0), 0.0
    finite = np.flatnonzero(x > -np.inf)
    best = sorted(finite.tolist(), key=lambda v: (-x[v], v))[:k] if len(finite) <= 4096 else \
        finite[np.lexsort((finite, -x[finite]))][:k].tolist()
    ids = np.array(sorted(best), np.int64)
    return st, ids, x[ids], logsumexp(x / temp)


def list_status(ids, z, lse, V, k_max, length):
    """Refusal of a teacher's list (its first `length` entries)."""
    if length < 0 or length > k_max:
        return ST_Q_BAD_LEN
    ids, z = np.asarray(ids[:length], np.int64), np.asarray(z[:length], np.float64)
    if ((ids < 0) | (ids >= V)).any():
        return ST_Q_BAD_ID
    if (np.diff(ids) <= 0).any():
        return ST_Q_UNSORTED
    if not np.isfinite(z).all() or (length and lse is not None and not np.isfinite(lse)):
        return ST_Q_NONFINITE
    return ST_OK


def distill_row(x, ids, z, temp=1.0, lse=None):
    """(loss, gradient, q, p over the vocabulary, P, Q) of one good row with a nonempty list."""
    x, z = np.asarray(x, np.float64), np.asarray(z, np.float64)
    ids = np.asarray(ids, np.int64)
    d = (x - x.max()) / temp  # (from the maximum: a row far from zero keeps its differences)
    logq = d - np.log(np.exp(d).sum())
    q = np.exp(logq)
    lp = z / temp - (logsumexp(z / temp) if lse is None else float(lse))
    p = np.exp(lp)
    with np.errstate(invalid="ignore"):
        loss = float(np.where(p > 0, p * (lp - logq[ids]), 0.0).sum())
    # the derivative of -p_j log q_j is p_j q_v - p_j [v = j]: the softmax times sum p, which with P is one
    grad = q.copy()
    P = Q = 0.0
    off = np.ones(len(x), bool)
    off[ids] = False
    if lse is not None:
        P, Q = max(0.0, 1.0 - float(p.sum())), float(q[off].sum())
        if P > 0 and Q > 0:
            loss += P * np.log(P / Q)
            grad[off] *= 1.0 - P / Q
        else:
            P = 0.0
            grad *= float(p.sum())
    grad[ids] -= p
    full = np.zeros(len(x))
    full[ids] = p
    return loss, grad / temp, q, full, P, Q
