"""Plain form of a beam search step in numpy and extended precision (test infrastructure)."""
import numpy as np


def lse(x):
    x = x.astype(np.longdouble)
    m = x.max()
    return m + np.log(np.exp(x - m).sum())


def select(rows, scores, n_out, finished=None, end_token=-1):
    """(parent, token, score, finished, len, status) of requests [R, beams]."""
    R, beams = scores.shape
    out = []
    for r in range(R):
        cand, status = [], set()
        for b in range(beams):
            s, x = scores[r, b], rows[r * beams + b]
            if np.isnan(s) or s == np.inf:
                status.add(23)
            elif s == -np.inf:
                continue
            elif finished is not None and finished[r, b]:
                cand.append((np.longdouble(s), b, 0.0, end_token, 1))
            elif np.isnan(x).any():
                status.add(1)
            elif (x == np.inf).any():
                status.add(2)
            elif (x > -np.inf).any():
                L = lse(x)
                live = np.flatnonzero(x > -np.inf)
                best = live[np.lexsort((live, -x[live].astype(np.float64)))][:n_out]  # logit desc, id asc
                for v in best:
                    cand.append((np.longdouble(s) + (np.longdouble(x[v]) - L), b, float(x[v]), int(v), int(v == end_token)))
        if status:
            out.append(([], min(status)))
            continue
        cand.sort(key=lambda c: (-c[0], c[1], -c[2], c[3]))
        out.append((cand[:n_out], 0))
    parent, token = np.full((R, n_out), -1, np.int32), np.zeros((R, n_out), np.int32)
    score, ended = np.full((R, n_out), -np.inf), np.zeros((R, n_out), np.int32)
    length, st = np.zeros(R, np.int32), np.zeros(R, np.int32)
    for r, (best, status) in enumerate(out):
        st[r], length[r] = status, len(best)
        for i, (s, b, _, v, e) in enumerate(best):
            parent[r, i], token[r, i], score[r, i], ended[r, i] = b, v, s, e
    return parent, token, score, ended, length, st
