"""Verification of drafted tokens in float64 (test infrastructure only).

Draft i of a sequence stands iff all before it do and u_i q_i(x_i) < p_i(x_i).
With n the number that stand, the next token is the least j with
d_0 + .. + d_j > u_K sum(d), where d = max(p_n - q_n, 0) while drafts remain
(p_n itself where that is 0 everywhere) and d = p_n after the last draft.
Entries that are not positive and finite weigh 0; -1 without any weight.

Pinned by: exact rationals (``fractions.Fraction``) on probabilities that are
multiples of a power of two, and the distribution of the emitted token, which
is the target's.
"""

from __future__ import annotations

import numpy as np


def _weights(d):
    d = np.asarray(d, np.float64)
    return np.where(np.isfinite(d) & (d > 0), d, 0.0)


def pick(d, u: float) -> int:
    """The least j whose running sum passes u * total; the last positive one if none; -1 without weight."""
    d = _weights(d)
    s = np.cumsum(d)
    if not s[-1] > 0:
        return -1
    over = np.flatnonzero((s > float(u) * s[-1]) & (d > 0))
    return int(over[0]) if over.size else int(np.flatnonzero(d > 0)[-1])


def verify(p, q, x, u, n_drafts: int):
    """One sequence: p [K+1, V], q [K, V] or None, x [K], u [K+1] -> (n, tokens of K + 1)."""
    K, V = len(x), p.shape[1]
    n = 0
    with np.errstate(invalid="ignore"):
        while n < n_drafts:
            if not 0 <= x[n] < V:
                break
            qx = 1.0 if q is None else float(q[n, x[n]])
            if not float(u[n]) * qx < float(p[n, x[n]]):
                break
            n += 1
        pn = np.asarray(p[n], np.float64)
        d = pn
        if n < n_drafts:
            if q is not None:
                d = pn - np.asarray(q[n], np.float64)
            else:
                d = pn.copy()
                if 0 <= x[n] < V:
                    d[x[n]] = 0.0
        t = pick(d, u[K])
        if t < 0 and n < n_drafts:
            t = pick(pn, u[K])
    return n, list(x[:n]) + [t] + [-1] * (K - n)
