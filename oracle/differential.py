"""Differential softmax attention over a logical KV sequence (test infrastructure only).

Heads come in pairs: query heads 2i and 2i + 1 are the two maps of head i, KV
heads 2j and 2j + 1 their keys, and the values of both side by side are one
value of 2 D elements; j = i // G.  With o = softmax(s1) V - lambda softmax(s2) V
the output is o / rms(o) * w * out_scale (no norm without w).  Visibility and
the empty key set are those of ``attention``.

Pinned by: ``attention.decode`` (each map against each half of the value, joined
by hand) and closed forms (equal maps with lambda = 1 give 0; lambda = 0 gives
the first map alone).
"""

from __future__ import annotations

import numpy as np


def attend(q, K, V, first, scale, lam, w=None, eps=1e-5, out_scale=1.0):
    """q float64 [N, Hq, D], query n at position first + n sees keys j <= first + n;
    K, V float64 [F, H, D]; lam float64 [N, Hq / 2]; w float64 [2 D] or None.

    Returns (out [N, Hq / 2, 2 D], lse [N, Hq], o before the norm, a): a is the
    attention of both maps over |V|, the second scaled by |lambda|.
    """
    N, Hq, D = q.shape
    F, H, _ = K.shape
    G = Hq // H
    o = np.zeros((N, Hq // 2, 2 * D))
    a = np.zeros_like(o)
    lse = np.full((N, Hq), -np.inf)
    for n in range(N):
        keys = min(F, first + n + 1)
        if keys <= 0:
            continue
        for i in range(Hq // 2):
            j = i // G
            v = np.concatenate([V[:keys, 2 * j], V[:keys, 2 * j + 1]], axis=1)
            for m, factor in ((0, 1.0), (1, -lam[n, i])):
                s = scale * (K[:keys, 2 * j + m] @ q[n, 2 * i + m])
                top = np.max(s)
                e = np.exp(s - top)
                z = np.sum(e)
                lse[n, 2 * i + m] = top + np.log(z)
                o[n, i] += factor * (e @ v) / z
                a[n, i] += abs(factor) * (e @ np.abs(v)) / z
    return finish(o, w, eps, out_scale), lse, o, a


def finish(o, w, eps, out_scale):
    """The norm and the scale."""
    if w is None:
        return o * out_scale
    return o / np.sqrt(np.mean(o * o, axis=-1, keepdims=True) + eps) * w * out_scale


def tolerance(out, o, a, w, eps, out_scale, c, half_step):
    """How far an output may be from ``out`` whose every term of o is off by at
    most c times its share of a, before one rounding of half_step.

    With d = c a the error of o, r = rms(d) / sqrt(rms(o)^2 + eps) bounds the
    relative error of the root by r (the triangle inequality of the norm), so the
    normed element moves by at most f (d + |o| r) / (1 - r), f = |w| out_scale /
    root; r >= 1 bounds nothing."""
    d = c * a
    if w is None:
        move = d * abs(out_scale)
    else:
        root = np.sqrt(np.mean(o * o, axis=-1, keepdims=True) + eps)
        r = np.sqrt(np.mean(d * d, axis=-1, keepdims=True)) / root
        assert np.all(r < 0.5), "the case says nothing: the difference of the maps cancels"
        move = np.abs(w * out_scale) / root * (d + np.abs(o) * r) / (1 - r)
    return move + half_step * (np.abs(out) + move)
