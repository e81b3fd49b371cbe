"""Per-head RMS norm and position rotation in float64 (test infrastructure only).

    y_d = x_d / sqrt(mean(x^2) + eps) * (w_d + offset)          (w not None)
    (a, b) -> (a cos - b sin, b cos + a sin)

for the pairs (i, i + rd/2) (halves) or (2i, 2i + 1) (pairs), i < rd/2; dims
from rd on pass.  The cosines and sines are the values of the given table, as
the library takes them.

Pinned by: a rotation matrix applied pair by pair, and a closed form (angle 0
changes nothing, angle pi negates the rotated dims).
"""

from __future__ import annotations

import numpy as np


def norm_rotate(x, cos_sin, pos, rd: int, pairs: bool, weight=None, eps: float = 1e-6, offset: float = 0.0):
    """x float64 [N, heads, D], cos_sin [positions, rd], pos int [N] -> (y, m).

    m [N, heads, D] is the size of the terms of y (|a| + |b| of its pair after
    the norm), which bounds the rounding of an fp32 evaluation."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        r = np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
        x = x / r * (np.asarray(weight, np.float64) + offset)
    y, m = x.copy(), np.abs(x)
    cs = np.asarray(cos_sin, np.float64)[np.asarray(pos)]
    for i in range(rd // 2):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rd // 2)
        c, s = cs[:, None, i], cs[:, None, rd // 2 + i]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        m[..., a] = m[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, m


def table(positions: int, rd: int, base: float = 1e6) -> np.ndarray:
    """fp32 [positions, rd]: cosines then sines of pos * base^(-2i/rd)."""
    a = np.arange(positions)[:, None] * base ** (-np.arange(0, rd, 2) / max(rd, 1))
    return np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)
