"""Norms before and after a block with its gate and residual scales, in float64 (test infrastructure only).

u = post(y), h = residual_scale r + scale act(g) u, x = norm(h).  Pinned by
torch's rms_norm in float64 (a library routine) and by hand on one row.
"""

from __future__ import annotations

import numpy as np


def rms(x, w, eps, offset=0.0):
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * (w + offset)


def residual_norm(r, y=None, gate=None, weight=None, post=None, eps=1e-6, offset=0.0, scale=1.0, residual_scale=1.0,
                  sigmoid=False):
    """Returns (x or None, h)."""
    h = residual_scale * r
    if y is not None:
        u = y if post is None else rms(y, post, eps, offset)
        if gate is not None:
            u = u * (1 / (1 + np.exp(-gate)) if sigmoid else gate)
        h = h + scale * u
    return (None if weight is None else rms(h, weight, eps, offset)), h
