"""The draft verification's sums: a long light tail, and the sizes at which the
kernel divides its work otherwise.

It takes a cluster of 8 CTAs a sequence while B * 8 fit the SMs, of 4 beyond,
fewer where V < 1024 per CTA, and searches a warp's chunk in a second step where
it is longer than 512 tokens (V over 512 * 16 * CTAs).
"""

from fractions import Fraction

import numpy as np
import pytest
import torch

from paged_kv_cache_append_gb300 import nk
from tests.test_gpu_verify import DEV, check, rows

pytestmark = pytest.mark.gpu


def light_tail(V, sign):
    """Weights whose first half sums to S1 and whose second to S2 = S1 (1 - sign 2^-37),
    so that u = 1/2 puts the border 2^-39 of the total below (above) the middle:
    four times what the kernel promises.  Every 128th of the first half is 64
    heavy tokens, then tokens below half a unit of a sum of 1 in fp32, then tokens
    below half a unit of the lost part's sum.  Added up as a pair of fp32 values a
    lane, the last ones are lost, 2^-34 of S1."""
    n = V // 128
    part = np.zeros(n, np.float32)
    part[:64] = 1
    part[256:n // 2] = 0.99 * 2.0 ** -25
    part[n // 2:] = 0.99 * 2.0 ** -42
    w = np.zeros(V, np.float32)
    w[:V // 2] = np.tile(part, 64)
    w[V // 2 - 1] = 2.0 ** -20                              # takes the border that lies below the middle
    exact = lambda a: sum(Fraction(float(v)) * int(c) for v, c in zip(*np.unique(a, return_counts=True)))  # noqa: E731
    s1 = exact(w[:V // 2])
    left = s1 * (1 - Fraction(sign, 2 ** 37))
    for j in range(4):
        w[V // 2 + j] = np.float32(float(left))
        left -= Fraction(float(w[V // 2 + j]))
        if left <= 0:
            break
    gap = (s1 - exact(w[V // 2:])) / s1 * 2 ** 37
    assert (w >= 0).all() and abs(gap - sign) < Fraction(1, 100)
    return w


@pytest.mark.parametrize("B", [2, 24])
@pytest.mark.parametrize("kind", ["no drafts", "draft rows", "certain drafts"])
@pytest.mark.parametrize("sign", [1, -1])
def test_a_long_light_tail(B, kind, sign):
    V = 1 << 22
    w = torch.from_numpy(light_tail(V, sign)).to(DEV)
    K = 0 if kind == "no drafts" else 1
    p, q = torch.zeros((B, K + 1, V), device=DEV), None
    p[:, 0] = w
    x = torch.full((B, K), 100, dtype=torch.int32, device=DEV)   # no weight: rejected
    if kind == "draft rows":
        q = p[:, :1].clone()
        p[:, 0] *= 2                                             # p - q = w
        q[:, 0, 100] = 1
    n, tok, _ = nk.verify_drafts(p, x, torch.full((B, K + 1), 0.5, device=DEV), draft=q)
    assert n.tolist() == [0] * B
    assert tok[:, 0].tolist() == [V // 2 - (sign > 0)] * B


@pytest.mark.parametrize("V", [1023, 1024, 2047, 2048, 2049, 4095, 4096, 8191, 8192, 8193, 32767, 32768, 32769, 65536,
                               65537])
@pytest.mark.parametrize("B", [2, 19, 20, 40])
@pytest.mark.parametrize("draft", [True, False])
def test_both_sides_of_every_division(V, B, draft):
    """Sums without rounding, random numbers on and off the borders."""
    rng = np.random.default_rng(V + B)
    K = 2
    p = rows(rng, (B, K + 1), V, 20)
    p[..., -1] += 2.0 ** -20
    q = rows(rng, (B, K), V, 20) if draft else None
    x = rng.integers(0, V, (B, K))
    if draft:
        q[np.arange(B)[:, None], np.arange(K), x] += p[np.arange(B)[:, None], np.arange(K), x]
    u = (rng.integers(0, 256, (B, K + 1)) / 256).astype(np.float32)
    u[0] = 0.0
    u[1] = np.float32(1 - 2.0 ** -24)
    check(p, q, x, u, fr=rng.integers(100, 1000, B))


@pytest.mark.parametrize("B", [8, 64])
@pytest.mark.parametrize("draft", [True, False])
def test_dense_rows_of_many_sequences(B, draft):
    """Softmax rows of an odd vocabulary, both cluster sizes with the second search step."""
    rng = np.random.default_rng(B)
    K, V = 2, 200003
    p = np.exp(rng.standard_normal((B, K + 1, V)).astype(np.float32) * 3 - 12)
    p /= p.sum(-1, keepdims=True)
    q = None
    if draft:
        q = p[:, :K] * np.exp(rng.standard_normal((B, K, V)).astype(np.float32) * 0.5)
        q /= q.sum(-1, keepdims=True)
    x = rng.integers(0, V, (B, K))
    u = rng.random((B, K + 1)).astype(np.float32)
    check(p, q, x, u, lens=rng.integers(0, K + 1, B), fr=rng.integers(100, 1000, B))
