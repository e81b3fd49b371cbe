"""The shared-prefix attention over keys and values far from unit scale.

V = (N(0, 1) with 1% outliers x20 + 0.5) * v_mul, K = N(0, 1) * k_mul with the
softmax scale 4 / (sqrt(D) k_mul): the magnitudes of test_gpu_value_range.py,
here for the prefix pass and the rows' own pages together.

Tolerances, derived, per query row from the stored values.  A score is off by at
most d = 2^-16 s max|q| max_j |k_j|_1 + 1e-4, s the softmax scale: 2^-17 of the
largest |q| for each element where q enters as two E4M3 terms, the same again for
fp32 sums over 256 dims (2^-24 * 256 of the same) and any other form of q; 1e-4
for the exponentials (2^-22 of exponents up to 2^8) and the sums.  Weights move by
2 d relatively, f16 weights and values by 2^-11 more each, so the output by
(2 d + 2^-10) A, A the oracle's attention over |V|, and half a bf16 step of the
output, 2^-8 of it; lse by d.  Weights below f16's normal range, 2^-14 of the row's
largest, lose up to 2^-25 each: 2^-25 n max|v| for n keys; values below it 2^-25.
"""

import math

import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import formats as OF
from paged_kv_cache_append_gb300.workloads import bf16_to_bits
from tests.test_gpu_shared import PROFILES, Batch

pytestmark = pytest.mark.gpu


def case(monkeypatch, profile, D, G, T, k_mul, v_mul):
    seen = []

    def values(shape, seed):
        g = torch.Generator().manual_seed(seed)
        x = torch.randn(shape, generator=g)
        i = len(seen) % 2 if len(shape) == 3 else 2          # keys and values in turn, then the queries
        seen.append(shape)
        if i == 1:
            x = torch.where(torch.rand(shape, generator=g) < 0.01, 20 * x, x) + 0.5
        return (x * (k_mul, v_mul, 1.0)[i]).to(torch.bfloat16)

    monkeypatch.setattr("tests.test_gpu_shared.normal", values)
    pages = 5
    b = Batch(profile, D, 2, G, T, pages, [64 * pages + x for x in (T, 70, 130)], seed=D)
    b.scale = 4 / math.sqrt(D) / k_mul
    return b, pages


def check(b, pages):
    out, lse = b.run(pages)
    q = OF.bf16_bits_to_f64(bf16_to_bits(b.q))
    for i in range(b.B):
        K, V = b.img.gather(0, b.tables[b.rows[i]], int(b.F[i]))
        o, l = OA.decode(q[i], K, V, int(b.F[i]), b.scale)
        a, _ = OA.decode(q[i], K, np.abs(V), int(b.F[i]), b.scale)
        d = 2.0 ** -16 * b.scale * np.abs(q[i]).max() * np.abs(K).sum(-1).max() + 1e-4
        got, gl = out[i].double().numpy(), lse[i].double().numpy()
        limit = 2.0 ** -8 * np.abs(o) + (2 * d + 2.0 ** -10) * a + 2.0 ** -25 * (len(K) * np.abs(V).max() + 1)
        assert np.all(np.isfinite(got))
        assert np.all(np.abs(got - o) <= limit), f"row {i}: {(np.abs(got - o) / limit).max()} of the tolerance"
        assert np.abs(gl - l).max() <= d


@pytest.mark.parametrize("v_mul", [2.0 ** -14, 2.0 ** -8, 2.0 ** 10, 2.0 ** 17, 2.0 ** 22])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("G,T", [(8, 1), (8, 4)])
def test_value_range(monkeypatch, profile, D, G, T, v_mul):
    if G * T > 16 and D == 256 and profile in ("bf16", "int8_g64"):
        pytest.skip("not a decode of this profile")
    check(*case(monkeypatch, profile, D, G, T, 1.0, v_mul))


@pytest.mark.parametrize("k_mul", [2.0 ** -8, 2.0 ** 8, 2.0 ** 17])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("profile", PROFILES)
def test_key_range(monkeypatch, profile, D, k_mul):
    check(*case(monkeypatch, profile, D, 4, 2, k_mul, 1.0))
