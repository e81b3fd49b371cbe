"""The differential chunks' line of work: tiles cut between clusters, clusters
with many tiles, and calls beside one another.

Tolerance: as derived in test_gpu_diff.py, with f16 weights (2^-11) for every
page type, values as f16 (2^-11 at the worst), and 9e-4 for the E4M3 queries
and the fp32 steps: c = 2^-10 + 9e-4.
"""

import numpy as np
import pytest
import torch

from paged_kv_cache_append_gb300 import nk
from tests.test_gpu_diff import DEV, PROFILES, Batch, dev, normal

pytestmark = pytest.mark.gpu
C_TOL = 2.0 ** -10 + 9e-4


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("D,H,G,F,chunk", [
    (128, 2, 3, [0, 900, 401, 64, 1537, 128], [0, 1, 84, 64, 85, 128]),   # TQ 42: tiles end inside a cluster's half
    (64, 4, 64, [300, 131], [97, 131]),                                   # TQ 2: many short tiles to a cluster
    (128, 2, 1, [5000], [257]),                                           # few tiles, each cut many times
])
def test_pieces(profile, D, H, G, F, chunk):
    b = Batch(profile, D, H, G, max(chunk), F, chunk=chunk, seed=11)
    b.check(*b.run(), c=C_TOL)
    assert nk.nk_status_read(True) == 0


@pytest.mark.parametrize("profile", ["bf16", "int8_g64", "k8v4"])
def test_values_that_fall_and_rise_along_a_row(profile):
    """The strips' lifts, in both CTAs of a pair: the second half of the keys carries values 2^18 times the first's."""
    b = Batch(profile, 128, 2, 2, 200, [1600, 700], chunk=[200, 150], seed=3)
    b.fill(1, 2, mul=2.0 ** -9)
    for r in range(b.B):
        n, at = int(b.F[r]) // 2, int(b.F[r]) - int(b.F[r]) // 2
        k, v = normal((1, n, b.H, b.D), 40 + r), (normal((1, n, b.H, b.D), 60 + r).float() * 2.0 ** 9).to(torch.bfloat16)
        row = int(b.rows[r])
        b.gpu.append(0, dev(b.tables), dev([row], torch.int32), dev([at], torch.int32), k.to(DEV), v.to(DEV))
        from paged_kv_cache_append_gb300.workloads import bf16_to_bits
        b.img.append(0, b.tables, np.array([row]), np.array([at]), bf16_to_bits(k), bf16_to_bits(v))
    b.check(*b.run(), c=C_TOL)


def test_rows_behind_a_chunk_and_refused_rows_keep_what_they_hold():
    b = Batch("k8v4", 128, 2, 4, 150, [400, 90, 300], chunk=[150, 40, 100], seed=5)
    shape = (3, 150, 4, 256)
    out, lse = torch.full(shape, 7.0, dtype=torch.bfloat16, device=DEV), torch.full((3, 150, 8), 7.0, device=DEV)
    b.d["chunk"] = dev([150, 40, 151], torch.int32)   # the last is longer than the call's chunk: refused
    b.run(out=out, lse=lse)
    torch.cuda.synchronize()
    assert nk.nk_status_read(True) == nk.STATUS_FRONTIER
    for r, n in ((0, 150), (1, 40), (2, 0)):
        assert bool((out[r, n:] == 7).all()) and bool((lse[r, n:] == 7).all())
        assert not bool((lse[r, :n] == 7).any())
    b.d["chunk"] = dev(b.chunk)
    b.check(*b.run(out=out, lse=lse), c=C_TOL)


@pytest.mark.parametrize("chunk", [None, [70, 70, 70]])
def test_one_table_row_in_every_place_of_the_batch(chunk):
    b = Batch("fp8_row", 128, 2, 4, 70 if chunk else 2, [500, 500, 500], chunk=chunk, seed=8)
    b.rows[:] = b.rows[0]
    b.d["rows"] = dev(b.rows)
    b.fill(5, 6)
    b.check(*b.run(), c=C_TOL)


@pytest.mark.parametrize("profile", ["bf16", "nvfp4_g16"])
def test_chunks_on_two_streams_and_in_two_graphs(profile):
    batches = [Batch(profile, 128, 2, 4, 200, [3000, 1000], chunk=[200, 130], seed=s) for s in (0, 50)]
    wants = [[x.clone() for x in b.run()] for b in batches]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        got = [b.run(stream=s) for b, s in zip(batches, (None, side))]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for g, w in zip(got, wants) for x, y in zip(g, w))
    graphs, outs = [], []
    for b in batches:
        ws = b.gpu.diff_prefill_workspace(b.B, b.T, b.Hq)
        res = [torch.zeros_like(wants[0][0]), torch.zeros_like(wants[0][1])]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.run(out=res[0], lse=res[1], workspace=ws)
        graphs.append((g, ws))
        outs.append(res)
    for k in range(6):
        with torch.cuda.stream(side if k % 2 else torch.cuda.current_stream()):
            for g, _ in graphs:
                g.replay()
        torch.cuda.synchronize()
    for res, want, b in zip(outs, wants, batches):
        for r in range(b.B):
            n = int(b.chunk[r])
            assert all(torch.equal(x[r, :n], y[r, :n]) for x, y in zip(res, want))


@pytest.mark.parametrize("chunk", [None, [130]])
@pytest.mark.parametrize("G", [2, 16])
def test_pages_beyond_four_gigabytes(chunk, G):
    """Page ids whose byte offsets pass 32 bits give the bits of the same pages at the front."""
    H, D, T, F, L = 4, 128, 130 if chunk else 2, 700, 8750
    far, near = (nk.Pool("bf16", 1, H, D, 64 * L, 8, M) for M in (8 * L, L))
    k, v = (normal((1, F, H, D), s).to(DEV) for s in (1, 2))
    q = normal((1, T, H * G, D), 3).to(DEV)
    lam = torch.full((H * G // 2,), 0.4, device=DEV)
    diff, row, got = nk.Diff(lam, None), dev([0], torch.int32), []
    for pool, first in ((near, 0), (far, 8 * L - 11)):
        t = torch.zeros((8, L), dtype=torch.int32, device=DEV)
        t[0, :11] = torch.arange(first, first + 11, dtype=torch.int32, device=DEV)
        pool.append(0, t, row, dev([0], torch.int32), k, v)
        if chunk:
            got.append(pool.diff_prefill(0, q, t, row, dev([F - 130], torch.int32), dev(chunk, torch.int32), 0.1, diff))
        else:
            got.append(pool.diff_decode(0, q, t, row, dev([F], torch.int32), 0.1, diff))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*got)) and bool((got[0][0] != 0).any())
