"""GPU parity of the draft verification: whole numbers, equal to the oracle's.

The oracle and the kernel both sum in more than 46 bits, in other orders, so
they agree unless a random number falls within 2^-45 of a border.  The inputs
are multiples of a power of two whose sums are exact, where they agree even
when it falls on one, or random, where it does not come that near.
"""

import numpy as np
import pytest
import torch

from oracle import verify as OV
from paged_kv_cache_append_gb300 import nk

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rows(rng, shape, V, bits):
    """Probabilities that are multiples of 2^-bits, mostly zero for few bits."""
    w = rng.integers(0, 2 ** bits // max(1, min(V, 2 ** (bits - 2))) + 1, (*shape, V))
    return (w / 2.0 ** bits).astype(np.float32)


def run(p, q, x, u, lens=None, fr=None, pad=0):
    dev = lambda v: None if v is None else torch.from_numpy(np.ascontiguousarray(v)).to(DEV)  # noqa: E731
    t, d = dev(p), dev(q)
    if pad:
        V = p.shape[-1]
        wide = lambda v: torch.full((*v.shape[:-1], V + pad), float("nan"), device=DEV).index_copy(  # noqa: E731
            -1, torch.arange(V, device=DEV), v)[..., :V] if v is not None else None
        t, d = wide(t), wide(d)
    n, tok, f = nk.verify_drafts(t, dev(x.astype(np.int32)), dev(u), draft=d,
                                 draft_len=None if lens is None else dev(lens.astype(np.int32)),
                                 frontiers=None if fr is None else dev(fr.astype(np.int32)))
    return n.cpu().numpy(), tok.cpu().numpy(), None if f is None else f.cpu().numpy()


def check(p, q, x, u, lens=None, fr=None, pad=0):
    n, tok, f = run(p, q, x, u, lens, fr, pad)
    for b in range(p.shape[0]):
        K = x.shape[1]
        kb = K if lens is None else min(max(int(lens[b]), 0), K)
        en, et = OV.verify(p[b], None if q is None else q[b], x[b].tolist(), u[b], kb)
        assert n[b] == en and tok[b].tolist() == et, f"row {b}: {n[b]} {tok[b]} against {en} {et}"
        if fr is not None:
            assert f[b] == fr[b] - (kb - en)


@pytest.mark.parametrize("V", [1, 2, 3, 31, 33, 1000, 12799, 12800, 12801, 50021, 204800, 204801])
@pytest.mark.parametrize("K", [0, 1, 4])
@pytest.mark.parametrize("draft", [True, False])
def test_exact_sums(V, K, draft):
    """Sums without rounding, random numbers on and off the borders."""
    rng = np.random.default_rng(V * 10 + K)
    B = 6
    p = rows(rng, (B, K + 1), V, 20)
    p[..., -1] += 2.0 ** -20                                  # never without weight
    q = rows(rng, (B, K), V, 20) if draft else None
    x = rng.integers(0, V, (B, K))
    if draft:                                                 # about half of the drafts stand
        q[np.arange(B)[:, None], np.arange(K), x] += p[np.arange(B)[:, None], np.arange(K), x]
    u = (rng.integers(0, 256, (B, K + 1)) / 256).astype(np.float32)
    u[0] = 0.0
    u[1] = np.float32(1 - 2.0 ** -24)
    check(p, q, x, u, fr=rng.integers(100, 1000, B))


@pytest.mark.parametrize("V", [500009, 1 << 20])
def test_slices_of_several_tiles(V):
    """A vocabulary beyond one staged tile per CTA: the border in the first,
    a middle and the last tile of a slice."""
    rng = np.random.default_rng(V)
    B = 12
    p = rows(rng, (B, 2), V, 20)
    q = rows(rng, (B, 1), V, 20)
    x = rng.integers(0, V, (B, 1))
    q[np.arange(B), 0, x[:, 0]] += 0.5                        # rejected
    u = np.stack([np.full(B, 0.99), (np.arange(B) + 0.3) / B], 1).astype(np.float32)
    check(p, q, x, u)


@pytest.mark.parametrize("seed", range(4))
def test_softmax_rows(seed):
    """Softmax rows of 131072 tokens, drafts from the draft's distribution, ragged lengths, padded rows."""
    rng = np.random.default_rng(seed)
    B, K, V = 8, 5, 131072
    z = rng.standard_normal((B, K + 1, V)).astype(np.float32) * 3
    zq = z[:, :K] + rng.standard_normal((B, K, V)).astype(np.float32) * 0.5
    soft = lambda a: (np.exp(a - a.max(-1, keepdims=True)) / np.exp(a - a.max(-1, keepdims=True)).sum(-1, keepdims=True))  # noqa: E731
    p, q = soft(z).astype(np.float32), soft(zq).astype(np.float32)
    x = np.array([[rng.choice(V, p=q[b, i].astype(np.float64) / q[b, i].astype(np.float64).sum()) for i in range(K)]
                  for b in range(B)])
    u = rng.random((B, K + 1)).astype(np.float32)
    check(p, q, x, u, lens=rng.integers(-1, K + 2, B), fr=rng.integers(100, 1000, B), pad=7 if seed % 2 else 0)


def test_many_drafts():
    """More drafts than a warp has lanes, the first rejected one behind 32."""
    rng = np.random.default_rng(1)
    B, K, V = 3, 70, 50
    p = rows(rng, (B, K + 1), V, 20) + np.float32(2.0 ** -20)
    q = p[:, :K].copy()
    x = rng.integers(0, V, (B, K))
    q[1, 40, x[1, 40]] += 1.0
    q[2, 69, x[2, 69]] += 1.0
    u = np.full((B, K + 1), 0.75, np.float32)
    check(p, q, x, u)


def test_equal_rows_fall_back_to_the_target():
    """A rejection where p and q give the same weight everywhere (u q(x) = p(x)
    with u rounded up to 1): the next token comes from the target's row."""
    p = np.array([[[0.25, 0.25, 0.5], [1, 0, 0]]], np.float32)
    check(p, p[:, :1].copy(), np.array([[1]]), np.array([[1.0, 0.6]], np.float32))


def test_entries_that_are_not_probabilities_weigh_nothing():
    nan, inf = np.nan, np.inf
    p = np.array([[[nan, 0.25, inf, -1, 0.25, 0.5], [nan, nan, nan, -1, inf, 0]]], np.float32)
    q = np.array([[[nan, 0.5, 0.1, 0.1, nan, 0.125]]], np.float32)
    s = torch.cuda.current_stream().cuda_stream
    for u in (0.0, 0.3, 0.99, 1.0, nan):
        check(p, q, np.array([[1]]), np.array([[0.9, u]], np.float32))
    nk.nk_status_read(True, s)
    n, tok, _ = run(p[:, 1:], None, np.zeros((1, 0)), np.array([[0.5]], np.float32))
    assert n[0] == 0 and tok[0].tolist() == [-1]              # no weight anywhere
    assert nk.nk_status_read(True, s) == nk.STATUS_TOKEN_RANGE


def test_drafted_token_outside_the_vocabulary():
    rng = np.random.default_rng(3)
    s = torch.cuda.current_stream().cuda_stream
    p, q = rows(rng, (2, 3), 40, 10) + np.float32(2.0 ** -10), rows(rng, (2, 2), 40, 10)
    u = np.full((2, 3), 0.5, np.float32)
    for x in ([[40, 1], [-1, 2]], [[1 << 30, 1], [-(1 << 31), 2]]):
        nk.nk_status_read(True, s)
        check(p, q, np.array(x), u)
        assert nk.nk_status_read(True, s) == nk.STATUS_TOKEN_RANGE
        check(p, None, np.array(x), u)


def test_many_sequences_and_repeats():
    """More sequences than fit the GPU at once; the same bits on every call."""
    rng = np.random.default_rng(5)
    B, K, V = 300, 2, 30011
    p = rng.random((B, K + 1, V)).astype(np.float32)
    q = rng.random((B, K, V)).astype(np.float32)
    x, u = rng.integers(0, V, (B, K)), rng.random((B, K + 1)).astype(np.float32)
    check(p, q, x, u)
    first = run(p, q, x, u)
    for _ in range(3):
        again = run(p, q, x, u)
        assert all(np.array_equal(a, b) for a, b in zip(first[:2], again[:2]))


def test_rows_past_32_bits():
    """Largest vocabulary, more than 2^31 probabilities on both sides: the last
    sequences' draws come from the last rows."""
    B, K, V = 20, 7, 1 << 24
    p, q = torch.zeros((B, K + 1, V), device=DEV), torch.zeros((B, K, V), device=DEV)
    x = torch.arange(B * K, dtype=torch.int32, device=DEV).view(B, K) * 100003 % V
    p.scatter_(2, x.long()[..., None], 0.75)
    p[:, K, V - 1], p[:, K, 5] = 0.5, 0.25                    # u = 0.5: behind token 5
    q.scatter_(2, x.long()[..., None], 1.0)
    p[B - 1, K - 1], q[B - 1, K - 1] = 0.0, 0.0               # the last draft of the last sequence falls
    p[B - 1, K - 1, V - 2], q[B - 1, K - 1, V - 2] = 0.5, 0.25
    n, tok, _ = nk.verify_drafts(p, x, torch.full((B, K + 1), 0.5, device=DEV), draft=q)
    assert n.tolist() == [K] * (B - 1) + [K - 1]
    assert torch.equal(tok[:-1, :K], x[:-1]) and tok[:-1, K].tolist() == [V - 1] * (B - 1)
    assert tok[-1].tolist() == x[-1, :K - 1].tolist() + [V - 2, -1]


def test_frontiers_in_place_and_other_stream():
    rng = np.random.default_rng(6)
    p, q = rows(rng, (4, 3), 500, 20), rows(rng, (4, 2), 500, 20)
    x, u = rng.integers(0, 500, (4, 2)), rng.random((4, 3)).astype(np.float32)
    ref = run(p, q, x, u, fr=np.arange(4) + 50)
    dev = [torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for v in (p, q, x.astype(np.int32), u)]
    fr = (torch.arange(4, dtype=torch.int32) + 50).to(DEV)
    acc, out = torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros((4, 3), dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    nk.nk_verify_drafts(dev[0].data_ptr(), 500, dev[1].data_ptr(), 500, dev[2].data_ptr(), None, dev[3].data_ptr(),
                        fr.data_ptr(), 4, 2, 500, acc.data_ptr(), out.data_ptr(), fr.data_ptr(), s.cuda_stream)
    s.synchronize()
    assert np.array_equal(acc.cpu(), ref[0]) and np.array_equal(out.cpu(), ref[1]) and np.array_equal(fr.cpu(), ref[2])


def test_refused_tensors():
    t = torch.rand((2, 3, 10), device=DEV)
    x, u = torch.zeros((2, 2), dtype=torch.int32, device=DEV), torch.rand((2, 3), device=DEV)
    for kw in (dict(target=t.half()), dict(tokens=x.long()), dict(uniforms=u[:, :2]), dict(draft=t),
               dict(draft_len=x[0, :1]), dict(frontiers=u[0]), dict(target=t.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            nk.verify_drafts(**dict(dict(target=t, tokens=x, uniforms=u), **kw))
