"""Pins of the oracle's differential attention, block norm and page growth (CPU), and the binding's refusals."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import block_norm as ON
from oracle import differential as OD
from oracle import pages as OP
from paged_kv_cache_append_gb300 import build, nk
from tests.test_oracle_serving import Fake

F32, I32, I64, U8 = torch.float32, torch.int32, torch.int64, torch.uint8


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nk.LIB_PATH):
        build.build()
    return nk.load()


def inputs(F, H, G, D, T, seed=0):
    g = np.random.default_rng(seed)
    return (g.standard_normal((T, H * G, D)), g.standard_normal((F, H, D)), g.standard_normal((F, H, D)),
            g.uniform(0.1, 0.9, (T, H * G // 2)), g.standard_normal(2 * D))


# ------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("F,H,G,D,T", [(9, 2, 1, 8, 1), (70, 4, 3, 8, 3), (2, 2, 2, 8, 4)])
def test_differential_is_the_difference_of_four_plain_attentions(F, H, G, D, T):
    q, K, V, lam, w = inputs(F, H, G, D, T)
    out, lse, o, a = OD.attend(q, K, V, F - T, 0.3, lam, w, 1e-5, 0.2)
    for i in range(H * G // 2):
        j = i // G
        for n in range(T):
            keys = F - T + n + 1
            both = []
            for m in (0, 1):
                halves = [OA._attend(q[n, 2 * i + m], K[:, 2 * j + m], V[:, 2 * j + v], keys, 0.3) for v in (0, 1)]
                both.append(np.concatenate([h[0] for h in halves]))
                assert keys <= 0 or np.isclose(lse[n, 2 * i + m], halves[0][1], rtol=1e-12)
            want = both[0] - lam[n, i] * both[1]
            assert np.allclose(o[n, i], want, rtol=1e-12, atol=1e-14)
            if keys > 0:
                assert np.allclose(out[n, i], want / np.sqrt(np.mean(want ** 2) + 1e-5) * w * 0.2, rtol=1e-12)
                assert np.all(a[n, i] >= np.abs(want) - 1e-12)
            else:
                assert not out[n, i].any() and lse[n, 2 * i] == -np.inf


def test_differential_closed_forms():
    q, K, V, lam, _ = inputs(40, 2, 2, 8, 2)
    q[:, 1::2], K[:, 1] = q[:, ::2], K[:, 0]
    out = OD.attend(q, K, V, 38, 0.3, np.ones_like(lam))[0]
    assert np.abs(out).max() < 1e-14                                  # equal maps, lambda 1
    out = OD.attend(q, K, V, 38, 0.3, 0 * lam)[0]                     # lambda 0: the first map
    ref = OA.decode(q[:, ::2], K[:, :1], V[:, :1], 40, 0.3)[0]
    assert np.allclose(out[..., :8], ref, rtol=1e-12)


def test_block_norm_is_torchs():
    g = np.random.default_rng(3)
    y, r, gate, w, p = (g.standard_normal(s) for s in ((4, 24), (4, 24), (4, 24), 24, 24))
    x, h = ON.residual_norm(r, y, gate, w, p, eps=1e-4, offset=1.0, scale=0.7, residual_scale=-1.2, sigmoid=True)
    t = {n: torch.from_numpy(v) for n, v in dict(y=y, r=r, g=gate, w=w + 1, p=p + 1).items()}
    u = torch.nn.functional.rms_norm(t["y"], (24,), t["p"], 1e-4)
    ht = -1.2 * t["r"] + 0.7 * torch.sigmoid(t["g"]) * u
    assert np.allclose(h, ht.numpy(), rtol=1e-12)
    assert np.allclose(x, torch.nn.functional.rms_norm(ht, (24,), t["w"], 1e-4).numpy(), rtol=1e-12)
    assert ON.residual_norm(r, residual_scale=2.0)[0] is None
    assert np.array_equal(ON.residual_norm(r, residual_scale=2.0)[1], 2 * r)
    row = ON.residual_norm(np.array([[3.0, 4.0]]), weight=np.array([1.0, 2.0]), eps=0.0)[0]
    assert np.allclose(row, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])


def state(C, L, M, used, seed=0):
    perm = np.random.default_rng(seed).permutation(M).astype(np.int32)
    tables, at = np.full((C, L), -7, np.int32), 0
    for row, n in enumerate(used):
        tables[row, :n] = perm[at:at + n]
        at += n
    free = np.full(M, -9, np.int32)
    free[:M - at] = perm[at:]
    return tables, np.asarray(used, np.int32), free, M - at


def test_grow_by_hand():
    tables, mapped = np.array([[5, -1, -1], [2, 4, 0]], np.int32), np.array([1, 3], np.int32)
    free = np.array([3, 1, -1, -1, -1, -1], np.int32)
    got = OP.grow(tables, [0, 1], [60, 64], mapped, free, 2, 70, 6, counts=[70, 1])
    # row 1 keeps two pages and returns 0; row 0 needs three: takes 0, then 1
    assert got["tables"].tolist() == [[5, 0, 1], [2, 4, 0]] and got["mapped"].tolist() == [3, 2]
    assert got["n_free"] == 1 and got["free"][0] == 3 and got["frontiers"].tolist() == [130, 65]
    assert got["positions"][0, :2].tolist() == [60, 61] and got["positions"][1].tolist() == [64] + [-1] * 69
    assert got["slots"][0, 3:5].tolist() == [5 * 64 + 63, 0] and got["slots"][1, 0] == 4 * 64
    assert got["status"] == 0


@pytest.mark.parametrize("seed", range(20))
def test_grow_keeps_every_page_once_and_trims_back(seed):
    g = np.random.default_rng(seed)
    C, L = int(g.integers(1, 9)), int(g.integers(1, 30))
    M = int(g.integers(max(L, C), C * L + 1))
    used = np.zeros(C, int)
    for row in range(C):
        used[row] = g.integers(0, min(L, M - used.sum()) + 1)
    st = state(C, L, M, used, seed)
    B, T = int(g.integers(1, C + 1)), int(g.integers(0, 200))
    rows = g.permutation(C)[:B]
    committed = np.array([g.integers(0, max(1, 64 * used[r] - 70) + 1) for r in rows])
    counts = g.integers(0, T + 1, B)
    got = OP.grow(st[0], rows, committed, st[1], st[2], st[3], T, M, counts)
    held = [int(x) for r in range(C) for x in got["tables"][r, :got["mapped"][r]]] + got["free"][:got["n_free"]].tolist()
    assert sorted(held) == list(range(M))
    for b, r in enumerate(rows):
        if got["frontiers"][b]:
            assert got["mapped"][r] == -(-got["frontiers"][b] // 64)
    # a step and its trim: the stack and the counts are as before
    a = OP.grow(st[0], rows, committed, st[1], st[2], st[3], 0, M)
    ok = got["frontiers"] > 0
    if ok.all():
        one = OP.grow(a["tables"], rows, committed, a["mapped"], a["free"], a["n_free"], T, M, counts)
        if (one["frontiers"] > 0).all():
            two = OP.grow(one["tables"], rows, committed, one["mapped"], one["free"], one["n_free"], 0, M)
            assert two["n_free"] == a["n_free"] and np.array_equal(two["free"][:a["n_free"]], a["free"][:a["n_free"]])
            assert np.array_equal(two["mapped"], a["mapped"])


# ------------------------------------------------------- refusals of the library

def diff(**kw):
    d = dict(lam=64, lambda_stride=0, norm_weight=64, eps=1e-5, out_scale=1.0)
    d.update(kw)
    return nk.DiffDesc(*d.values())


def test_null_arguments_are_refused(lib):
    assert lib.nk_paged_diff_decode_attention(None, 8, None, 0, None, None, None, 1, 1, 1.0, None, None, None, None, 0,
                                              None) == -1
    assert lib.nk_paged_diff_prefill_attention(None, 8, None, 0, None, None, None, None, 1, 1, 1.0, None, None, None,
                                               None, 0, None) == -1
    n = ctypes.c_size_t()
    assert lib.nk_diff_decode_workspace_bytes(None, 1, 1, 2, ctypes.byref(n)) == -1
    assert lib.nk_diff_prefill_workspace_bytes(None, 1, 1, 2, ctypes.byref(n)) == -1
    assert lib.nk_pages_grow(*[None] * 11, 1, 1, *[None] * 4) == -1
    assert lib.nk_residual_norm(None, 64, 1, *[None, 0] * 5, None) == -1


def norm(**kw):
    """A status of nk_residual_norm that no launch follows."""
    d = dict(weight=64, post=64, eps=1e-6, offset=0.0, scale=1.0, rscale=1.0, sigmoid=0, wide=0, dim=64, N=4, y=64, ys=64,
             gate=64, gs=64, res=64, rs=64, ro=64, ros=64, x=64, xs=64)
    d.update(kw)
    desc = nk.BlockNormDesc(*list(d.values())[:8])
    return nk.load().nk_residual_norm(ctypes.byref(desc), *list(d.values())[8:], None)


@pytest.mark.parametrize("kw,code", [
    (dict(res=None), -1), (dict(ro=None, x=None, weight=None), -1), (dict(weight=None), -1), (dict(x=None), -1),
    (dict(y=None), -1), (dict(y=None, gate=None), -1), (dict(dim=0), -4), (dict(dim=68), -4), (dict(dim=16392), -4),
    (dict(N=0), -2), (dict(eps=0.0), -1), (dict(eps=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(rscale=float("nan")), -1), (dict(offset=float("inf")), -1), (dict(sigmoid=2), -1), (dict(wide=-1), -1),
    (dict(y=72), -5), (dict(gate=8), -5), (dict(res=68), -5), (dict(ro=72), -5), (dict(x=66), -5), (dict(weight=72), -5),
    (dict(post=72), -5), (dict(ys=68), -5), (dict(gs=4), -5), (dict(rs=2), -5), (dict(ros=65), -5), (dict(xs=12), -5),
    (dict(ros=56), -2), (dict(xs=0), -2), (dict(xs=-56), -2)])
def test_residual_norm_refuses(lib, kw, code):
    assert norm(**kw) == code, nk.load().nk_last_error()


# ------------------------------------------------------- refusals of the binding

def args_diff(prefill=False, **kw):
    d = dict(pool=0, layer=0, q=Fake(2, 3, 8, 64), tables=Fake(3, 5, dtype=I32), rows=Fake(2, dtype=I32),
             lengths=Fake(2, dtype=I32), chunk=Fake(2, dtype=I32) if prefill else None, scale=0.1, heads=4, tokens=0,
             width=128, out=Fake(2, 3, 4, 128), lse=Fake(2, 3, 8, dtype=F32), ws=64)
    d.update(kw)
    desc = diff()
    return nk._args().diff(prefill, d["pool"], 64, 3, 5, d["layer"], d["q"], d["tables"], d["rows"], d["lengths"],
                           d["chunk"], d["scale"], ctypes.addressof(desc), d["heads"], d["tokens"], d["width"], d["out"],
                           d["lse"], d["ws"], 0, 0)


@pytest.mark.parametrize("prefill", [False, True])
def test_diff_arguments(lib, prefill):
    assert args_diff(prefill) == -1                   # reaches the library, which refuses the NULL pool
    assert args_diff(prefill, tokens=6) == -1
    for kw in (dict(q=Fake(2, 3, 7, 64)), dict(q=Fake(2, 3, 8, 32)), dict(q=Fake(6, 8, 64)),
               dict(q=Fake(2, 3, 8, 64, dtype=torch.float16)), dict(q=Fake(2, 3, 8, 64, device=1)),
               dict(q=Fake(2, 3, 8, 64, stride=(1536, 64, 192, 1))), dict(tables=Fake(3, 4, dtype=I32)),
               dict(tables=Fake(3, 5, dtype=I64)), dict(rows=Fake(3, dtype=I32)), dict(lengths=Fake(2, 1, dtype=I32)),
               dict(heads=8), dict(tokens=5), dict(width=64), dict(out=Fake(2, 3, 8, 64)), dict(out=Fake(2, 3, 4, 64)),
               dict(lse=Fake(2, 3, 4, dtype=F32)), dict(lse=Fake(2, 3, 8)),
               dict(ws=torch.zeros(64, dtype=U8))) + ((dict(chunk=Fake(3, dtype=I32)),) if prefill else ()):
        with pytest.raises(ValueError):
            args_diff(prefill, **kw)
    with pytest.raises(TypeError):
        args_diff(prefill, layer=None)


def args_norm(**kw):
    d = dict(dim=64, y=Fake(4, 64), res=Fake(4, 64), gate=Fake(4, 64), x=Fake(4, 64), ro=Fake(4, 64), wide=False)
    d.update(kw)
    desc = nk.BlockNormDesc(64, 64, 0.0, 0.0, 1.0, 1.0, 0, int(d["wide"]))   # eps 0 is refused behind these checks
    return nk._args().residual_norm(ctypes.addressof(desc), d["dim"], d["y"], d["res"], d["gate"], d["x"], d["ro"],
                                    d["wide"], 0, 0)


def test_residual_norm_arguments(lib):
    three = dict(y=Fake(2, 2, 64), res=Fake(2, 2, 64), gate=Fake(2, 2, 64), x=Fake(2, 2, 64), ro=Fake(2, 2, 64))
    for kw in ({}, dict(dim=0), dict(gate=None), dict(gate=Fake(64)), three, dict(y=Fake(4, 64, stride=(200, 1))),
               dict(res=Fake(4, 64, dtype=F32), ro=Fake(4, 64, dtype=F32), wide=True)):
        assert args_norm(**kw) == -1, nk.load().nk_last_error()
        assert b"eps" in nk.load().nk_last_error()
    for kw in (dict(dim=128), dict(y=Fake(3, 64)), dict(y=Fake(4, 64, dtype=F32)), dict(gate=Fake(32)),
               dict(gate=Fake(1, 64)), dict(x=Fake(4, 64, stride=(1, 4))), dict(ro=Fake(4, 64, dtype=F32)),
               dict(res=Fake(4, 64, dtype=F32)), dict(res=Fake(64)), dict(x=Fake(4, 64, device=1)),
               dict(y=Fake(4, 64, device=-1)), dict(three, y=Fake(2, 2, 64, stride=(512, 64, 1)))):
        with pytest.raises(ValueError):
            args_norm(**kw)


def args_grow(**kw):
    d = dict(pool=0, T=4, tables=Fake(3, 5, dtype=I32), rows=Fake(2, dtype=I32), committed=Fake(2, dtype=I32),
             counts=Fake(2, dtype=I32), keep=Fake(3, dtype=I32), mapped=Fake(3, dtype=I32), mapped_out=Fake(3, dtype=I32),
             free=Fake(12, dtype=I32), n=Fake(1, dtype=I32), n_out=Fake(1, dtype=I32), frontiers=Fake(2, dtype=I32),
             positions=Fake(2, 4, dtype=I32), slots=Fake(2, 4, dtype=I64))
    d.update(kw)
    return nk._args().grow(d["pool"], 3, 5, 12, *list(d.values())[1:], 0, 0)


def test_grow_arguments(lib):
    for kw in ({}, dict(counts=None, keep=None), dict(positions=None, slots=None),
               dict(T=0, positions=Fake(2, 0, dtype=I32), slots=Fake(2, 0, dtype=I64))):
        assert args_grow(**kw) == -1
        assert b"null" in nk.load().nk_last_error()
    for kw in (dict(tables=Fake(3, 6, dtype=I32)), dict(rows=Fake(3, dtype=I32)), dict(committed=Fake(2, 1, dtype=I32)),
               dict(counts=Fake(3, dtype=I32)), dict(keep=Fake(2, dtype=I32)), dict(mapped=Fake(2, dtype=I32)),
               dict(mapped_out=Fake(3, dtype=I64)), dict(free=Fake(11, dtype=I32)), dict(n=Fake(2, dtype=I32)),
               dict(n_out=Fake(dtype=I32)), dict(frontiers=Fake(2)), dict(positions=Fake(2, 3, dtype=I32)),
               dict(slots=Fake(2, 4, dtype=I32)), dict(T=-1), dict(tables=Fake(3, 5, dtype=I32, device=-1))):
        with pytest.raises(ValueError):
            args_grow(**kw)
