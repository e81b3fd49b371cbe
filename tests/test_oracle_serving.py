"""CPU pins of the rotation and verification oracles, and the refusals of the
calls around the cache that are decided on the host."""

import ctypes
import os
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import rope as OR
from oracle import verify as OV
from paged_kv_cache_append_gb300 import build, nk


# ---------------------------------------------------------------- rotation

@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("rd", [0, 16, 48, 64])
def test_rotation_is_the_pair_matrix(pairs, rd):
    rng = np.random.default_rng(rd + pairs)
    x, cs = rng.standard_normal((3, 2, 64)), OR.table(50, rd)
    pos = np.array([0, 7, 49])
    y, _ = OR.norm_rotate(x, cs, pos, rd, pairs)
    for n in range(3):
        R = np.eye(64)
        for i in range(rd // 2):
            a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rd // 2)
            c, s = float(cs[pos[n], i]), float(cs[pos[n], rd // 2 + i])
            R[a, a], R[a, b], R[b, a], R[b, b] = c, -s, s, c
        np.testing.assert_allclose(y[n], x[n] @ R.T, rtol=0, atol=1e-13)


def test_rotation_closed_forms_and_norm():
    x = np.random.default_rng(0).standard_normal((2, 3, 64))
    cs = np.zeros((2, 32), np.float32)
    cs[0, :16], cs[1, :16] = 1.0, -1.0           # angle 0, angle pi
    y, _ = OR.norm_rotate(x, cs, np.array([0, 1]), 32, False)
    np.testing.assert_array_equal(y[0], x[0])
    np.testing.assert_array_equal(y[1, :, :32], -x[1, :, :32])
    np.testing.assert_array_equal(y[1, :, 32:], x[1, :, 32:])
    z, _ = OR.norm_rotate(x, cs, np.array([0, 0]), 32, False, weight=np.ones(64), eps=0.0)
    np.testing.assert_allclose(np.mean(z * z, axis=-1), 1.0, rtol=1e-13)
    z1, _ = OR.norm_rotate(x, cs, np.array([0, 0]), 32, False, weight=np.zeros(64), eps=0.0, offset=1.0)
    np.testing.assert_allclose(z1, z, rtol=1e-15)


# ---------------------------------------------------------------- verification

def _exact(p, q, x, u, kb):
    """The definition in rationals; every input an exact binary fraction."""
    K, V = len(x), p.shape[1]
    F = lambda v: Fraction(float(v))  # noqa: E731
    n = 0
    while n < kb and F(u[n]) * (F(q[n, x[n]]) if q is not None else 1) < F(p[n, x[n]]):
        n += 1
    d = [F(v) for v in p[n]]
    if n < kb:
        d = [max(a - (F(q[n, j]) if q is not None else int(j == x[n])), Fraction(0)) for j, a in enumerate(d)]
        if sum(d) == 0:
            d = [F(v) for v in p[n]]
    total, s = sum(d), Fraction(0)
    for j, w in enumerate(d):
        s += w
        if s > F(u[K]) * total:
            return n, list(x[:n]) + [j] + [-1] * (K - n)
    raise AssertionError("no token")


def _dyadic_rows(rng, rows, V, bits=12):
    """Probabilities that are multiples of 2^-bits and sum to 1."""
    cuts = np.sort(rng.integers(0, 2 ** bits + 1, (rows, V - 1)), axis=1)
    full = np.concatenate([np.zeros((rows, 1), int), cuts, np.full((rows, 1), 2 ** bits)], axis=1)
    return (np.diff(full, axis=1) / 2 ** bits).astype(np.float32)


@pytest.mark.parametrize("seed", range(20))
@pytest.mark.parametrize("draft", [True, False])
def test_verification_against_rationals(seed, draft):
    rng = np.random.default_rng(seed)
    K, V = int(rng.integers(0, 5)), int(rng.integers(1, 9))
    p, q = _dyadic_rows(rng, K + 1, V), _dyadic_rows(rng, K, V) if draft else None
    x = rng.integers(0, V, K).tolist()
    u = (rng.integers(0, 64, K + 1) / 64).astype(np.float32)
    kb = int(rng.integers(0, K + 1))
    assert OV.verify(p, q, x, u, kb) == _exact(p, q, x, u, kb)


def test_emitted_token_has_the_targets_distribution():
    """The sum over drafts and random numbers of the first emitted token is p
    itself: drafts drawn from q (each token as often as q says), u on a grid."""
    p = np.array([[4, 1, 2, 1], [2, 2, 2, 2]], np.float32) / 8
    q = np.array([[1, 3, 2, 2]], np.float32) / 8
    hits = np.zeros(4)
    grid = 24
    for x, times in enumerate((1, 3, 2, 2)):
        for i in range(grid):
            for j in range(grid):
                _, t = OV.verify(p, q, [x], [i / grid, (j + 0.5) / grid], 1)
                hits[t[0]] += times
    np.testing.assert_allclose(hits / hits.sum(), p[0], atol=1 / grid)


# ---------------------------------------------------------------- refusals (host)

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nk.LIB_PATH):
        build.build()
    return nk.load()


def _rope(**kw):
    d = dict(cos_sin=64, positions=10, rotary_dim=32, layout=0, eps=1e-6, weight_offset=0.0, reserved=0,
             q_weight=None, k_weight=None)
    d.update(kw)
    return nk.RopeDesc(*[d[n] for n, _ in nk.RopeDesc._fields_])


def _norm_rope(lib, rope=None, D=64, q=(64, 256, 64), Hq=4, k=(64, 128, 64), H=2, pos=64, N=3, qo=(64, 256, 64),
               ko=(64, 128, 64)):
    ref = lambda t: ctypes.byref(nk.Rows(*t)) if t else None  # noqa: E731
    return lib.nk_qk_norm_rope(ctypes.byref(rope or _rope()), D, ref(q), Hq, ref(k), H, pos, N, ref(qo), ref(ko), None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=96), -4), (dict(rope=_rope(rotary_dim=40)), -4), (dict(rope=_rope(rotary_dim=80)), -4),
    (dict(rope=_rope(rotary_dim=-16)), -4), (dict(rope=_rope(layout=2)), -1), (dict(rope=_rope(positions=0)), -2),
    (dict(rope=_rope(cos_sin=None)), -1), (dict(rope=_rope(cos_sin=68)), -5), (dict(rope=_rope(q_weight=8)), -5),
    (dict(rope=_rope(eps=-1.0)), -1), (dict(rope=_rope(eps=float("nan"))), -1),
    (dict(rope=_rope(weight_offset=float("inf"))), -1), (dict(q=None), -1), (dict(qo=None), -1), (dict(pos=None), -1),
    (dict(q=None, qo=None, k=None, ko=None), -1), (dict(N=0), -2), (dict(Hq=0), -2), (dict(H=-1), -2),
    (dict(q=(72, 256, 64)), -5), (dict(q=(64, 260, 64)), -5), (dict(ko=(64, 128, 60)), -5), (dict(q=(None, 8, 8)), -1),
    (dict(N=1 << 30, Hq=4), -2), (dict(qo=(64, 0, 64)), -2), (dict(qo=(64, 256, 0)), -2), (dict(qo=(64, 192, 64)), -2),
    (dict(ko=(64, 64, 128)), -2), (dict(ko=(64, 56, 1 << 40)), -2), (dict(ko=(64, -120, 64)), -2)])
def test_norm_rope_refusals(lib, kw, code):
    assert _norm_rope(lib, **kw) == code
    assert nk.load().nk_last_error()


def _verify(lib, target=64, ts=100, draft=64, ds=100, tokens=64, B=2, K=3, V=100, u=64, fr=None, acc=64, out=64,
            fro=None):
    return lib.nk_verify_drafts(target, ts, draft, ds, tokens, None, u, fr, B, K, V, acc, out, fro, None)


@pytest.mark.parametrize("kw,code", [
    (dict(target=None), -1), (dict(u=None), -1), (dict(acc=None), -1), (dict(out=None), -1), (dict(tokens=None), -1),
    (dict(fr=64), -1), (dict(fro=64), -1), (dict(B=0), -2), (dict(K=-1), -2), (dict(K=1025), -2), (dict(V=0), -2),
    (dict(V=(1 << 24) + 1, ts=1 << 25, ds=1 << 25), -2), (dict(ts=99), -2), (dict(ds=99), -2)])
def test_verify_refusals(lib, kw, code):
    assert _verify(lib, **kw) == code


def test_pool_calls_refuse_null(lib):
    n = ctypes.c_size_t()
    assert lib.nk_shared_decode_workspace_bytes(None, 1, 1, 8, ctypes.byref(n)) == -1
    assert lib.nk_paged_shared_decode_attention(None, 8, None, 0, None, None, None, None, 1, 1, 1.0, None, None, -1,
                                                None, 0, None) == -1
    assert lib.nk_paged_kv_append_rope(None, 0, None, None, None, None, None, None, None, None, 0, None, 1, 1,
                                       None) == -1


def test_python_wrappers_refuse_cpu_tensors(lib):
    with pytest.raises(ValueError):
        nk.Rope(torch.zeros((4, 32)), 32)
    with pytest.raises(ValueError):
        nk.verify_drafts(torch.zeros((1, 2, 5)), torch.zeros((1, 1), dtype=torch.int32), torch.zeros((1, 2)))


class Fake:
    """A tensor as far as the argument checks look: shape, strides, type, device, address."""

    def __init__(self, *shape, stride=None, dtype=torch.bfloat16, device=0, ptr=64):
        step, st = 1, []
        for n in reversed(shape):
            st.append(step)
            step *= n
        self.shape, self.dtype = torch.Size(shape), dtype
        self._stride, self._device, self._ptr = stride or tuple(reversed(st)), device, ptr

    def stride(self):
        return self._stride

    def get_device(self):
        return self._device

    def data_ptr(self):
        return self._ptr


def _args_norm(**kw):
    d = dict(q=Fake(3, 4, 64), k=Fake(3, 2, 64), pos=Fake(3, dtype=torch.int32), qo=Fake(3, 4, 64), ko=Fake(3, 2, 64),
             rope=_rope(layout=9), hd=0)
    d.update(kw)
    return nk._args().norm_rope(d["q"], d["k"], d["pos"], d["qo"], d["ko"], ctypes.addressof(d["rope"]), d["hd"], 0, 0)


I32, F32 = torch.int32, torch.float32


@pytest.mark.parametrize("bad", [
    dict(q=Fake(3, 4, 64, dtype=F32)), dict(q=Fake(3, 4, 64, device=1)), dict(q=Fake(3, 4, 64, device=-1)),
    dict(q=Fake(4, 64)), dict(q=Fake(3, 4, 64, stride=(256, 64, 2))), dict(k=Fake(2, 2, 64)), dict(k=Fake(3, 2, 128)),
    dict(qo=Fake(3, 5, 64)), dict(ko=Fake(3, 2, 64, dtype=F32)), dict(pos=Fake(3)), dict(pos=Fake(4, dtype=I32)),
    dict(pos=Fake(3, dtype=I32, stride=(2,))), dict(hd=128), dict(q=Fake(1, 2, 3, 4, 64)),
    dict(q=Fake(2, 3, 4, 64, stride=(1000, 256, 64, 1)), k=Fake(2, 3, 2, 64))])
def test_argument_checks_norm_rope(lib, bad):
    assert _args_norm() == -1                       # good arguments reach the library, which refuses the layout
    with pytest.raises(ValueError):
        _args_norm(**bad)


def test_argument_checks_sizes_of_one_and_rows_apart(lib):
    """Strides of dimensions of size 1 say nothing; [B, 1] tokens may be any stride apart."""
    odd = Fake(1, 1, 64, stride=(7, 3, 1))
    assert _args_norm(q=odd, qo=odd, k=odd, ko=odd, pos=Fake(1, dtype=I32, stride=(5,))) == -1
    apart = dict(q=Fake(2, 1, 4, 64, stride=(1000, 3, 64, 1)), qo=Fake(2, 1, 4, 64), k=Fake(2, 1, 2, 64),
                 ko=Fake(2, 1, 2, 64), pos=Fake(2, 1, dtype=I32))
    assert _args_norm(**apart) == -1


def _args_verify(**kw):
    d = dict(p=Fake(2, 3, 10, dtype=F32), q=Fake(2, 2, 10, dtype=F32), x=Fake(2, 2, dtype=I32), dl=None,
             u=Fake(2, 3, dtype=F32), f=None, acc=Fake(2, dtype=I32, ptr=0), out=Fake(2, 3, dtype=I32), after=None)
    d.update(kw)
    return nk._args().verify(d["p"], d["q"], d["x"], d["dl"], d["u"], d["f"], d["acc"], d["out"], d["after"], 0, 0)


@pytest.mark.parametrize("bad", [
    dict(p=Fake(2, 3, 10)), dict(p=Fake(6, 10, dtype=F32)), dict(p=Fake(2, 0, 10, dtype=F32)),
    dict(p=Fake(2, 3, 10, dtype=F32, stride=(30, 9, 1))), dict(p=Fake(2, 3, 10, dtype=F32, stride=(40, 12, 1))),
    dict(q=Fake(2, 3, 10, dtype=F32)), dict(q=Fake(2, 2, 9, dtype=F32)), dict(x=Fake(2, 2, dtype=torch.int64)),
    dict(x=Fake(2, 3, dtype=I32)), dict(u=Fake(2, 2, dtype=F32)), dict(dl=Fake(3, dtype=I32)),
    dict(f=Fake(2, dtype=F32), after=Fake(2, dtype=I32))])
def test_argument_checks_verify(lib, bad):
    assert _args_verify() == -1                     # reaches the library, which refuses the NULL output
    assert _args_verify(p=Fake(2, 3, 10, dtype=F32, stride=(36, 12, 1))) == -1
    with pytest.raises(ValueError):
        _args_verify(**bad)


def _args_append(**kw):
    d = dict(layer=0, t=Fake(3, 5, dtype=I32), r=Fake(2, dtype=I32), w=Fake(2, dtype=I32), k=Fake(2, 4, 2, 64),
             v=Fake(2, 4, 2, 64), q=Fake(2, 4, 8, 64), qo=Fake(2, 4, 8, 64), c=None, hd=64)
    d.update(kw)
    return nk._args().append_rope(0, 2, 64, 3, 5, d["layer"], d["t"], d["r"], d["w"], d["k"], d["v"], d["q"], d["qo"],
                                  d["c"], ctypes.addressof(_rope()), d["hd"], 0, 0)


@pytest.mark.parametrize("bad", [
    dict(t=Fake(2, 5, dtype=I32)), dict(r=Fake(3, dtype=I32)), dict(w=Fake(2)), dict(k=Fake(2, 4, 3, 64)),
    dict(k=Fake(8, 2, 64)), dict(v=Fake(2, 3, 2, 64)), dict(q=Fake(2, 5, 8, 64)), dict(q=Fake(2, 4, 8, 128)),
    dict(qo=Fake(2, 4, 7, 64)), dict(q=None), dict(c=Fake(1, dtype=I32)), dict(hd=128)])
def test_argument_checks_append_rope(lib, bad):
    assert _args_append() == -1                     # reaches the library, which refuses the NULL pool
    assert _args_append(q=None, qo=None) == -1
    with pytest.raises(ValueError):
        _args_append(**bad)


def _args_shared(**kw):
    d = dict(q=Fake(2, 1, 8, 64), t=Fake(3, 5, dtype=I32), r=Fake(2, dtype=I32), f=Fake(2, dtype=I32),
             s=Fake(1, dtype=I32), o=Fake(2, 1, 8, 64), l=Fake(2, 1, 8, dtype=F32))
    d.update(kw)
    return nk._args().shared_decode(0, 64, 3, 5, 0, d["q"], d["t"], d["r"], d["f"], d["s"], 0.1, d["o"], d["l"], -1, 64,
                                    64, 0, 0)


@pytest.mark.parametrize("bad", [
    dict(q=Fake(2, 1, 8, 128)), dict(q=Fake(2, 8, 64)), dict(q=Fake(2, 1, 8, 64, stride=(1024, 512, 64, 1))),
    dict(t=Fake(3, 6, dtype=I32)), dict(r=Fake(1, dtype=I32)), dict(f=Fake(2, dtype=F32)), dict(s=Fake(2, dtype=I32)),
    dict(s=Fake(1)), dict(o=Fake(2, 1, 4, 64)), dict(l=Fake(2, 1, 8))])
def test_argument_checks_shared_decode(lib, bad):
    assert _args_shared() == -1                     # reaches the library, which refuses the NULL pool
    with pytest.raises(ValueError):
        _args_shared(**bad)
