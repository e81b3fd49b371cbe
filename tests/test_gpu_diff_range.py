"""The differential attentions where their softmax and their values move far.

Tolerances as derived in test_gpu_diff.py: c = 2^-10 + 1e-4 for the weights, the
values and the fp32 steps, and for the scores of E4M3 queries (chunks and decodes
of more than 8 query rows over FP8-row keys of head_dim 128) 2 e more, e = 2^-17
max|q| max sum|k| |scale|.  What a case adds to that stands at the case.
"""

import numpy as np
import pytest
import torch

from paged_kv_cache_append_gb300 import nk
from paged_kv_cache_append_gb300.workloads import bf16_to_bits
from tests.test_gpu_diff import DEV, PROFILES, Batch, dev, f64, normal

pytestmark = pytest.mark.gpu
BASE = 2.0 ** -10 + 1e-4
#: G, T, chunk: decodes of 1, 4, 8, 10 and 64 query rows; a chunk of many tiles to a cluster, one that is cut
FORMS = {"one": (1, 1, None), "packed": (2, 2, None), "eight": (4, 2, None), "ten": (5, 2, None), "tiles": (16, 4, None),
         "chunk": (2, 90, [90, 61]), "cut": (1, 9, [9, 4])}


def e4m3_scores(b, keys):
    """Twice the error of a score whose query is taken in two E4M3 terms."""
    if b.D != 128 or b.profile not in ("fp8_row", "k8v4"):
        return 0.0
    most = float(keys.float().abs().sum(-1).max())
    return 2 * 2.0 ** -17 * float(b.q.float().abs().max()) * most * abs(b.scale)


def set_row(b, r, k, v, at=0):
    """Tokens at .. of row r of the batch, on the GPU and in the oracle; k, v bf16 [n, H, D]."""
    row = int(b.rows[r])
    b.gpu.append(0, dev(b.tables), dev([row], torch.int32), dev([at], torch.int32), k[None].contiguous().to(DEV),
                 v[None].contiguous().to(DEV))
    b.img.append(0, b.tables, np.array([row]), np.array([at]), bf16_to_bits(k[None]), bf16_to_bits(v[None]))


def batch(profile, D, form, F, **kw):
    G, T, chunk = FORMS[form]
    return Batch(profile, D, 2, G, T, F, chunk=chunk, **kw)


def signs(n, seed):
    return torch.where(torch.rand(n, generator=torch.Generator().manual_seed(seed)) < 0.5, -1.0, 1.0)


def direct_queries(b, coef, seed):
    """Queries coef[head] u + noise along one direction u of signs; returns u."""
    u = signs(b.D, seed)
    q = coef[None, None, :, None] * u + 0.25 * normal(tuple(b.q.shape), seed + 1).float()
    b.q = q.to(torch.bfloat16)
    b.d["q"] = b.q.to(DEV)
    return u


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", list(FORMS))
def test_maxima_that_rise_in_steps(profile, D, form):
    """Keys along the queries' direction, larger step by step: a map's largest score rises by up to 10 in base 2 four
    times (more than the 8 that a reference may lag), by less for other heads, and falls for some.  |s| stays below 32."""
    b = batch(profile, D, form, [1500, 700])
    coef = torch.tensor([(1.0, 0.6, -0.8, 0.3, 0.0, 1.0, 0.9)[i % 7] for i in range(b.Hq)])
    beta = 28 / (2 * b.scale * D)   # the last step's score of coef 1: 28
    u = direct_queries(b, beta * coef, 31)
    most = torch.zeros(1, b.D)
    for r, F in enumerate(b.F):
        F = int(F)
        step = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0])[torch.bucketize(torch.arange(F), torch.tensor(
            [70, 64 * 3 + 17 + 16 * r, F // 2, F - 150]), right=True)]
        k = (step[:, None, None] * u + 0.5 * normal((F, b.H, D), 41 + r).float()).to(torch.bfloat16)
        set_row(b, r, k, normal((F, b.H, D), 51 + r))
        most = torch.cat((most, k.flatten(0, 1).float()))
    b.check(*b.run(), c=BASE + e4m3_scores(b, most))
    assert nk.nk_status_read(True) == 0


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", list(FORMS))
def test_values_that_rise_along_a_row(profile, D, form):
    """Values, and with them the pages' value scales, 2^-9 times a normal one first, then 1, then 2^9: what a kernel
    carries for their range changes over results that it has."""
    b = batch(profile, D, form, [1500, 700])
    for r, F in enumerate(b.F):
        F = int(F)
        size = torch.tensor([2.0 ** -9, 1.0, 2.0 ** 9])[torch.bucketize(torch.arange(F), torch.tensor(
            [F // 3, F - 190]), right=True)]
        v = (size[:, None, None] * normal((F, b.H, D), 61 + r).float()).to(torch.bfloat16)
        set_row(b, r, normal((F, b.H, D), 71 + r), v)
    b.check(*b.run(), c=BASE + (8e-4 if e4m3_scores(b, torch.ones(1, D)) else 0.0))
    assert nk.nk_status_read(True) == 0


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form,F", [(f, [1500, 700]) for f in FORMS if f != "chunk"] + [("chunk", [90, 61])]
                         + [(f, [16, 16]) for f in ("packed", "eight", "tiles")])
def test_small_weights_beside_one_that_dominates(profile, D, form, F):
    """The first key takes nearly all of the softmax and its value is zero, so that the output is made of the others'
    weights, about 2^-19 of it and the same for all (one key for all of them), of values of one sign.

    A weight is held to 2^-11 from 2^-20 of the largest on, below it to 2^-31 of the largest: with weights of at least
    2^-21.6, which the case asserts, 2^-9.4 at the worst."""
    b = batch(profile, D, form, F)
    coef = torch.ones(b.Hq)
    beta = 13.2 / (b.scale * D)
    u = direct_queries(b, beta * coef, 81)
    other = 0.25 * signs(D, 83)
    keys = []
    for r, n in enumerate(b.F):
        n = int(n)
        k = other.expand(n, b.H, D).clone()
        k[0] = u
        v = 512 * (1 + 0.3 * normal((n, b.H, D), 91 + r).float())
        v[0] = 0
        keys.append(k)
        set_row(b, r, k.to(torch.bfloat16), v.to(torch.bfloat16))
    for r in range(b.B):   # the weights that the queries give: one key for all but the first
        K, _ = b.img.gather(0, b.tables[b.rows[r]], 2)
        s = b.scale * np.einsum("tjgmd,njmd->ntjgm", f64(b.q[r]).reshape(b.T, b.H // 2, b.G, 2, D),
                                K.reshape(2, b.H // 2, 2, D))
        assert np.all((s[0] - s[1]) / np.log(2) > 15) and np.all((s[0] - s[1]) / np.log(2) < 21.6)
    b.check(*b.run(), c=BASE + 2.0 ** -9.4 + e4m3_scores(b, torch.cat([k.flatten(0, 1) for k in keys])))


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_an_infinite_value_stays_in_its_dim(form, D, bad):
    """Without a norm an infinity or a NaN among BF16 values reaches its own output dim and no other, whatever shares
    its strip of dims."""
    b = batch("bf16", D, form, [300, 200], norm=False)
    want = b.reference()
    page, at, head, d = int(b.tables[b.rows[0], 1]), 17, 1, 21
    b.gpu.planes[0][1].view(torch.bfloat16).view(-1, 2, 64, D)[page, head, at, d] = bad
    out, lse = b.run()
    torch.cuda.synchronize()
    n = want[0][0].shape[0]
    assert not torch.isfinite(out[0, :n, :, head * D + d]).any()
    out[0, :n, :, head * D + d] = torch.from_numpy(want[0][0][:, :, head * D + d]).to(out)
    b.check(out, lse)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** -3, 1.0, 2.0 ** 14, 2.0 ** 40])
def test_a_dim_far_above_its_neighbours(form, D, size):
    """One dim of every 16 holds values up to about `size`, its neighbours 2^-13 of that.

    On the tensor cores a BF16 value is exact from 2^-11 of the largest in its strip of dims on, and within 2^-19 of the
    largest below: 2^-19 of a dim's largest for each of its neighbours, against their own size of 2^-13, is 2^-6 of a
    neighbour at the worst, so an output (no norm) may be off by (1 + lambda) 2^-19 of the largest."""
    b = batch("bf16", D, form, [300, 200], norm=False)
    scale = torch.full((D,), size * 2.0 ** -15)
    scale[3::16] = size * 2.0 ** -2      # normal values stay below 4.5
    most = 0.0
    for r, n in enumerate(b.F):
        v = (normal((int(n), b.H, D), 15 + r).float() * scale).to(torch.bfloat16)
        v[0, :, 3::16] = size * 0.5       # a strip's first page holds its size
        most = max(most, float(v.float().abs().max()))
        set_row(b, r, normal((int(n), b.H, D), 25 + r), v)
    out, lse = b.run()
    torch.cuda.synchronize()
    for r, (o, l, raw, a) in enumerate(b.reference()):
        n = o.shape[0]
        got, s = out[r, :n].double().cpu().numpy(), 0.2
        lam = np.abs(b.lam.double().numpy())[None, :, None]
        tol = s * (BASE * a + (0.0 if FORMS[form][0] * FORMS[form][1] <= 8 and b.chunk is None else
                               (1 + lam) * 2.0 ** -19 * most))
        tol = tol + 2.0 ** -8 * (np.abs(o) + tol)
        assert np.all(np.abs(got - o) <= tol), (r, np.max(np.abs(got - o) - tol))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", ["chunk", "tiles"])
@pytest.mark.parametrize("size", [2.0 ** -90, 2.0 ** -3, 0.25, 1.0, 2.0 ** 14, 2.0 ** 15, 2.0 ** 90])
def test_one_bf16_value_comes_back(D, form, size):
    """A token that sees one key, lambda 0, no norm, a scale of 1: its output is the key's value as the tensor cores
    take it, exact from 2^-11 of the largest of a strip (one in every 8 dims is `size`) on, within 2^-19 of it below."""
    G, T, _ = FORMS[form]
    b = Batch("bf16", D, 2, G, T, [1, 1], chunk=[1, 1] if form == "chunk" else None, norm=False)
    g = torch.Generator().manual_seed(7)
    small = torch.zeros(0)
    for r in range(2):
        v = size * signs(2 * D, r) * 2.0 ** (-24 * torch.rand(2 * D, generator=g))
        v[::8] = size
        v = v.to(torch.bfloat16)
        small = torch.cat((small, v.float()[None])) if r else v.float()[None]
        set_row(b, r, normal((1, 2, D), 5 + r), v.view(1, 2, D))
    b.diff = nk.Diff(torch.zeros(b.Hq // 2, device=DEV), None, 1e-5, 1.0)
    out, _ = b.run()
    torch.cuda.synchronize()
    got = (out[:, 0] if form == "chunk" else out[:, -1]).double().cpu()   # of a decode the last token sees the key
    want = small.double()[:, None].expand_as(got)
    large = want.abs() >= size * 2.0 ** -11
    assert torch.equal(got[large], want[large])
    assert bool(((got - want).abs() <= 2.0 ** -19 * size + 2.0 ** -8 * want.abs())[~large].all())


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("D", [64, 128])
def test_a_chunk_and_the_decode_agree(profile, D):
    """The last tokens of a chunk are a decode of them over the same pages: each within its own tolerance of the
    definition, so within the sum of both of one another."""
    b = Batch(profile, D, 2, 2, 5, [705, 133], chunk=[5, 5])
    out, lse = b.run()
    b.check(out, lse)
    for T in (1, 5):
        one = Batch(profile, D, 2, 2, T, [705, 133])
        one.q = b.q[:, -T:].contiguous()
        one.d["q"] = one.q.to(DEV)
        one.check(*one.run())
