"""GPU parity of the differential attentions against the oracle in 64 bits.

Tolerances, derived: every term p v of a map's sum is off by at most c of its
size, a = sum p |v| over both maps, and oracle.differential.tolerance carries
that through the norm to the output and its one rounding to bf16 (2^-8).
 * weights: f16 2^-11 (BF16 pages in the decode: two terms, 2^-16);  values: f16
   products of INT8-G64 and FP8-row, 2^-11 (the tensor-core form keeps FP8-row
   values exactly, BF16 ones to 2^-19 of their strip's largest);  so c0 = 2^-10;
 * the decode takes q exactly (f16 or bf16); the prefill over FP8-row keys of
   head_dim 128 takes q in two E4M3 terms, each element to 2^-17 of the largest:
   with |q| <= 4.5, sum |k| <= 128 and a scale of 1/11 a score is off by at most
   2^-17 * 4.5 * 128 / 11 = 4e-4, a weight by as much and the sum of the weights
   too: 8e-4 more;
 * fp32 sums of D products, the exponential (2 ulp) and the reference's fold
   (|s| 2^-24): below 1e-4 with |s| < 30 and D <= 128.
So c = 2^-10 + 1e-4 (decode), the same + 8e-4 (prefill); lse within 1e-3.
"""

import math

import numpy as np
import pytest
import torch

from oracle import differential as OD
from oracle import formats as OF
from oracle.store import PoolImage
from paged_kv_cache_append_gb300 import nk
from paged_kv_cache_append_gb300.workloads import bf16_to_bits

pytestmark = pytest.mark.gpu
DEV = "cuda"
PROFILES = ["bf16", "int8_g64", "fp8_row", "nvfp4_g16", "k8v4"]
EPS, OUT_SCALE = 1e-5, 0.2


def normal(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV) if dtype is None else torch.tensor(a, dtype=dtype, device=DEV)


def f64(t):
    return OF.bf16_bits_to_f64(bf16_to_bits(t))


class Batch:
    """A pool of rows with F tokens each, filled on the GPU and in the oracle; stale bytes are NaN patterns."""

    def __init__(self, profile, D, H, G, T, F, order="page_major", seed=0, C=None, norm=True, per_token=False, slack=1,
                 chunk=None):
        B = len(F)
        C = C or B
        self.profile, self.B, self.T, self.H, self.Hq, self.D, self.G = profile, B, T, H, H * G, D, G
        self.F = np.asarray(F, np.int32)
        self.chunk = None if chunk is None else np.asarray(chunk, np.int32)   # prefill: F = prefix + chunk
        L = max(1, -(-max(F) // 64)) + slack
        M = max(L, C * L)
        rng = np.random.default_rng(seed + D + 7 * G)
        self.tables = rng.permutation(M).astype(np.int32)[:C * L].reshape(C, L)
        self.rows = rng.permutation(C)[:B].astype(np.int32)
        self.gpu = nk.Pool(profile, 1, H, D, 64 * L, C, M, order=order)
        self.img = PoolImage(profile, 1, H, D, M, order=order)
        for p in self.gpu.planes[0]:
            p.fill_(0xFF if profile in ("bf16", "fp8_row", "k8v4") else 0x7F)
        self.fill(1000 + seed, 2000 + seed)
        self.q = normal((B, T, self.Hq, D), 5 + seed)
        self.scale = 1 / math.sqrt(D)
        g = torch.Generator().manual_seed(70 + seed)
        self.lam = 0.1 + 0.7 * torch.rand((B, T, self.Hq // 2) if per_token else (self.Hq // 2,), generator=g)
        self.w = (1 + 0.2 * torch.randn(2 * D, generator=g)).to(torch.bfloat16) if norm else None
        self.diff = nk.Diff(self.lam.to(DEV), None if self.w is None else self.w.to(DEV), EPS, OUT_SCALE)
        self.d = dict(tables=dev(self.tables), rows=dev(self.rows), F=dev(self.F), q=self.q.to(DEV))
        if chunk is not None:
            self.d["prefix"], self.d["chunk"] = dev(self.F - self.chunk), dev(self.chunk)

    def fill(self, k_seed, v_seed, mul=1.0):
        """Keys, and values times mul, of every row, from its first token on."""
        for b in range(self.B):
            n = int(self.F[b])
            if n:
                k = normal((1, n, self.H, self.D), k_seed + b)
                v = (normal((1, n, self.H, self.D), v_seed + b).float() * mul).to(torch.bfloat16)
                row = int(self.rows[b])
                self.gpu.append(0, dev(self.tables), dev([row], torch.int32), dev([0], torch.int32), k.to(DEV), v.to(DEV))
                self.img.append(0, self.tables, np.array([row]), np.array([0]), bf16_to_bits(k), bf16_to_bits(v))

    def run(self, **kw):
        d = self.d
        if self.chunk is None:
            return self.gpu.diff_decode(0, d["q"], d["tables"], d["rows"], d["F"], self.scale, self.diff, **kw)
        return self.gpu.diff_prefill(0, d["q"], d["tables"], d["rows"], d["prefix"], d["chunk"], self.scale, self.diff,
                                     **kw)

    def reference(self):
        """Per row: (out, lse, o, a), of the chunk's tokens in a prefill."""
        lam = np.broadcast_to(self.lam.double().numpy(), (self.B, self.T, self.Hq // 2))
        res = []
        for b in range(self.B):
            n = self.T if self.chunk is None else int(self.chunk[b])
            F = int(self.F[b])
            K, V = self.img.gather(0, self.tables[self.rows[b]], F)
            res.append(OD.attend(f64(self.q[b, :n]), K, V, F - n, self.scale, lam[b, :n],
                                 None if self.w is None else self.w.double().numpy(), EPS, OUT_SCALE))
        return res

    def check(self, out, lse, c=None):
        torch.cuda.synchronize()
        if c is None:
            c = 2.0 ** -10 + 1e-4
            if self.chunk is not None:
                c = 2.0 ** -10 + 9e-4
        w = None if self.w is None else self.w.double().numpy()
        for b, (o, l, raw, a) in enumerate(self.reference()):
            n = o.shape[0]
            got, gl = out[b, :n].double().cpu().numpy(), lse[b, :n].double().cpu().numpy()
            assert np.all(np.isfinite(got))
            seen = np.isfinite(l)
            assert np.array_equal(np.isfinite(gl), seen) and np.all(gl[~seen] == -np.inf)
            assert not seen.any() or np.abs(gl[seen] - l[seen]).max() <= 1e-3, np.abs(gl[seen] - l[seen]).max()
            empty = ~seen[:, ::2]
            assert not got[empty].any()
            if seen.any():
                some = ~empty
                tol = OD.tolerance(o[some], raw[some], a[some], w, EPS, OUT_SCALE, c, 2.0 ** -8)
                excess = np.abs(got[some] - o[some]) - tol
                assert excess.max() <= 0, (b, excess.max(), tol[excess > 0].max())


# ------------------------------------------------------------------ decode

SHAPES = [(2, 1, 1), (2, 4, 1), (4, 2, 3), (2, 3, 5), (2, 8, 2), (2, 5, 7), (2, 16, 4)]


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G,T", SHAPES)
def test_decode_shapes(profile, D, H, G, T):
    """1, 4, 6, 15, 16, 35 and 64 query rows: packed maps, one and two column tiles, one to four blocks of rows."""
    b = Batch(profile, D, H, G, T, [T, 64 + T, 200, 129])
    b.check(*b.run())


@pytest.mark.parametrize("profile", PROFILES)
def test_decode_lengths(profile):
    """Lengths around pages; rows that see nothing, or only from a later token on."""
    b = Batch(profile, 64, 2, 4, 3, [0, 1, 2, 3, 63, 64, 65, 128])
    b.check(*b.run())


@pytest.mark.parametrize("profile,D", [("bf16", 128), ("fp8_row", 64), ("k8v4", 128)])
def test_decode_long_and_uneven(profile, D):
    """One long row among short ones: the split plan, and partials of rows without a page in a split."""
    b = Batch(profile, D, 2, 2, 2, [3001, 5, 64, 1900])
    b.check(*b.run())


@pytest.mark.parametrize("profile", PROFILES)
def test_decode_one_row_of_many_splits(profile):
    b = Batch(profile, 64, 2, 1, 1, [9000])
    b.check(*b.run())


@pytest.mark.parametrize("kw", [dict(order="head_major"), dict(C=7), dict(norm=False), dict(per_token=True)])
def test_decode_forms(kw):
    for profile in ("bf16", "nvfp4_g16"):
        b = Batch(profile, 128, 4, 2, 2, [100, 300, 2], **kw)
        b.check(*b.run())


def test_decode_negative_and_zero_scale():
    for scale in (-0.11, 0.0):
        for profile in ("bf16", "int8_g64"):
            b = Batch(profile, 64, 2, 2, 2, [100, 70])
            b.scale = scale
            b.check(*b.run())


def test_decode_maps_of_very_different_queries():
    """Map 1's queries 2^-30 of map 2's: each map has its own f16 scale."""
    for profile in ("fp8_row", "nvfp4_g16"):
        b = Batch(profile, 64, 2, 2, 2, [100, 170])
        b.q[:, :, ::2] *= 2.0 ** -30
        b.d["q"] = b.q.to(DEV)
        b.check(*b.run())


def test_the_same_bits_on_every_call_and_a_workspace_of_nan():
    for profile, F in (("k8v4", [4000, 900, 64]), ("bf16", [700, 1, 0])):
        b = Batch(profile, 128, 2, 4, 1, F)
        want = [x.clone() for x in b.run()]
        ws = b.gpu.diff_decode_workspace(b.B, b.T, b.Hq)
        for _ in range(3):
            ws.fill_(0xFF)
            got = b.run(workspace=ws)
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_a_nan_reaches_the_rows_that_see_it_and_no_other():
    """In a key: the head's outputs; the other rows and pairs are as without it."""
    b = Batch("bf16", 64, 4, 1, 1, [300, 200])
    want = [x.clone() for x in b.run()]
    torch.cuda.synchronize()
    page, at = int(b.tables[b.rows[0], 2]), 17
    b.gpu.planes[0][0].view(torch.bfloat16).view(-1, 4, 64, 64)[page, 3, at, 5] = float("nan")   # KV head 3: pair 1
    out, lse = b.run()
    torch.cuda.synchronize()
    assert torch.isnan(out[0, 0, 1]).all() and torch.isnan(lse[0, 0, 3])
    assert torch.equal(out[0, 0, 0], want[0][0, 0, 0]) and torch.equal(out[1], want[0][1])
    assert torch.equal(lse[0, 0, :3], want[1][0, 0, :3]) and torch.equal(lse[1], want[1][1])


@pytest.mark.parametrize("mul", [2.0 ** -14, 2.0 ** 20])
@pytest.mark.parametrize("chunk", [None, [40, 70]])
def test_values_of_any_magnitude(mul, chunk):
    """Values far below and above f16's range, through the norm."""
    for profile in PROFILES:
        if mul < 1 and profile in ("nvfp4_g16", "k8v4"):
            continue   # below the smallest E4M3 scale: the codec stores zeros
        b = Batch(profile, 64, 2, 2, 1 if chunk is None else 70, [130, 70], chunk=chunk)
        b.fill(1000, 2000, mul)
        b.check(*b.run())


def test_bad_lengths_rows_and_pages_are_reported():
    b = Batch("fp8_row", 64, 2, 2, 1, [100, 100, 100])
    nk.nk_status_read(True)
    want = [x.clone() for x in b.run()]
    torch.cuda.synchronize()
    b.d["F"] = dev([100, 64 * b.tables.shape[1] + 1, 100], torch.int32)
    b.d["rows"] = dev([int(b.rows[0]), int(b.rows[1]), 3], torch.int32)
    out, lse = b.run()
    assert nk.nk_status_read(True) == nk.STATUS_FRONTIER
    assert torch.equal(out[0], want[0][0]) and not out[1:].any() and (lse[1:] == -math.inf).all()
    b = Batch("fp8_row", 64, 2, 2, 1, [100, 100])
    b.tables[b.rows[1], 1] = b.gpu.M
    b.d["tables"] = dev(b.tables)
    b.run()
    assert nk.nk_status_read(True) == nk.STATUS_PAGE_RANGE


# ------------------------------------------------------------------ prefill

@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", [(2, 1), (4, 2), (2, 5), (2, 8), (2, 48)])
def test_prefill_shapes(profile, D, H, G):
    """Whole and partial tiles of query rows, groups that do not divide 128, ragged chunks, a chunk of one, of none."""
    T = 140 if G == 1 else 70 if G < 8 else 37 if G == 8 else 5
    b = Batch(profile, D, H, G, T, [T, 100 + T // 2, 65, 30, 77], chunk=[T, T // 2, 1, 0, min(T, 13)])
    out = torch.full((b.B, T, b.Hq // 2, 2 * D), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((b.B, T, b.Hq), 9.0, device=DEV)
    b.check(*b.run(out=out, lse=lse))
    for i, n in enumerate(b.chunk):   # rows behind the chunk are as they were
        assert (out[i, n:] == 9).all() and (lse[i, n:] == 9).all()


@pytest.mark.parametrize("profile", PROFILES)
def test_prefill_long_prefix(profile):
    """Few query rows over many pages: ranges of pages joined at the end."""
    b = Batch(profile, 64, 2, 2, 9, [2000, 1203], chunk=[9, 3])
    b.check(*b.run())


@pytest.mark.parametrize("kw", [dict(order="head_major"), dict(C=6), dict(norm=False), dict(per_token=True)])
def test_prefill_forms(kw):
    for profile in ("bf16", "k8v4"):
        b = Batch(profile, 128, 4, 2, 66, [66, 300], chunk=[66, 40], **kw)
        b.check(*b.run())


def test_prefill_negative_and_zero_scale():
    for scale in (-0.11, 0.0):
        for profile in ("bf16", "int8_g64"):
            b = Batch(profile, 64, 2, 2, 40, [100, 40], chunk=[40, 40])
            b.scale = scale
            b.check(*b.run())


def test_prefill_same_bits_over_a_workspace_of_nan():
    for profile in ("bf16", "fp8_row"):
        b = Batch(profile, 128, 2, 4, 50, [900, 50], chunk=[50, 20])
        want = [x.clone() for x in b.run()]
        ws = b.gpu.diff_prefill_workspace(b.B, b.T, b.Hq)
        ws.fill_(0xFF)
        got = b.run(workspace=ws)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_prefill_agrees_with_the_decode():
    """The last token of a chunk is a decode of one token over the same pages."""
    for profile in PROFILES:
        b = Batch(profile, 128, 2, 2, 5, [205, 133], chunk=[5, 5])
        out, lse = b.run()
        o, l = b.gpu.diff_decode(0, b.d["q"][:, -1:].contiguous(), b.d["tables"], b.d["rows"], b.d["F"], b.scale, b.diff)
        torch.cuda.synchronize()
        assert (lse[:, -1:] - l).abs().max() <= 2e-3 and (out[:, -1:].float() - o.float()).abs().max() <= 0.05


def test_prefill_bad_lengths_are_reported():
    b = Batch("bf16", 64, 2, 2, 8, [100, 100], chunk=[8, 8])
    nk.nk_status_read(True)
    want = [x.clone() for x in b.run()]
    torch.cuda.synchronize()
    for bad in (dict(chunk=[8, 9]), dict(chunk=[8, -1]), dict(prefix=[92, -1]), dict(prefix=[92, 64 * b.tables.shape[1]]),
                dict(rows=[int(b.rows[0]), 2])):
        keep = dict(b.d)
        for k, v in bad.items():
            b.d[k] = dev(v, torch.int32)
        out, lse = b.run()
        assert nk.nk_status_read(True) == nk.STATUS_FRONTIER
        assert torch.equal(out[0], want[0][0]) and not out[1].any() and (lse[1] == -math.inf).all()
        b.d = keep


# ------------------------------------------------------------------ refusals and use

def test_refused_pools_and_arguments():
    p = nk.Pool("fp8_row", 1, 2, 256, 128, 2, 4)
    for f in (p.diff_decode_workspace, p.diff_prefill_workspace):
        with pytest.raises(nk.NkError, match="head_dim"):
            f(1, 1, 4)
    p = nk.Pool("fp8_row", 1, 3, 64, 128, 2, 4)
    with pytest.raises(nk.NkError, match="even"):
        p.diff_decode_workspace(1, 1, 6)
    b = Batch("fp8_row", 64, 2, 2, 1, [100, 100])
    for f in (b.gpu.diff_decode_workspace, b.gpu.diff_prefill_workspace):
        for args in ((0, 1, 4), (3, 1, 4), (1, 0, 4), (1, 1, 3), (1, 1, 0)):
            with pytest.raises(nk.NkError):
                f(*args)
    with pytest.raises(nk.NkError, match="64"):
        b.gpu.diff_decode_workspace(1, 33, 4)
    with pytest.raises(nk.NkError, match="64"):
        b.gpu.diff_prefill_workspace(1, 1, 130)
    with pytest.raises(nk.NkError, match="workspace"):
        b.run(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    for eps, scale in ((0.0, 1.0), (float("nan"), 1.0), (1e-5, float("inf"))):
        b.diff = nk.Diff(b.lam.to(DEV), b.w.to(DEV), eps, scale)
        with pytest.raises(nk.NkError):
            b.run()
    for lam, w in ((b.lam, None), (b.lam.to(DEV), b.w), (torch.empty((0, 2), device=DEV), None),
                   (b.lam.to(DEV).double(), None)):
        with pytest.raises(ValueError):
            nk.Diff(lam, w)


def test_lambda_from_learned_vectors():
    g = torch.Generator().manual_seed(1)
    v = [(0.2 * torch.randn((6, 64), generator=g)).to(DEV) for _ in range(4)]
    d = nk.Diff.from_vectors(*v, lambda_init=0.3, heads=6)
    want = (v[0] * v[1]).double().sum(-1).exp() - (v[2] * v[3]).double().sum(-1).exp() + 0.3
    assert torch.allclose(d.lam.double(), want, rtol=1e-5, atol=1e-6) and abs(d.desc.out_scale - 0.7) < 1e-6
    d = nk.Diff.from_vectors(*[x[0] for x in v], lambda_init=0.3, heads=6)
    assert torch.equal(d.lam, d.lam[:1].expand(6))


def test_two_streams_with_workspaces_of_their_own():
    batches = [Batch("k8v4", 128, 2, 4, 1, [3000, 2900, 64], seed=s) for s in (0, 50)]
    wants = [[x.clone() for x in b.run()] for b in batches]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        got = [b.run(stream=s) for b, s in zip(batches, (None, side))]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for g, w in zip(got, wants) for x, y in zip(g, w))


@pytest.mark.parametrize("profile", ["int8_g64", "k8v4"])
def test_a_captured_layer_grows_appends_attends_and_norms(profile):
    """Pages from the lengths, the rotated append, the attention, the projection's stand-in and the block's norms, one
    graph replayed over page edges, against the oracle of the final step."""
    D, H, G, B, T, S = 64, 2, 2, 3, 2, 512
    Hq, dim = H * G, H * G * D
    pool = nk.Pool(profile, 1, H, D, S, B, 3 * S // 64)
    tables, mapped, free, n = pool.free_pages()
    rows, done = dev([2, 0, 1], torch.int32), dev([0, 61, 120], torch.int32)
    g = torch.Generator().manual_seed(3)
    cos = torch.randn((S, D), generator=g).to(DEV)
    rope = nk.Rope(cos, D, q_weight=normal((D,), 1).to(DEV), k_weight=normal((D,), 2).to(DEV))
    lam = 0.1 + 0.7 * torch.rand(Hq // 2, generator=g)
    diff = nk.Diff(lam.to(DEV), normal((2 * D,), 4).to(DEV), EPS, OUT_SCALE)
    block = nk.ResidualNorm(normal((dim,), 5).to(DEV), post_weight=normal((dim,), 6).to(DEV), scale=0.5)
    x = [torch.zeros((B, T, h, D), dtype=torch.bfloat16, device=DEV) for h in (Hq, H, H)]
    res = normal((B, T, dim), 7).to(DEV)
    ws = pool.diff_decode_workspace(B, T, Hq)
    img = PoolImage(profile, 1, H, D, pool.M)
    state = {}

    def step():
        f, pos, slots = pool.grow(tables, rows, done, mapped, free, n, T)
        q = pool.append_rope(0, tables, rows, done, x[1], x[2], rope, q=x[0])
        out, lse = pool.diff_decode(0, q, tables, rows, f, D ** -0.5, diff, workspace=ws)
        state.update(f=f, slots=slots, q=q, out=out, lse=lse)
        state["y"] = nk.residual_norm(out.view(B, T, dim), res, block)
        done.copy_(f)

    # rows 1 and 2 begin with tokens of an earlier call
    pool.grow(tables, rows, torch.zeros_like(done), mapped, free, n, 120, counts=done)
    first = [normal((B, 120, H, D), 20 + i).to(DEV) for i in range(2)]
    pool.append(0, tables, rows, torch.zeros_like(done), *first, counts=done)
    for i in range(3):
        x[i].copy_(normal(tuple(x[i].shape), 30 + i))
    nk.nk_status_read(True)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(40):
        for i in range(3):
            x[i].copy_(normal(tuple(x[i].shape), 100 + 3 * r + i))
        graph.replay()
    torch.cuda.synchronize()
    assert nk.nk_status_read(True) == 0
    F = state["f"].cpu().numpy()
    assert F.tolist() == [82, 143, 202]
    # the pages hold what the append wrote: the oracle reads them as they are
    for i, p in enumerate(pool.planes[0]):
        img.planes[0][i][:] = p.cpu().numpy()
    tab = tables.cpu().numpy()
    w = diff.norm_weight.double().cpu().numpy()
    for b in range(B):
        K, V = img.gather(0, tab[int(rows[b])], int(F[b]))
        o, l, raw, a = OD.attend(f64(state["q"][b].cpu()), K, V, F[b] - T, D ** -0.5,
                                 np.broadcast_to(lam.double().numpy(), (T, Hq // 2)), w, EPS, OUT_SCALE)
        tol = OD.tolerance(o, raw, a, w, EPS, OUT_SCALE, 2.0 ** -10 + 1e-4, 2.0 ** -8)
        assert np.all(np.abs(state["out"][b].double().cpu().numpy() - o) <= tol)
        slots = state["slots"][b].cpu().numpy()
        assert [int(s) for s in slots] == [int(tab[int(rows[b]), p // 64]) * 64 + p % 64 for p in range(F[b] - T, F[b])]
    want = nk.residual_norm(state["out"].view(B, T, dim), res, block)
    assert all(torch.equal(p, q) for p, q in zip(want, state["y"]))
