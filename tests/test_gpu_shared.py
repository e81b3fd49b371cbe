"""GPU parity of the shared-prefix attention against the oracle, and of the
serving step that uses it with the rotated append and the draft verification.

Tolerances, derived.  Beyond half a bf16 step of the output (2^-8 of it):
softmax weights and INT8-G64 and FP8-row values are rounded to f16 (2^-12 each;
2^-17 for the two-term weights over BF16 pages), so the output moves by at most
2^-9 A, A = sum p |v| / sum p, which the oracle gives as the
attention over |V|.  Scores over FP8-row keys take q in two E4M3 terms, each
element to 2^-17 of the largest: with |q| <= 4.5, sum |k| <= 256 and a scale of
1/8 to 1/16 a score is off by at most 2^-17 * 4.5 * 256 / 16 = 6e-4, a weight by
that much relatively, the output by twice that of A and lse by 6e-4.  fp32 sums
over 256 dims add 2^-16 of |q| |k|.  So out: 2^-8 |out| + (2^-9 + 2e-3) A, lse
1e-3.
"""

import math

import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import formats as OF
from oracle import rope as OR
from oracle import verify as OV
from oracle.store import PoolImage
from paged_kv_cache_append_gb300 import nk
from paged_kv_cache_append_gb300.workloads import bf16_to_bits

pytestmark = pytest.mark.gpu
DEV = "cuda"
PROFILES = ["bf16", "int8_g64", "fp8_row", "nvfp4_g16", "k8v4"]


def normal(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV) if dtype is None else torch.tensor(a, dtype=dtype, device=DEV)


class Batch:
    """A pool whose B rows share `pages` pages, filled on the GPU and in the oracle."""

    def __init__(self, profile, D, H, G, T, pages, F, order="page_major", seed=0, C=None):
        B = len(F)
        self.B, self.T, self.H, self.Hq, self.D = B, T, H, H * G, D
        C = C or B
        S = max(max(F), 64 * pages, 1) + 64
        L = -(-S // 64)
        M = max(L, C, pages + C * (L - pages))
        rng = np.random.default_rng(seed + D + 7 * G)
        perm = rng.permutation(M).astype(np.int32)
        self.tables = np.zeros((C, L), np.int32)
        self.tables[:, :pages] = perm[:pages]
        self.tables[:, pages:] = perm[pages:pages + C * (L - pages)].reshape(C, L - pages)
        self.rows = rng.permutation(C)[:B].astype(np.int32)
        self.F = np.asarray(F, np.int32)
        self.gpu = nk.Pool(profile, 1, H, D, S, C, M, order=order)
        self.img = PoolImage(profile, 1, H, D, M, order=order)
        for p in self.gpu.planes[0]:                 # stale bytes: NaN patterns past every frontier
            p.fill_(0xFF if profile in ("bf16", "fp8_row", "k8v4") else 0x7F)
        kv = [normal((max(1, 64 * pages), H, D), 900 + seed + i) for i in range(2)]
        if pages:
            self._append(int(self.rows[0]), 0, kv[0][:64 * pages], kv[1][:64 * pages])
        for b in range(B):
            n0 = min(64 * pages, int(self.F[b]))
            n = int(self.F[b]) - n0
            if n:
                self._append(int(self.rows[b]), n0, normal((n, H, D), 1000 + b), normal((n, H, D), 2000 + b))
        self.q = normal((B, T, self.Hq, D), 5 + seed)
        self.scale = 1 / math.sqrt(D)
        self.d = dict(tables=dev(self.tables), rows=dev(self.rows), F=dev(self.F), q=self.q.to(DEV))

    def _append(self, row, at, k, v):
        self.gpu.append(0, dev(self.tables), dev([row], torch.int32), dev([at], torch.int32), k[None].to(DEV),
                        v[None].to(DEV))
        self.img.append(0, self.tables, np.array([row]), np.array([at]), bf16_to_bits(k[None]), bf16_to_bits(v[None]))

    def run(self, pages, **kw):
        shared = dev([pages], torch.int32)
        out, lse = self.gpu.shared_decode(0, self.d["q"], self.d["tables"], self.d["rows"], self.d["F"], shared,
                                          self.scale, **dict(dict(share_from=0), **kw))
        torch.cuda.synchronize()
        return out.cpu(), lse.cpu()

    def reference(self, q=None):
        q = OF.bf16_bits_to_f64(bf16_to_bits(self.q if q is None else q))
        o, l, a = [], [], []
        for b in range(self.B):
            K, V = self.img.gather(0, self.tables[self.rows[b]], int(self.F[b]))
            x, y = OA.decode(q[b], K, V, int(self.F[b]), self.scale)
            o.append(x)
            l.append(y)
            a.append(OA.decode(q[b], K, np.abs(V), int(self.F[b]), self.scale)[0])
        return np.stack(o), np.stack(l), np.stack(a)


def check(out, lse, ref):
    o, l, a = ref
    got = out.float().numpy().astype(np.float64)
    assert np.all(np.isfinite(got))
    excess = np.abs(got - o) - (2.0 ** -8 * np.abs(o) + (2.0 ** -9 + 2e-3) * a)
    assert np.all(excess <= 0), f"out excess {excess.max()}"
    gl = lse.numpy().astype(np.float64)
    fin = np.isfinite(l)
    assert np.array_equal(np.isfinite(gl), fin)
    assert not fin.any() or np.abs(gl[fin] - l[fin]).max() <= 1e-3, np.abs(gl[fin] - l[fin]).max()


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,G,T", [(2, 8, 1), (1, 4, 4), (2, 8, 2), (1, 1, 1), (1, 5, 3)])
def test_shared_shapes(profile, D, H, G, T):
    """Own parts that end inside a page, of T tokens alone, of several pages."""
    b = Batch(profile, D, H, G, T, 3, [192 + T, 192 + 64, 192 + 130, 192 + 200])
    check(*b.run(3), b.reference())


@pytest.mark.parametrize("profile", ["fp8_row", "nvfp4_g16", "k8v4"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_verify_rows_beyond_the_warp_kernel(profile, D):
    """T * G = 32: the rows' own pages run on the tensor-core decode, and the
    batch's 256 query rows take two prefix tiles."""
    b = Batch(profile, D, 2, 8, 4, 5, [330, 324, 400, 383, 384, 385, 512, 700])
    check(*b.run(5), b.reference())


@pytest.mark.parametrize("profile", ["bf16", "int8_g64"])
def test_verify_32_rows_warp_kernel(profile):
    b = Batch(profile, 128, 1, 8, 4, 4, [260, 300, 511])
    check(*b.run(4), b.reference())


@pytest.mark.parametrize("profile", PROFILES)
def test_long_prefix_every_split(profile):
    """More pages than page ranges, eight rows (one without keys)."""
    n = 170
    F = [64 * n + x for x in (1, 2, 63, 64, 65, 300)] + [64 * n - 1, 0]
    b = Batch(profile, 64, 1, 4, 1, n, F)
    out, lse = b.run(n)
    check(out, lse, b.reference())
    assert torch.all(out[7] == 0) and torch.all(torch.isneginf(lse[7]))


@pytest.mark.parametrize("profile", ["bf16", "k8v4"])
@pytest.mark.parametrize("pages", [0, 1, 2, 3, 4, 100, -1])
def test_any_number_of_shared_pages(profile, pages):
    """Fewer shared pages than the rows have in common, none, and numbers that
    only some rows or no row can use: the same results (rows that do not see
    all of them are attended by themselves)."""
    b = Batch(profile, 128, 2, 4, 2, 3, [194, 193, 150, 300, 66, 1])
    s = torch.cuda.current_stream().cuda_stream
    nk.nk_status_read(True, s)
    check(*b.run(min(pages, 3) if pages < 100 else pages), b.reference())
    assert nk.nk_status_read(True, s) == 0


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("D,B,G,T,pages", [(64, 8, 1, 3, 24), (64, 6, 8, 4, 26), (128, 2, 1, 1, 25), (128, 3, 16, 2, 15),
                                           (128, 8, 4, 4, 26), (256, 2, 8, 1, 25), (256, 8, 4, 4, 13)])
def test_many_pages_per_range(profile, D, B, G, T, pages):
    """So many KV heads that a range is many pages: the rings, the score
    buffers and the parities go around several times; 2 to 192 query rows, so
    that warps and whole pipelines are without rows."""
    if T * G > (16 if D == 256 and profile in ("bf16", "int8_g64") else 32):
        pytest.skip("not a decode of this profile")
    H = 38
    b = Batch(profile, D, H, G, T, pages, [64 * pages + T + 30 * i for i in range(B)])
    out, lse = b.run(pages)
    o2, l2 = (x.cpu() for x in b.gpu.decode(0, b.d["q"], b.d["tables"], b.d["rows"], b.d["F"], b.scale))
    # every head against the decode (A <= max |v| < 6 for N(0, 1) values; both sides rounded), three against the oracle
    assert (out.float() - o2.float()).abs().max() <= 2.0 ** -7 * o2.float().abs().max() + 2 * (2.0 ** -9 + 2e-3) * 6
    assert (lse - l2).abs().max() <= 2e-3
    rows = [r for h in (0, 17, H - 1) for r in range(h * G, (h + 1) * G)]
    q = OF.bf16_bits_to_f64(bf16_to_bits(b.q))
    for i in (0, B - 1):
        K, V = b.img.gather(0, b.tables[b.rows[i]], int(b.F[i]))
        heads = [0, 17, H - 1]
        o, l = OA.decode(q[i][:, rows], K[:, heads], V[:, heads], int(b.F[i]), b.scale)
        a, _ = OA.decode(q[i][:, rows], K[:, heads], np.abs(V[:, heads]), int(b.F[i]), b.scale)
        check(out[i][:, rows], lse[i][:, rows], (o, l, a))


@pytest.mark.parametrize("profile,G,T", [("bf16", 8, 1), ("k8v4", 8, 4), ("int8_g64", 4, 2)])
@pytest.mark.parametrize("share_from", [-1, 1, 20, 21, 1 << 20, 1 << 40])
def test_the_choice_does_not_change_results(profile, G, T, share_from):
    """Whichever side of `share_from` the call falls on, also one row."""
    for F in ([64 * 20 + 9, 64 * 20 + 100, 64 * 20 + T, 64 * 20 + 64], [64 * 20 + 33]):
        b = Batch(profile, 128, 2, G, T, 20, F)
        check(*b.run(20, share_from=share_from), b.reference())


@pytest.mark.parametrize("seed", range(4))
def test_random_batches_against_the_decode(seed):
    """Any profile, heads, lengths and rows that do not take part, over a
    workspace of NaN: both ways to divide the SMs, within the two calls'
    tolerances (a softmax scale s / sqrt(D) scales the scores' errors by s)."""
    rng = np.random.default_rng(500 + seed)
    stream = torch.cuda.current_stream().cuda_stream
    done = 0
    while done < 25:
        profile, D = rng.choice(PROFILES), int(rng.choice([64, 128, 256]))
        G, T, H = int(rng.choice([1, 2, 4, 5, 8, 16])), int(rng.choice([1, 1, 2, 3, 4])), int(rng.choice([1, 2, 3, 5, 8, 16]))
        if G * T > (16 if D == 256 and profile in ("bf16", "int8_g64") else 32):
            continue
        done += 1
        B, pages = int(rng.integers(1, 9)), int(2 ** rng.uniform(0, 8))
        F = [int(rng.integers(0, 64 * pages + 1)) if rng.random() < 0.1
             else 64 * pages + T + int(2 ** rng.uniform(0, rng.choice([6, 11]))) for _ in range(B)]
        S = max(F) + 64
        L = -(-S // 64)
        M = pages + B * (L - pages)
        pool = nk.Pool(str(profile), 1, H, D, S, B, M, order=str(rng.choice(["page_major", "head_major"])))
        perm = rng.permutation(M).astype(np.int32)
        tables = np.concatenate([np.tile(perm[:pages], (B, 1)), perm[pages:].reshape(B, L - pages)], 1)
        tables, rows, F = dev(tables), dev(rng.permutation(B).astype(np.int32)), dev(np.array(F, np.int32))
        g = torch.Generator(DEV).manual_seed(int(rng.integers(1 << 30)))
        new = lambda *shape: torch.randn(shape, device=DEV, generator=g).bfloat16()  # noqa: E731
        for b in range(B):
            pool.append(0, tables, rows[b:b + 1].contiguous(), dev([0], torch.int32), new(1, 64 * L, H, D), new(1, 64 * L, H, D))
        q, s = new(B, T, H * G, D), float(rng.choice([1, 3, -1]))
        o2, l2 = pool.decode(0, q, tables, rows, F, s / math.sqrt(D))
        ws = torch.full((pool.shared_workspace(B, T, H * G).numel(),), 0xFF, dtype=torch.uint8, device=DEV)
        nk.nk_status_read(True, stream)
        for _ in range(2):
            out, lse = pool.shared_decode(0, q, tables, rows, F, dev([pages], torch.int32), s / math.sqrt(D),
                                          workspace=ws, share_from=0)
        assert nk.nk_status_read(True, stream) == 0
        what = f"{profile} D {D} G {G} T {T} H {H} pages {pages} F {F.tolist()}"
        limit = 2.0 ** -7 * o2.float().abs().max() + 2 * (2.0 ** -9 + 2e-3 * abs(s)) * 6
        assert (out.float() - o2.float()).abs().max() <= limit, what
        fin = torch.isfinite(l2)
        assert torch.equal(torch.isfinite(lse), fin), what
        assert not fin.any() or (lse - l2)[fin].abs().max() <= 2e-3 * abs(s), what


def test_head_major_and_spare_table_rows():
    b = Batch("fp8_row", 128, 3, 4, 1, 6, [400, 500, 385], order="head_major", C=7)
    check(*b.run(6), b.reference())


def test_one_row():
    b = Batch("k8v4", 128, 2, 8, 1, 20, [64 * 20 + 77])
    check(*b.run(20), b.reference())


def test_many_kv_heads():
    """More KV heads than SMs / rows: one page range per tile, one split per row."""
    b = Batch("nvfp4_g16", 64, 160, 1, 1, 4, [257, 300, 270, 320, 260])
    check(*b.run(4), b.reference())


@pytest.mark.parametrize("profile", PROFILES)
def test_close_to_the_decode_and_repeatable(profile):
    """Against nk_paged_decode_attention on the same pool (both sides within
    their tolerance of the oracle), and the same bits on every call."""
    b = Batch(profile, 128, 2, 8, 1, 12, [64 * 12 + 10 * i + 1 for i in range(8)])
    out, lse = b.run(12)
    o2, l2 = b.gpu.decode(0, b.d["q"], b.d["tables"], b.d["rows"], b.d["F"], b.scale)
    ref = b.reference()
    check(out, lse, ref)
    check(o2.cpu(), l2.cpu(), ref)
    for _ in range(3):
        again = b.run(12)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_tables_that_differ_in_the_prefix_are_reported():
    b = Batch("bf16", 64, 1, 4, 1, 4, [300, 301, 302])
    s = torch.cuda.current_stream().cuda_stream
    nk.nk_status_read(True, s)
    b.run(4)
    assert nk.nk_status_read(True, s) == 0
    t = b.tables.copy()
    t[b.rows[1], 2] = t[b.rows[1], 4]
    b.d["tables"] = dev(t)
    b.run(4)
    assert nk.nk_status_read(True, s) == nk.STATUS_PREFIX


def test_bad_rows_and_pages_do_not_fault():
    """A frontier past the table, a table row and page ids outside: recorded,
    the other rows unaffected."""
    b = Batch("fp8_row", 64, 1, 4, 1, 3, [200, 230, 260])
    ref = b.reference()
    s = torch.cuda.current_stream().cuda_stream
    b.d["F"] = dev(np.array([200, 1 << 30, 260], np.int32))
    nk.nk_status_read(True, s)
    out, lse = b.run(3)
    assert nk.nk_status_read(True, s) & nk.STATUS_FRONTIER
    check(out[[0, 2]], lse[[0, 2]], [r[[0, 2]] for r in ref])
    b.d["F"] = dev(b.F)
    b.d["rows"] = dev(np.array([b.rows[0], -1, b.rows[2]], np.int32))
    out, lse = b.run(3)
    check(out[[0, 2]], lse[[0, 2]], [r[[0, 2]] for r in ref])
    b.d["rows"] = dev(b.rows)
    t = b.tables.copy()
    t[b.rows[1], 3] = b.gpu.M + 5
    b.d["tables"] = dev(t)
    nk.nk_status_read(True, s)
    out, lse = b.run(3)
    assert nk.nk_status_read(True, s) & nk.STATUS_PAGE_RANGE
    check(out[[0, 2]], lse[[0, 2]], [r[[0, 2]] for r in ref])


def test_the_least_frontier_takes_no_part():
    """frontiers - T must not wrap around: a row of -2^31 valid tokens is a bad row, not one behind the prefix."""
    b = Batch("bf16", 64, 1, 4, 2, 3, [200, 230, 260])
    ref = b.reference()
    b.d["F"] = dev(np.array([200, -2 ** 31, 260], np.int32))
    s = torch.cuda.current_stream().cuda_stream
    nk.nk_status_read(True, s)
    out, lse = b.run(3)
    assert nk.nk_status_read(True, s) == nk.STATUS_FRONTIER
    check(out[[0, 2]], lse[[0, 2]], [r[[0, 2]] for r in ref])
    assert torch.all(out[1] == 0) and torch.all(torch.isneginf(lse[1]))


@pytest.mark.parametrize("profile,D", [("bf16", 128), ("bf16", 256), ("fp8_row", 64), ("fp8_row", 256), ("k8v4", 128)])
@pytest.mark.parametrize("plane", [0, 1])
@pytest.mark.parametrize("page,token", [(1, 5), (4, 63), (6, 3)])
def test_a_visible_nan_is_not_lost(profile, D, plane, page, token):
    """A key or value of NaN in a shared page (1, 4) or in a row's own (6) makes
    the outputs that see it NaN, and no others: as the plain decode."""
    if profile == "k8v4" and plane == 1:
        pytest.skip("E2M1 codes have no NaN")
    b = Batch(profile, D, 2, 4, 1, 6, [64 * 6 + x for x in (1, 4, 70, 200)])
    rows = b.gpu.planes[0][plane].view(b.gpu.M, b.H, 64, -1)
    rows[int(b.tables[b.rows[2], page]), 1, token] = 0xFF
    out, lse = b.run(6)
    ref, _ = b.gpu.decode(0, b.d["q"], b.d["tables"], b.d["rows"], b.d["F"], b.scale)
    nan = torch.zeros(out.shape, dtype=torch.bool)
    nan[slice(None) if page < 6 else 2, :, 4:] = True
    assert torch.equal(out.isnan(), nan) and torch.equal(ref.cpu().isnan(), nan)
    assert torch.equal(lse.isnan(), nan[..., 0]) if plane == 0 else not lse.isnan().any()


def test_pool_past_32_bits():
    """Planes of 5 GB, every page behind the first 4 GB: the rotated append and
    the attention give a small pool's bits."""
    D, H, G, pages = 128, 8, 4, 6
    F = [64 * pages + x for x in (3, 70)]
    small = Batch("bf16", D, H, G, 1, pages, F)
    L, M = 20000, 40000
    big = nk.Pool("bf16", 1, H, D, 64 * L, 2, M)
    far = small.tables + np.int32(M - 1 - small.tables.max())
    wide = np.full((2, L), M, np.int32)
    wide[:, :far.shape[1]] = far
    assert int(far.min()) * H * 64 * D * 2 > 2 ** 32
    for p, s in zip(big.planes[0], small.gpu.planes[0]):
        p = p.view(M, -1)
        p[torch.from_numpy(far.ravel()).to(DEV).long()] = s.view(small.gpu.M, -1)[dev(small.tables.ravel()).long()]
    rope = nk.Rope(dev(OR.table(1024, D)), D, q_weight=normal(D, 1).to(DEV), k_weight=normal(D, 2).to(DEV))
    x = normal((2, 1, H * G + 2 * H, D), 7).to(DEV)
    q, k, v = x.split([H * G, H, H], 2)
    got = []
    for pool, tables in ((small.gpu, small.d["tables"]), (big, dev(wide))):
        qr = pool.append_rope(0, tables, small.d["rows"], small.d["F"], k, v, rope, q=q)
        o, l = pool.shared_decode(0, qr, tables, small.d["rows"], small.d["F"] + 1, dev([pages], torch.int32),
                                  small.scale, share_from=0)
        got.append((qr, o, l))
    for a, c in zip(*got):
        assert torch.equal(a, c)
    for p, s in zip(big.planes[0], small.gpu.planes[0]):
        assert torch.equal(p.view(M, -1)[torch.from_numpy(far.ravel()).to(DEV).long()],
                           s.view(small.gpu.M, -1)[dev(small.tables.ravel()).long()])


def test_two_graphs_that_share_a_workspace():
    """Two captured calls of different shapes over one workspace, replayed in
    turn on one stream with other numbers of shared pages and frontiers."""
    a = Batch("fp8_row", 128, 2, 8, 1, 20, [64 * 20 + 9 * i + 1 for i in range(8)])
    b = Batch("k8v4", 128, 4, 4, 4, 12, [64 * 12 + 50 * i + 5 for i in range(5)])
    ws = torch.empty(max(x.gpu.shared_workspace(x.B, x.T, x.Hq).numel() for x in (a, b)), dtype=torch.uint8, device=DEV)
    graphs, outs, shared = [], [], [dev([20], torch.int32), dev([12], torch.int32)]
    for x, n in zip((a, b), shared):
        x.gpu.shared_decode(0, x.d["q"], x.d["tables"], x.d["rows"], x.d["F"], n, x.scale, workspace=ws, share_from=0)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(x.gpu.shared_decode(0, x.d["q"], x.d["tables"], x.d["rows"], x.d["F"], n, x.scale,
                                            workspace=ws, share_from=0))
        graphs.append(g)
    refs = [x.reference() for x in (a, b)]
    for take in ((20, 12), (7, 3), (0, 12), (20, 0)):     # pages attended once: the same results
        for n, t in zip(shared, take):
            n.fill_(t)
        for _ in range(2):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for (o, l), ref in zip(outs, refs):
            check(o.cpu(), l.cpu(), ref)


def test_refusals():
    b = Batch("bf16", 64, 1, 4, 1, 2, [140, 150])
    with pytest.raises(nk.NkError) as e:
        b.run(2, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.code == -7
    for bad in (dict(q=b.d["q"].float()), dict(q=b.d["q"][..., :32]), dict(shared_pages=b.d["F"]),
                dict(frontiers=b.d["F"][:1]), dict(table_rows=b.d["rows"].long()), dict(out=b.d["q"][:1]),
                dict(tables=b.d["tables"][:1])):
        kw = dict(dict(q=b.d["q"], tables=b.d["tables"], table_rows=b.d["rows"], frontiers=b.d["F"],
                       shared_pages=dev([2], torch.int32), scale=b.scale), **bad)
        with pytest.raises(ValueError):
            b.gpu.shared_decode(0, **kw)
    with pytest.raises(nk.NkError) as e:
        b.gpu.shared_decode(0, b.d["q"], b.d["tables"], b.d["rows"], b.d["F"], dev([2], torch.int32), float("nan"))
    assert e.value.code == -1
    big = normal((2, 9, 4, 64), 1).to(DEV)          # 36 query rows per KV head
    with pytest.raises(nk.NkError) as e:
        b.gpu.shared_decode(0, big, b.d["tables"], b.d["rows"], b.d["F"], dev([2], torch.int32), b.scale)
    assert e.value.code == -4


def test_two_streams_with_their_own_workspaces():
    """Two calls in flight at once, each with its own workspace and outputs."""
    bs = [Batch("k8v4", 128, 2, 8, 1, 40, [64 * 40 + 9 * i + 1 for i in range(8)], seed=s) for s in (0, 50)]
    refs = [b.run(40) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    shared = dev([40], torch.int32)
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for b, s in zip(bs, streams):
            with torch.cuda.stream(s):
                outs.append(b.gpu.shared_decode(0, b.d["q"], b.d["tables"], b.d["rows"], b.d["F"], shared, b.scale,
                                                share_from=0))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(outs):
        assert torch.equal(o.cpu(), refs[i % 2][0]) and torch.equal(l.cpu(), refs[i % 2][1])


# ------------------------------------------------------------- the serving step

@pytest.mark.parametrize("profile,D", [("bf16", 64), ("k8v4", 128), ("fp8_row", 256), ("int8_g64", 128),
                                       ("nvfp4_g16", 64)])
def test_speculative_steps_in_one_graph(profile, D):
    """One captured graph per step: rotated append of K + 1 tokens with their
    queries, shared-prefix verify attention, verification of the drafts and the
    trimmed frontier, which the next step's positions follow.  Three replays
    with new inputs against the oracle, step by step."""
    B, H, G, K, V, pages = 3, 2, 4, 3, 1000, 5
    T = K + 1
    batch = Batch(profile, D, H, G, T, pages, [64 * pages + x for x in (5, 60, 126)])
    pool, img = batch.gpu, batch.img
    Hq = H * G
    cs = OR.table(1024, D)
    w = [(1 + 0.2 * torch.randn(D, generator=torch.Generator().manual_seed(i))).to(torch.bfloat16) for i in (1, 2)]
    rope = nk.Rope(dev(cs), D, q_weight=w[0].to(DEV), k_weight=w[1].to(DEV))
    committed = dev(batch.F)                              # tokens that stand
    qkv = torch.zeros((B, T, Hq + 2 * H, D), dtype=torch.bfloat16, device=DEV)
    target = torch.zeros((B, K + 1, V), device=DEV)
    draft = torch.zeros((B, K, V), device=DEV)
    tokens, u = torch.zeros((B, K), dtype=torch.int32, device=DEV), torch.zeros((B, K + 1), device=DEV)
    shared, ws = dev([pages], torch.int32), pool.shared_workspace(B, T, Hq)
    out, lse = torch.zeros((B, T, Hq, D), dtype=torch.bfloat16, device=DEV), torch.zeros((B, T, Hq), device=DEV)
    q_out = torch.zeros_like(out)

    def step():
        q, k, v = qkv.split([Hq, H, H], 2)
        pool.append_rope(0, batch.d["tables"], batch.d["rows"], committed, k, v, rope, q=q, q_out=q_out)
        frontier = committed + T
        pool.shared_decode(0, q_out, batch.d["tables"], batch.d["rows"], frontier, shared, batch.scale, out=out,
                           lse=lse, workspace=ws, share_from=0)
        n, tok, after = nk.verify_drafts(target, tokens, u, draft=draft, frontiers=frontier)
        committed.copy_(after)
        return n, tok

    rng = np.random.default_rng(9)
    graph, result = None, None
    F = batch.F.astype(np.int64)
    for turn in range(4):
        x = normal((B, T, Hq + 2 * H, D), 40 + turn)
        p = rng.random((B, K + 1, V)).astype(np.float32)
        p /= p.sum(-1, keepdims=True)
        dq = (p[:, :K] * (1 + 0.5 * rng.random((B, K, V)))).astype(np.float32)
        dq /= dq.sum(-1, keepdims=True)
        ids, uu = rng.integers(0, V, (B, K)), rng.random((B, K + 1)).astype(np.float32)
        for t, h in ((qkv, x), (target, torch.from_numpy(p)), (draft, torch.from_numpy(dq)),
                     (tokens, torch.from_numpy(ids.astype(np.int32))), (u, torch.from_numpy(uu))):
            t.copy_(h)
        torch.cuda.synchronize()
        if turn == 0:
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                result = step()
            torch.cuda.synchronize()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    result = step()
            graph.replay()
            torch.cuda.synchronize()
        # the GPU's own stored keys are within a code step of the oracle's (tests/test_gpu_rope.py);
        # the attention is checked on the bytes that the append stored
        for i, plane in enumerate(pool.planes[0]):
            img.planes[0][i][...] = plane.cpu().numpy().reshape(img.planes[0][i].shape)
        batch.F = (F + T).astype(np.int32)
        for b in range(B):
            qr, m = OR.norm_rotate(x[b, :, :Hq].double().numpy(), cs, F[b] + np.arange(T), D, False,
                                   w[0].double().numpy())
            got = q_out[b].cpu().double().numpy()
            assert np.all(np.abs(got - qr) <= 2.0 ** -8 * np.abs(qr) + 2.0 ** -16 * m)
        check(out.cpu(), lse.cpu(), batch.reference(q_out.cpu()))
        for b in range(B):
            n, t = OV.verify(p[b], dq[b], ids[b].tolist(), uu[b], K)
            assert int(result[0][b]) == n and result[1][b].tolist() == t
            F[b] += n + 1
        assert committed.cpu().tolist() == F.tolist()


def test_norm_rope_feeds_the_fused_append_decode():
    """nk_qk_norm_rope straight before nk_paged_append_decode_attention (which
    starts before its predecessor ends): the same as the rotated append followed
    by the decode, over BF16 pages bit for bit in the pages."""
    D, H, G, T = 128, 2, 8, 1
    a, b = (Batch("bf16", D, H, G, T, 0, [300, 63, 64, 1000]) for _ in range(2))
    rope = nk.Rope(dev(OR.table(2048, D)), D, q_weight=normal(D, 1).to(DEV), k_weight=normal(D, 2).to(DEV))
    x = normal((4, T, H * G + 2 * H, D), 77).to(DEV)
    q, k, v = x.split([H * G, H, H], 2)
    at = a.d["F"]
    for _ in range(3):
        q1, k1 = nk.qk_norm_rope(q, k, at[:, None].contiguous(), rope)
        o1, l1 = a.gpu.append_decode(0, q1, k1, v.contiguous(), a.d["tables"], a.d["rows"], at + T, a.scale)
    q2 = b.gpu.append_rope(0, b.d["tables"], b.d["rows"], at, k, v, rope, q=q)
    o2, l2 = b.gpu.decode(0, q2, b.d["tables"], b.d["rows"], at + T, b.scale)
    assert torch.equal(q1, q2)
    for p1, p2 in zip(a.gpu.planes[0], b.gpu.planes[0]):
        assert torch.equal(p1, p2)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
