"""GPU parity of the per-head norm + rotation and of the append that does both.

Tolerances, derived.  An fp32 evaluation of one output is off by at most
2^-16 of the size of its two terms |a| + |b|: the sum of up to 256 squares by
256 * 2^-24 (its root by half of that, 2^-17), the reciprocal root, the scale,
the weight and the rotation by a few 2^-23.  A bf16 result adds half a step,
2^-8 of its value.  A stored scale s is the binary16 (E4M3) rounding of
amax / 127, amax / 448 (amax / 6): half a step, 2^-11 (2^-4) of it, or half a
subnormal step.  A stored value c * s is off by half a code step times s:
1/2 (INT8), 2^-4 of the value or 2^-10 s near zero (E4M3), 1/4, 1/2 or 1 below
2, 4 and 8 (E2M1).
"""

import numpy as np
import pytest
import torch

from oracle import rope as OR
from paged_kv_cache_append_gb300 import nk

pytestmark = pytest.mark.gpu
DEV = "cuda"
PROFILES = ["bf16", "int8_g64", "fp8_row", "nvfp4_g16", "k8v4"]
FP32 = 2.0 ** -16


def normal(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def weights(D, seed):
    return (1 + 0.3 * torch.randn(D, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16)


def check_bf16(got, ref, m, what=""):
    err = np.abs(f64(got) - ref) - (2.0 ** -8 * np.abs(ref) + FP32 * m)
    assert np.all(err <= 0), f"{what}: worst excess {err.max()}"


def make_rope(D, rd, pairs, norm, positions=512, offset=0.0):
    cs = OR.table(positions, rd) if rd else np.zeros((positions, 0), np.float32)
    wq, wk = (weights(D, 1), weights(D, 2)) if norm else (None, None)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    rope = nk.Rope(torch.from_numpy(cs).to(DEV), rd, interleaved=pairs, q_weight=dev(wq), k_weight=dev(wk), eps=1e-6,
                   weight_offset=offset)
    return rope, cs, None if wq is None else f64(wq), None if wk is None else f64(wk)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rd", [0, 16, 48, 64])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope(D, rd, pairs, norm):
    N, Hq, H = 13, 5, 3
    rope, cs, wq, wk = make_rope(D, rd, pairs, norm)
    q, k = normal((N, Hq, D), 3), normal((N, H, D), 4, 7.0)
    pos = np.random.default_rng(D + rd).integers(0, 512, N).astype(np.int32)
    qo, ko = nk.qk_norm_rope(q.to(DEV), k.to(DEV), torch.from_numpy(pos).to(DEV), rope)
    for got, x, w in ((qo, q, wq), (ko, k, wk)):
        ref, m = OR.norm_rotate(f64(x), cs, pos, rd, pairs, w)
        check_bf16(got, ref, m)


@pytest.mark.parametrize("D,rd", [(64, 64), (128, 128), (256, 256), (128, 96), (256, 112)])
@pytest.mark.parametrize("pairs", [False, True])
def test_norm_rope_long_and_strided(D, rd, pairs):
    """Long enough for several heads per unit, from one fused row, weights
    stored as w - 1, in place."""
    N, Hq, H = 20011, 9, 5
    rope, cs, wq, wk = make_rope(D, rd, pairs, True, offset=1.0)
    x = normal((N, Hq + 2 * H, D), 5).to(DEV)
    before = x.clone()
    q, k, v = x.split([Hq, H, H], 1)
    pos = torch.randint(0, 512, (N,), dtype=torch.int32, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    qo, ko = nk.qk_norm_rope(q, k, pos, rope)
    sample = np.random.default_rng(1).integers(0, N, 300)
    sample[:2] = 0, N - 1
    p = pos.cpu().numpy()[sample]
    for got, src, w in ((qo, before[:, :Hq], wq), (ko, before[:, Hq:Hq + H], wk)):
        ref, m = OR.norm_rotate(f64(src[sample]), cs, p, rd, pairs, w, offset=1.0)
        check_bf16(got[sample], ref, m)
    nk.qk_norm_rope(q, k, pos, rope, q_out=q, k_out=k)     # in place on the fused rows
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, before[:, Hq + H:])


def test_norm_rope_one_operand_and_one_token():
    """Queries alone and keys alone (the C call), N = 1: the same bits as together."""
    D, Hq, H = 128, 7, 2
    rope, *_ = make_rope(D, 64, False, True)
    q, k = normal((1, Hq, D), 8).to(DEV), normal((1, H, D), 9).to(DEV)
    pos = torch.tensor([300], dtype=torch.int32, device=DEV)
    qo, ko = nk.qk_norm_rope(q, k, pos, rope)
    a, b = torch.zeros_like(q), torch.zeros_like(k)
    s = torch.cuda.current_stream().cuda_stream
    rows = lambda t: nk.Rows(t.data_ptr(), t.stride(0), t.stride(1))  # noqa: E731
    nk.nk_qk_norm_rope(rope.desc, D, rows(q), Hq, None, 0, pos.data_ptr(), 1, rows(a), None, s)
    nk.nk_qk_norm_rope(rope.desc, D, None, 0, rows(k), H, pos.data_ptr(), 1, None, rows(b), s)
    assert torch.equal(a, qo) and torch.equal(b, ko)


def test_norm_rope_positions_out_of_range_are_skipped():
    rope, cs, *_ = make_rope(64, 64, False, False)
    q, k = normal((4, 2, 64), 1).to(DEV), normal((4, 1, 64), 2).to(DEV)
    pos = torch.tensor([3, -1, 512, 511], dtype=torch.int32, device=DEV)
    qo, ko = torch.full_like(q, 9), torch.full_like(k, 9)
    nk.nk_status_read(True, torch.cuda.current_stream().cuda_stream)
    nk.qk_norm_rope(q, k, pos, rope, q_out=qo, k_out=ko)
    assert nk.nk_status_read(True, torch.cuda.current_stream().cuda_stream) == nk.STATUS_FRONTIER
    assert torch.all(qo[1:3] == 9) and torch.all(ko[1:3] == 9)
    ref, m = OR.norm_rotate(f64(q), cs, np.array([3, 0, 0, 511]), 64, False)
    check_bf16(qo[[0, 3]], ref[[0, 3]], m[[0, 3]])


def test_norm_rope_strides_past_32_bits():
    """Tokens 2^30 + 64 elements apart (the last one 4 GB and more into the
    buffer), in place: the bits of the packed rows."""
    rope, *_ = make_rope(64, 32, True, True)
    step = 2 ** 30 + 64
    buf = torch.empty(2 * step + 4 * 64, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((3, 4, 64), (step, 64, 1))
    x.copy_(normal((3, 4, 64), 6))
    pos = torch.tensor([1, 2, 500], dtype=torch.int32, device=DEV)
    ref = nk.qk_norm_rope(x[:, :3].contiguous(), x[:, 3:].contiguous(), pos, rope)
    nk.qk_norm_rope(x[:, :3], x[:, 3:], pos, rope, q_out=x[:, :3], k_out=x[:, 3:])
    assert torch.equal(x[:, :3], ref[0]) and torch.equal(x[:, 3:], ref[1])


def test_norm_rope_captured_on_another_stream():
    """Captured on a side stream and replayed with other rows and positions."""
    rope, cs, wq, wk = make_rope(128, 128, False, True)
    q, k = torch.zeros((9, 4, 128), dtype=torch.bfloat16, device=DEV), torch.zeros((9, 2, 128), dtype=torch.bfloat16, device=DEV)
    qo, ko, pos = torch.empty_like(q), torch.empty_like(k), torch.zeros(9, dtype=torch.int32, device=DEV)
    nk.qk_norm_rope(q, k, pos, rope, q_out=qo, k_out=ko)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        nk.qk_norm_rope(q, k, pos, rope, q_out=qo, k_out=ko)
    for turn in range(3):
        x, y = normal((9, 4, 128), 50 + turn), normal((9, 2, 128), 60 + turn)
        p = np.random.default_rng(turn).integers(0, 512, 9).astype(np.int32)
        q.copy_(x), k.copy_(y), pos.copy_(torch.from_numpy(p))
        g.replay()
        for got, src, w in ((qo, x, wq), (ko, y, wk)):
            ref, m = OR.norm_rotate(f64(src), cs, p, 128, False, w)
            check_bf16(got, ref, m)


def test_norm_rope_extremes():
    """A zero row stays zero under the norm, the largest bf16 magnitudes stay
    finite without it, and infinities and NaN stay in their own rows."""
    D = 64
    rope, *_ = make_rope(D, 64, False, True)
    q = normal((4, 1, D), 3)
    q[0] = 0
    q[1, 0, 5] = float("inf")
    q[2, 0, 40] = float("nan")
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    qo, _ = nk.qk_norm_rope(q.to(DEV), q.to(DEV), pos, rope)
    assert torch.all(qo[0] == 0) and torch.isfinite(qo[3]).all()
    assert not torch.isfinite(qo[1]).all() and not torch.isfinite(qo[2]).all()
    plain, *_ = make_rope(D, 64, False, False)
    big = torch.full((1, 1, D), 2.0 ** 100).to(torch.bfloat16)
    out, _ = nk.qk_norm_rope(big.to(DEV), big.to(DEV), pos[:1], plain)
    assert torch.equal(out.cpu(), big)


# ------------------------------------------------------------------- append

def decoded(profile, side, code, scale, D):
    """(values, scales repeated per element) of code / scale rows (uint8 tensors [n, bytes])."""
    kind = {"bf16": "b", "int8_g64": "i", "fp8_row": "f", "nvfp4_g16": "n", "k8v4": "fn"[side]}[profile]
    if kind == "b":
        return f64(code.view(torch.bfloat16)), None, kind
    if kind == "i":
        s = np.repeat(f64(scale.view(torch.float16)), 64, axis=-1)
        return f64(code.view(torch.int8)) * s, s, kind
    if kind == "f":
        s = np.repeat(f64(scale.view(torch.float16)), D, axis=-1)
        return f64(code.view(torch.float8_e4m3fn).float()) * s, s, kind
    s = np.repeat(f64(scale.view(torch.float8_e4m3fn).float()), 16, axis=-1)
    lut = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
    c = code.cpu().numpy()
    v = np.stack([lut[c & 15], lut[c >> 4]], axis=-1).reshape(c.shape[0], -1)
    return v * s, s, kind


def check_stored(kind, got, s, ref, m, D):
    """Stored values against the exact rows ref [n, D]."""
    if kind == "b":
        assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + FP32 * m)
        return
    group = {"i": 64, "f": D, "n": 16}[kind]
    top = {"i": 127.0, "f": 448.0, "n": 6.0}[kind]
    amax = np.repeat(np.abs(ref).reshape(-1, group).max(1), group).reshape(ref.shape)
    want = amax / top
    rel, sub = (2.0 ** -4, 2.0 ** -10) if kind == "n" else (2.0 ** -11, 2.0 ** -25)
    # m of the group's largest element is at most the group's largest m
    mm = np.repeat(m.reshape(-1, group).max(1), group).reshape(ref.shape) / top
    assert np.all(np.abs(s - want) <= rel * want + sub + 2 * FP32 * mm)
    v = np.abs(ref) / np.maximum(s, 1e-30)
    half = {"i": 0.5, "f": np.maximum(2.0 ** -4 * v, 2.0 ** -10),
            "n": np.where(v < 2.1, 0.25, np.where(v < 4.1, 0.5, 1.0))}[kind]
    assert np.all(np.abs(got - ref) <= np.where(s > 0, half * s * (1 + 2.0 ** -10), np.abs(ref)) + FP32 * m)


class Appended:
    """A pool with an append_rope call on it and everything to check it with."""

    def __init__(self, profile, D, Hq, H, T, at, counts=None, rd=64, pairs=False, norm=True, order="page_major",
                 S=300, fused=True, positions=512):
        B = len(at)
        L = -(-S // 64)
        self.pool = nk.Pool(profile, 2, H, D, S, B, B * L, order=order)
        rng = np.random.default_rng(D + T)
        self.tables = rng.permutation(B * L).astype(np.int32).reshape(B, L)
        self.rope, self.cs, self.wq, self.wk = make_rope(D, rd, pairs, norm, positions)
        x = normal((B, T, Hq + 2 * H, D), 11, 1.5).to(DEV)
        self.q, self.k, self.v = x.split([Hq, H, H], 2)
        if not fused:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        self.rows = rng.permutation(B).astype(np.int32)
        self.at, self.T, self.counts = np.asarray(at, np.int32), T, counts
        self.rd, self.pairs, self.D, self.H, self.profile, self.order = rd, pairs, D, H, profile, order
        self.d = {n: torch.from_numpy(v).to(DEV) for n, v in
                  (("tables", self.tables), ("rows", self.rows), ("at", self.at))}
        self.dcounts = None if counts is None else torch.tensor(counts, dtype=torch.int32, device=DEV)
        self.q_out = torch.full((B, T, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)

    def run(self, layer=1):
        return self.pool.append_rope(layer, self.d["tables"], self.d["rows"], self.d["at"], self.k, self.v, self.rope,
                                     q=self.q, q_out=self.q_out, counts=self.dcounts)

    def live(self, b):
        return self.T if self.counts is None else min(max(self.counts[b], 0), self.T)

    def plane_rows(self, plane, layer, b, n):
        """Byte rows [n, H, bytes] of row b's appended tokens."""
        p = self.pool.planes[layer][plane]
        w = self.pool.row_bytes[plane]
        p = p.view(self.H, self.pool.M, 64, w).transpose(0, 1) if self.order == "head_major" \
            else p.view(self.pool.M, self.H, 64, w)
        pos = np.arange(n) + self.at[b]
        g = self.tables[self.rows[b]][pos >> 6].astype(np.int64)
        return p[torch.from_numpy(g).to(DEV), :, torch.from_numpy(pos & 63).to(DEV)]

    def check(self, layer=1):
        bf16 = self.profile == "bf16"
        for b in range(len(self.at)):
            n = self.live(b)
            pos = np.arange(n) + self.at[b]
            ref, m = OR.norm_rotate(f64(self.q[b, :n]), self.cs, pos, self.rd, self.pairs, self.wq)
            check_bf16(self.q_out[b, :n], ref, m, "q_out")
            assert torch.all(self.q_out[b, n:] == 9.0)
            if n == 0:
                continue
            kref, km = OR.norm_rotate(f64(self.k[b, :n]), self.cs, pos, self.rd, self.pairs, self.wk)
            vref = f64(self.v[b, :n])
            for side, (r, mm) in enumerate(((kref, km), (vref, np.abs(vref)))):
                code = self.plane_rows(side, layer, b, n).reshape(n * self.H, -1).contiguous()
                scale = None if bf16 else self.plane_rows(2 + side, layer, b, n).reshape(n * self.H, -1).contiguous()
                got, s, kind = decoded(self.profile, side, code, scale, self.D)
                check_stored(kind, got, s, r.reshape(-1, self.D), mm.reshape(-1, self.D), self.D)


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("pairs,rd,norm", [(False, 64, True), (True, 48, True), (False, 16, False)])
def test_append_rope(profile, D, pairs, rd, norm):
    a = Appended(profile, D, 6, 3, 5, [0, 61, 250], rd=rd, pairs=pairs, norm=norm)
    a.run()
    a.check()
    assert all(not p.any() for p in a.pool.planes[0])       # the other layer is untouched


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("order", ["page_major", "head_major"])
def test_append_rope_ragged_long(profile, order):
    """Several heads per unit, ragged counts (zero among them), both plane orders."""
    a = Appended(profile, 128, 16, 6, 1500, [3, 100, 0, 64], counts=[1500, 0, 1, 777], order=order, S=1700,
                 positions=1700)
    a.run()
    a.check()


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_rope_without_rope_is_the_append(profile, D):
    """rotary_dim 0 and no norm: every byte of every plane equals nk_paged_kv_append's."""
    a = Appended(profile, D, 4, 2, 70, [0, 33], rd=0, norm=False, fused=False)
    with torch.no_grad():
        a.k[0, 0] = 0                                         # zero scales
        a.v[0, 1, :, :16] = 0
        a.k[1, 2] *= 1e30                                     # saturated scales
        a.v[1, 3, 0, 3] = -1e-30
    a.run()
    plain = nk.Pool(profile, 2, a.H, D, 300, 2, a.pool.M)
    plain.append(1, a.d["tables"], a.d["rows"], a.d["at"], a.k, a.v)
    for x, y in zip(a.pool.planes[1], plain.planes[1]):
        assert torch.equal(x, y)
    assert torch.equal(a.q_out, a.q)


@pytest.mark.parametrize("profile", PROFILES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [3, 5000])
def test_append_rope_without_rope_of_any_bits(profile, D, T):
    """Every bit pattern a row can hold (infinities, NaN, subnormals, both
    zeros), few tokens and many: the append's bytes.  Only a NaN of a BF16 key
    or query may change its payload."""
    a = Appended(profile, D, 4, 3, T, [0, 33], rd=0, norm=False, fused=False, S=5100, positions=5100)
    g = torch.Generator().manual_seed(D + T)
    for x in (a.q, a.k, a.v):
        bits = torch.randint(-2 ** 15, 2 ** 15, x.shape, dtype=torch.int16, generator=g)
        bits[:, ::2] &= -0x4001                               # every other token of magnitudes below 2
        x.copy_(bits.view(torch.bfloat16))
    a.run()
    plain = nk.Pool(profile, 2, a.H, D, 5100, 2, a.pool.M)
    plain.append(1, a.d["tables"], a.d["rows"], a.d["at"], a.k, a.v)
    same = lambda x, y: torch.equal(x.isnan(), y.isnan()) and torch.equal(  # noqa: E731
        x.view(torch.int16)[~x.isnan()], y.view(torch.int16)[~y.isnan()])
    for i, (x, y) in enumerate(zip(a.pool.planes[1], plain.planes[1])):
        assert same(x.view(torch.bfloat16), y.view(torch.bfloat16)) if profile == "bf16" and i == 0 else torch.equal(x, y)
    assert same(a.q_out, a.q)


def test_append_rope_equals_norm_rope_then_append_in_bf16():
    """Over a BF16 pool the result is rounded once either way: the same bits."""
    a = Appended("bf16", 128, 8, 2, 9, [60, 7])
    a.run()
    pos = torch.from_numpy((a.at[:, None] + np.arange(9)).astype(np.int32)).to(DEV)
    q, k = nk.qk_norm_rope(a.q, a.k, pos, a.rope)
    plain = nk.Pool("bf16", 2, 2, 128, 300, 2, a.pool.M)
    plain.append(1, a.d["tables"], a.d["rows"], a.d["at"], k, a.v.contiguous())
    assert torch.equal(a.q_out, q)
    for x, y in zip(a.pool.planes[1], plain.planes[1]):
        assert torch.equal(x, y)


def test_append_rope_bad_rows_positions_and_pages_are_skipped():
    a = Appended("fp8_row", 64, 2, 2, 3, [0, 319, 400, 10, 20], S=320, rd=16)
    bad = a.tables.copy()
    bad[a.rows[3], 0] = a.pool.M                              # row 3: page id out of range
    a.d["tables"] = torch.from_numpy(bad).to(DEV)
    rows = a.rows.copy()
    rows[4] = 5                                               # row 4: table row out of range
    a.d["rows"] = torch.from_numpy(rows).to(DEV)
    s = torch.cuda.current_stream().cuda_stream
    nk.nk_status_read(True, s)
    a.run()
    assert nk.nk_status_read(True, s) == nk.STATUS_FRONTIER | nk.STATUS_PAGE_RANGE
    written = sum(int((p.view(-1, a.pool.row_bytes[0]) != 0).any(1).sum()) for p in a.pool.planes[1][:1])
    assert written == 2 * (3 + 1)                             # row 0 whole, row 1 its first token
    assert torch.all(a.q_out[1, 1:] == 9) and torch.all(a.q_out[2] == 9) and torch.all(a.q_out[4] == 9)
    assert not torch.any(a.q_out[3] == 9)                     # its queries do not need the page


def test_append_rope_position_past_the_table_is_skipped():
    a = Appended("bf16", 64, 2, 1, 4, [510], S=600, rd=64)
    a.run()
    assert not torch.any(a.q_out[0, :2] == 9) and torch.all(a.q_out[0, 2:] == 9)
    nk.nk_status_read(True, torch.cuda.current_stream().cuda_stream)


def test_append_rope_refusals():
    a = Appended("bf16", 64, 2, 1, 4, [0], rd=64)
    p, d = a.pool, a.d
    args = lambda **k: dict(dict(layer=0, tables=d["tables"], table_rows=d["rows"], write_pos=d["at"], k=a.k, v=a.v,  # noqa: E731
                                 rope=a.rope, q=a.q), **k)
    with pytest.raises(nk.NkError):
        p.append_rope(**args(layer=2))
    for bad in (dict(v=a.v[:, :2]), dict(k=a.k.float()), dict(q=a.q[:, :3]), dict(table_rows=d["rows"].long()),
                dict(tables=d["tables"][:, :2]), dict(q=None, q_out=a.q_out), dict(q_out=a.q_out[:, :2]),
                dict(k=a.k.new_zeros((1, 4, 1, 128))[..., ::2])):
        with pytest.raises(ValueError):
            p.append_rope(**args(**bad))
    p.append_rope(**args(k=a.k.transpose(2, 3).contiguous().transpose(2, 3)))   # the stride of one head says nothing
    odd = torch.zeros(4 * 68, dtype=torch.bfloat16, device=DEV)[4:260].view(1, 4, 1, 64)   # 8-byte aligned base
    with pytest.raises(nk.NkError):
        p.append_rope(**args(k=odd))
