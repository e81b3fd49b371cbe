"""Measured cases of the operators around the paged cache, with their plain forms.

Four operators of one serving step over the typed growing KV pool:

* ``norm_rope``  per-head RMS norm of queries and keys with the position
                 rotation in the same pass (``nk.qk_norm_rope``);
* ``append``     append of keys and values to the paged cache with the norm and
                 the rotation applied on the way, and the step's queries
                 rotated in the same pass (``Pool.append_rope``);
* ``shared``     decode / verify attention of a batch whose rows share a long
                 prefix of pages, the prefix attended once for all rows
                 (``Pool.shared_decode``);
* ``verify``     verification of drafted tokens against the target's
                 probabilities from given random numbers (``nk.verify_drafts``).

``run`` computes the plain form in elementary torch operations, or calls the
library when ``own`` is true.  ``exact`` computes the definition in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
P = 64
PROFILES = ("bf16", "int8_g64", "fp8_row", "nvfp4_g16", "k8v4")
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
#: (query heads, KV heads, head_dim) of the workloads and tests of this library
HEADS = ((8, 2, 128), (16, 2, 256), (32, 4, 128), (4, 4, 64), (12, 2, 64), (16, 4, 128), (20, 4, 128))


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of a full compact batch: 8 tokens, latency
        dict(name="norm_rope_step", op="norm_rope", N=8, Hq=16, H=2, D=256, rd=64, pairs=False, norm=True, fused=True),
        # a prefill chunk of the chunked-prefill workload's heads, whole-head rotation
        dict(name="norm_rope_chunk", op="norm_rope", N=2048, Hq=16, H=2, D=256, rd=256, pairs=False, norm=True,
             fused=True),
        # a long prompt in one pass, odd length, interleaved pairs, separate q and k tensors
        dict(name="norm_rope_prompt", op="norm_rope", N=32749, Hq=32, H=4, D=128, rd=128, pairs=True, norm=True,
             fused=False),
        # decode step into FP8-row pages
        dict(name="append_step_fp8", op="append", profile="fp8_row", B=8, T=1, Hq=16, H=2, D=256, rd=64, pairs=False,
             norm=True, ragged=False),
        # 4-token verify step into BF16 pages, rotation without norm
        dict(name="append_verify_bf16", op="append", profile="bf16", B=8, T=4, Hq=32, H=4, D=128, rd=128, pairs=False,
             norm=False, ragged=False),
        # ragged prefill chunks of the whole batch into FP8-row pages
        dict(name="append_chunk_fp8", op="append", profile="fp8_row", B=8, T=2048, Hq=16, H=2, D=256, rd=256,
             pairs=False, norm=True, ragged=True),
        # a short system prompt under four rows: the smallest shared call, latency
        dict(name="shared_small_bf16", op="shared", profile="bf16", B=4, T=1, Hq=8, H=2, D=128, pages=32, private=100),
        # FP8-row pages, 32768 tokens of capacity, most of it shared
        dict(name="shared_fp8", op="shared", profile="fp8_row", B=8, T=1, Hq=16, H=2, D=256, pages=480, private=2000),
        # long documents: 131072 tokens, 4-token verify, K8V4 pages
        dict(name="shared_verify_k8v4", op="shared", profile="k8v4", B=8, T=4, Hq=32, H=4, D=128, pages=1920,
             private=8000),
        # one request, three drafts
        dict(name="verify_one", op="verify", B=1, K=3, V=32768, draft=True),
        # the full compact batch, four drafts
        dict(name="verify_batch", op="verify", B=8, K=4, V=131072, draft=True),
        # many requests of several pools at once, odd vocabulary
        dict(name="verify_many", op="verify", B=64, K=7, V=200003, draft=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm_rope", "append", "shared", "verify"))
    if op == "verify":
        V = _log_int(rng, 1000, 200003)
        return dict(op=op, B=_log_int(rng, 1, 64), K=rng.randint(1, 7), V=V, draft=rng.random() < 0.8)
    Hq, H, D = rng.choice(HEADS)
    rd = rng.choice((D, D, D // 2, D // 4, 48))
    if op == "norm_rope":
        top = 32749 * 36 * 128 // ((Hq + H) * D)
        return dict(op=op, N=_log_int(rng, 1, min(top, 32749)), Hq=Hq, H=H, D=D, rd=rd, pairs=rng.random() < 0.5,
                    norm=rng.random() < 0.7, fused=rng.random() < 0.7)
    if op == "append":
        top = 2048 * 8 * 20 * 256 // (8 * (Hq + 2 * H) * D)
        return dict(op=op, profile=rng.choice(("bf16", "fp8_row")), B=rng.randint(1, 8),
                    T=_log_int(rng, 1, min(top, 2048)), Hq=Hq, H=H, D=D, rd=rd, pairs=rng.random() < 0.5,
                    norm=rng.random() < 0.7, ragged=rng.random() < 0.5)
    B, T = rng.randint(2, 8), rng.choice((1, 1, 2, 4))
    T = T if T * (Hq // H) <= (32 if D < 256 else 16) else 1
    return dict(op=op, profile=rng.choice(PROFILES), B=B, T=T, Hq=Hq, H=H, D=D,
                pages=_log_int(rng, 4, 1600 if D < 256 else 480), private=_log_int(rng, T, 4000))


# ------------------------------------------------ what a case fixes without a seed

def _counts(c):
    """Valid tokens of each row of an append."""
    B, T = c["B"], c["T"]
    return [max(1, T - (b * T) // (3 * B)) if c["ragged"] else T for b in range(B)]


def _frontiers(c):
    """Valid tokens of each row of a shared call: the shared pages and a private tail of its own length."""
    return [P * c["pages"] + max(c["T"], c["private"] - (37 * b) % max(1, c["private"] // 2)) for b in range(c["B"])]


def _row_bytes(profile, D):
    fp8, nv = D + 2, D // 2 + D // 16
    return {"bf16": 4 * D, "int8_g64": 2 * (D + 2 * (D // 64)), "fp8_row": 2 * fp8, "nvfp4_g16": 2 * nv,
            "k8v4": fp8 + nv}[profile]


def work(c):
    if c["op"] == "norm_rope":
        n = c["N"] * (c["Hq"] + c["H"]) * c["D"]
        return {"bytes": 4 * n + c["N"] * (4 * c["rd"] + 4), "flops": 7 * n}
    if c["op"] == "append":
        n, D = sum(_counts(c)), c["D"]
        q = 4 * c["Hq"] * D
        return {"bytes": n * (q + 4 * c["H"] * D + c["H"] * _row_bytes(c["profile"], D) + 4 * c["rd"]),
                "flops": 7 * n * (c["Hq"] + 2 * c["H"]) * D}
    if c["op"] == "shared":
        F = _frontiers(c)
        tokens = P * c["pages"] + sum(f - P * c["pages"] for f in F)
        rows = c["B"] * c["T"] * c["Hq"]
        return {"bytes": tokens * c["H"] * _row_bytes(c["profile"], c["D"]) + rows * (4 * c["D"] + 4),
                "flops": 4 * c["D"] * c["Hq"] * c["T"] * sum(F)}
    # of each row one row of target probabilities and, unless every draft passed, one of draft probabilities
    n = c["B"] * c["V"]
    return {"bytes": 4 * n * (2 if c["draft"] else 1) + c["B"] * c["K"] * 16, "flops": 4 * n}


# ------------------------------------------------------------------ the inputs

def _gen(seed, stream):
    g = torch.Generator(device=DEV)
    g.manual_seed((seed * 1009 + stream) % (1 << 62))
    return g


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def _rope_inputs(c, seed, rows):
    """cos / sin table (angles in 64 bits, rounded once) and norm weights."""
    rd = c["rd"]
    inv = 1e6 ** (-torch.arange(0, rd, 2, device=DEV, dtype=torch.float64) / max(rd, 1))
    a = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * inv
    g = _gen(seed, 1)
    w = [(1 + 0.2 * torch.randn(c["D"], generator=g, device=DEV)).to(torch.bfloat16) for _ in range(2)]
    return torch.cat((a.cos(), a.sin()), 1).float().contiguous(), w if c["norm"] else [None, None]


def _qkv(c, n, g, fused, v):
    """q, k (and v) rows of a projection: views of one fused row, or tensors of their own."""
    Hq, H, D = c["Hq"], c["H"], c["D"]
    sizes = [Hq, H] + ([H] if v else [])
    if not fused:
        return [_normal((n, h, D), g) for h in sizes]
    x = _normal((n, sum(sizes), D), g)
    return list(x.split(sizes, 1))


def _tables(B, shared, need, M, L, g):
    """Block tables of B rows over a random order of the pool's pages: `shared` common ones, then each row's own."""
    perm = torch.randperm(M, generator=g, device=DEV).to(torch.int32)
    t = torch.zeros((B, L), dtype=torch.int32, device=DEV)
    t[:, :shared] = perm[:shared]
    t[:, shared:shared + need] = perm[shared:shared + B * need].view(B, need)
    return t


def _planes(profile, M, H, D):
    widths = {"bf16": [2 * D] * 2, "int8_g64": [D, D, D // 32, D // 32], "fp8_row": [D, D, 2, 2],
              "nvfp4_g16": [D // 2] * 2 + [D // 16] * 2, "k8v4": [D, D // 2, 2, D // 16]}[profile]
    return [torch.zeros(M * H * P * w, dtype=torch.uint8, device=DEV) for w in widths]


def _kinds(profile):
    return {"bf16": ("bf16",) * 2, "int8_g64": ("int8",) * 2, "fp8_row": ("fp8",) * 2, "nvfp4_g16": ("nv",) * 2,
            "k8v4": ("fp8", "nv")}[profile]


def _stored(kind, x):
    """Codes and scales (bytes) of values x [..., D]."""
    x, D = x.float(), x.shape[-1]
    if kind == "bf16":
        return x.to(torch.bfloat16).view(torch.uint8), None
    if kind == "fp8":
        s = (x.abs().amax(-1, keepdim=True) / 448).clamp(max=65504).half()
        sf = s.float()
        c = torch.where(sf > 0, x / sf, 0.0).clamp(-448, 448).to(torch.float8_e4m3fn)
        return c.view(torch.uint8), s.view(torch.uint8)
    if kind == "int8":
        g = x.unflatten(-1, (D // 64, 64))
        s = (g.abs().amax(-1) / 127).clamp(max=65504).half()
        sf = s.float().unsqueeze(-1)
        c = torch.where(sf > 0, g / sf, 0.0).round().clamp(-127, 127).to(torch.int8)
        return c.flatten(-2).view(torch.uint8), s.view(torch.uint8)
    g = x.unflatten(-1, (D // 16, 16))
    s = (g.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    sf = s.float().unsqueeze(-1)
    v = torch.where(sf > 0, g / sf, 0.0).flatten(-2)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = torch.bucketize(v.abs(), edges).to(torch.uint8) + 8 * (v < 0).to(torch.uint8)
    return code[..., 0::2] + 16 * code[..., 1::2], s.view(torch.uint8)


def _values(kind, codes, scales, D, dtype=torch.float32):
    """The values that code rows and scale rows (bytes, [..., row bytes]) stand for."""
    if kind == "bf16":
        return codes.view(torch.bfloat16).to(dtype)
    if kind == "fp8":
        return codes.view(torch.float8_e4m3fn).to(dtype) * scales.view(torch.float16).to(dtype)
    if kind == "int8":
        s = scales.view(torch.float16).to(dtype).unsqueeze(-1)
        return (codes.view(torch.int8).to(dtype).unflatten(-1, (D // 64, 64)) * s).flatten(-2)
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device, dtype=dtype)
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).to(dtype).unsqueeze(-1)
    return (v.unflatten(-1, (D // 16, 16)) * s).flatten(-2)


def _pool(c, M, S, C):
    """The planes, and the library's pool over planes of its own where it runs."""
    if not own:
        return None, _planes(c["profile"], M, c["H"], c["D"])
    from paged_kv_cache_append_gb300 import nk
    pool = nk.Pool(c["profile"], 1, c["H"], c["D"], S, C, M)
    return pool, pool.planes[0]


def _rope(c, table, w):
    if not own:
        return None
    from paged_kv_cache_append_gb300 import nk
    return nk.Rope(table, c["rd"], interleaved=c["pairs"], q_weight=w[0], k_weight=w[1], eps=1e-6)


def prepare(c, seed):
    g = _gen(seed, 0)
    st = {"c": c}
    if c["op"] == "norm_rope":
        N = c["N"]
        st["table"], st["w"] = _rope_inputs(c, seed, 65536)
        st["q"], st["k"] = _qkv(c, N, g, c["fused"], True)[:2]
        start = int(torch.randint(0, 65536 - N, (1,), generator=g, device=DEV))
        st["pos"] = torch.arange(start, start + N, dtype=torch.int32, device=DEV)
        st["q_out"] = torch.zeros((N, c["Hq"], c["D"]), dtype=torch.bfloat16, device=DEV)
        st["k_out"] = torch.zeros((N, c["H"], c["D"]), dtype=torch.bfloat16, device=DEV)
        st["rope"] = _rope(c, st["table"], st["w"])
    elif c["op"] == "append":
        B, T, H, D = c["B"], c["T"], c["H"], c["D"]
        L = -(-(T + 1000) // P)
        M = max(B * L, B)
        st["pool"], st["planes"] = _pool(c, M, L * P, B)
        st["table"], st["w"] = _rope_inputs(c, seed, L * P)
        q, k, v = _qkv(c, B * T, g, True, True)
        st["q"], st["k"], st["v"] = (x.unflatten(0, (B, T)) for x in (q, k, v))
        st["tables"] = _tables(B, 0, L, M, L, g)
        st["rows"] = torch.arange(B, dtype=torch.int32, device=DEV)
        st["at"] = torch.randint(0, 1000, (B,), generator=g, device=DEV).to(torch.int32)
        st["counts"] = torch.tensor(_counts(c), dtype=torch.int32, device=DEV)
        st["q_out"] = torch.zeros((B, T, c["Hq"], D), dtype=torch.bfloat16, device=DEV)
        st["rope"] = _rope(c, st["table"], st["w"])
    elif c["op"] == "shared":
        B, T, H, D, n = c["B"], c["T"], c["H"], c["D"], c["pages"]
        F = _frontiers(c)
        L = -(-max(F) // P)
        M = max(n + B * (L - n), L, B)
        st["pool"], st["planes"] = _pool(c, M, L * P, B)
        kinds = _kinds(c["profile"])
        for i, kind in enumerate(kinds):
            codes, scales = _stored(kind, _normal((M, H, P, D), g))
            st["planes"][i].copy_(codes.reshape(-1))
            if scales is not None:
                st["planes"][2 + i].copy_(scales.reshape(-1))
        st["tables"] = _tables(B, n, L - n, M, L, g)
        st["rows"] = torch.arange(B, dtype=torch.int32, device=DEV)
        st["frontiers"] = torch.tensor(F, dtype=torch.int32, device=DEV)
        st["shared"] = torch.tensor([n], dtype=torch.int32, device=DEV)
        st["q"] = _normal((B, T, c["Hq"], D), g)
        st["scale"] = 1 / math.sqrt(D)
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros((B, T, c["Hq"]), dtype=torch.float32, device=DEV)
        if own:
            st["ws"] = st["pool"].shared_workspace(B, T, c["Hq"])
    else:
        B, K, V = c["B"], c["K"], c["V"]
        z = torch.empty((B, K + 1, V), device=DEV).normal_(0, 3, generator=g)
        zq = z[:, :K] + torch.empty((B, K, V), device=DEV).normal_(0, 0.4, generator=g)
        st["target"] = z.softmax(-1)
        dq = zq.softmax(-1)
        # a draft from the draft model's distribution (the greedy one where no distribution is kept)
        e = torch.empty((B, K, V), device=DEV).exponential_(generator=g)
        st["tokens"] = ((dq / e) if c["draft"] else dq).argmax(-1).to(torch.int32)
        st["draft"] = dq if c["draft"] else None
        st["len"] = torch.tensor([K - (b % 3 == 2) * min(K, 2) for b in range(B)], dtype=torch.int32, device=DEV)
        st["u"] = torch.rand((B, K + 1), generator=g, device=DEV)
        st["frontiers"] = torch.randint(K + 1, 100000, (B,), generator=g, device=DEV).to(torch.int32)
    return st


# ------------------------------------------------------------------ plain forms

def _normed_rotated(x, w, table, pos, c):
    """x [N, heads, D] -> fp32, normed (w not None) and rotated by the table rows of pos [N]."""
    x, rd = x.float(), c["rd"]
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    cs = table[pos.long()].unsqueeze(-2)
    cos, sin = cs[..., :rd // 2], cs[..., rd // 2:]
    y = x.clone()
    if c["pairs"]:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y[..., 0:rd:2], y[..., 1:rd:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rd // 2], x[..., rd // 2:rd]
        y[..., :rd // 2], y[..., rd // 2:rd] = a * cos - b * sin, b * cos + a * sin
    return y


def _plane_outputs(profile, planes, M, H, D):
    """The planes as the types they hold: BF16 values, or E4M3 codes and binary16 scales."""
    if profile == "bf16":
        return [p.view(torch.bfloat16).view(M, H, P, D) for p in planes]
    return ([p.view(torch.float8_e4m3fn).view(M, H, P, D) for p in planes[:2]] +
            [p.view(torch.float16).view(M, H, P) for p in planes[2:]])


def _live(st):
    """(row, token) of every valid token of an append, its position, page group and page offset."""
    c = st["c"]
    t = torch.arange(c["T"], device=DEV)
    live = t[None] < st["counts"][:, None]
    b, t = live.nonzero(as_tuple=True)
    pos = st["at"].long()[b] + t
    return b, t, pos, st["tables"][b, pos // P].long(), pos % P


def run(st):
    c = st["c"]
    if c["op"] == "norm_rope":
        if own:
            from paged_kv_cache_append_gb300 import nk
            return nk.qk_norm_rope(st["q"], st["k"], st["pos"], st["rope"], q_out=st["q_out"], k_out=st["k_out"])
        return [_normed_rotated(st[n], w, st["table"], st["pos"], c).to(torch.bfloat16)
                for n, w in zip(("q", "k"), st["w"])]
    if c["op"] == "append":
        M, H, D = st["planes"][0].numel() // (c["H"] * P * c["D"] * (2 if c["profile"] == "bf16" else 1)), c["H"], c["D"]
        if own:
            st["pool"].append_rope(0, st["tables"], st["rows"], st["at"], st["k"], st["v"], st["rope"], q=st["q"],
                                   q_out=st["q_out"], counts=st["counts"])
            return [st["q_out"]] + _plane_outputs(c["profile"], st["planes"], M, H, D)
        b, t, pos, g, o = _live(st)
        st["q_out"][b, t] = _normed_rotated(st["q"][b, t], st["w"][0], st["table"], pos, c).to(torch.bfloat16)
        k = _normed_rotated(st["k"][b, t], st["w"][1], st["table"], pos, c)
        for i, x in enumerate((k, st["v"][b, t])):
            codes, scales = _stored(_kinds(c["profile"])[i], x)
            st["planes"][i].view(M, H, P, -1)[g, :, o] = codes
            if scales is not None:
                st["planes"][2 + i].view(M, H, P, -1)[g, :, o] = scales
        return [st["q_out"]] + _plane_outputs(c["profile"], st["planes"], M, H, D)
    if c["op"] == "shared":
        if own:
            return st["pool"].shared_decode(0, st["q"], st["tables"], st["rows"], st["frontiers"], st["shared"],
                                            st["scale"], out=st["out"], lse=st["lse"], workspace=st["ws"])
        return _shared_plain(st)
    if own:
        from paged_kv_cache_append_gb300 import nk
        return nk.verify_drafts(st["target"], st["tokens"], st["u"], draft=st["draft"], draft_len=st["len"],
                                frontiers=st["frontiers"])
    return _verify_plain(st)


def _page_values(st, side, pages):
    """fp32 values [..., H, 64, D] of one side (0: K, 1: V) of page groups `pages` [...]."""
    c = st["c"]
    H, D = c["H"], c["D"]
    kind = _kinds(c["profile"])[side]
    M = _pages(st)
    codes = st["planes"][side].view(M, H, P, -1)[pages]
    scales = st["planes"][2 + side].view(M, H, P, -1)[pages] if kind != "bf16" else None
    return _values(kind, codes, scales, D)


def _pages(st):
    """Page groups of the pool."""
    c = st["c"]
    width = {"bf16": 2 * c["D"], "nv": c["D"] // 2}.get(_kinds(c["profile"])[0], c["D"])
    return st["planes"][0].numel() // (c["H"] * P * width)


def _shared_plain(st):
    c = st["c"]
    B, T, Hq, H, D, n = c["B"], c["T"], c["Hq"], c["H"], c["D"], c["pages"]
    q = st["q"].float().view(B, T, H, Hq // H, D) * st["scale"]
    pages = st["tables"].long()
    ks, vs = (_page_values(st, s, pages[0, :n]).transpose(0, 1).reshape(H, n * P, D) for s in (0, 1))
    kp, vp = (_page_values(st, s, pages[:, n:]).transpose(1, 2).reshape(B, H, -1, D) for s in (0, 1))
    zs = torch.einsum("bthgd,hkd->bthgk", q, ks)
    zp = torch.einsum("bthgd,bhkd->bthgk", q, kp)
    seen = torch.arange(kp.shape[2], device=DEV) + n * P
    last = st["frontiers"][:, None].long() - T + torch.arange(T, device=DEV)
    hidden = seen > last[..., None]
    zp = zp.masked_fill(hidden[:, :, None, None], -math.inf)
    vp = vp.masked_fill((seen >= st["frontiers"][:, None])[:, None, :, None], 0.0)
    m = torch.maximum(zs.amax(-1), zp.amax(-1)).unsqueeze(-1)
    zs, zp = (zs - m).exp_(), (zp - m).exp_()
    total = zs.sum(-1) + zp.sum(-1)
    o = torch.einsum("bthgk,hkd->bthgd", zs, vs) + torch.einsum("bthgk,bhkd->bthgd", zp, vp)
    o = (o / total.unsqueeze(-1)).to(torch.bfloat16).reshape(B, T, Hq, D)
    return [o, (m.squeeze(-1) + total.log()).reshape(B, T, Hq)]


def _verify_plain(st):
    """Sums in 64 bits: a token's probability is near the rounding of a sum in 32."""
    c = st["c"]
    B, K, V = c["B"], c["K"], c["V"]
    p, q, x, ln = st["target"], st["draft"], st["tokens"].long().unsqueeze(-1), st["len"]
    px = p[:, :K].gather(-1, x).squeeze(-1).double()
    qx = q.gather(-1, x).squeeze(-1).double() if q is not None else torch.ones_like(px)
    ok = (st["u"][:, :K].double() * qx < px) & (torch.arange(K, device=DEV) < ln[:, None])
    n = ok.int().cumprod(-1).sum(-1)
    b = torch.arange(B, device=DEV)
    d = p[b, n].double()
    cut = n < ln
    at = n.clamp(max=K - 1)
    if q is not None:
        d = torch.where(cut[:, None], d - q[b, at].double(), d).clamp(min=0)
    else:
        d[b, x[b, at, 0]] = torch.where(cut, 0.0, d[b, x[b, at, 0]])
    s = d.cumsum(-1)
    new = (s <= (st["u"][:, K].double() * s[:, -1])[:, None]).sum(-1).clamp(max=V - 1)
    i = torch.arange(K + 1, device=DEV)
    padded = torch.cat((st["tokens"], st["tokens"][:, :1]), 1)
    tokens = torch.where(i < n[:, None], padded, torch.where(i == n[:, None], new[:, None].int(), -1))
    return [n.int(), tokens.int(), st["frontiers"] - (ln - n.int())]


# ------------------------------------------------------------------ definitions

def _exact_rows(x, w, table, pos, c):
    """The norm and rotation in 64 bits, the rotation as a product of complex numbers."""
    x, h = x.double(), c["rd"] // 2
    if w is not None:
        x = x / (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / c["D"] + 1e-6).sqrt() * w.double()
    cs = table.double()[pos.long()]
    turn = torch.complex(cs[:, :h], cs[:, h:])[:, None]
    head, rest = x[..., :c["rd"]], x[..., c["rd"]:]
    if c["pairs"]:
        z = torch.view_as_complex(head.unflatten(-1, (h, 2)).contiguous()) * turn
        return torch.cat((torch.view_as_real(z).flatten(-2), rest), -1)
    z = torch.complex(head[..., :h].contiguous(), head[..., h:].contiguous()) * turn
    return torch.cat((z.real, z.imag, rest), -1)


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "norm_rope":
        return [_exact_rows(st[n], w, st["table"], st["pos"], c) for n, w in zip(("q", "k"), st["w"])]
    if c["op"] == "append":
        D, H, B = c["D"], c["H"], c["B"]
        M = st["tables"].numel()
        q_out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
        fp8 = c["profile"] == "fp8_row"
        planes = [torch.zeros((M, P, H, D), dtype=torch.float64, device=DEV) for _ in range(2)]
        scales = [torch.zeros((M, P, H), dtype=torch.float64, device=DEV) for _ in range(2)]
        for b, n in enumerate(_counts(c)):
            pos = torch.arange(n, device=DEV) + int(st["at"][b])
            q_out[b, :n] = _exact_rows(st["q"][b, :n], st["w"][0], st["table"], pos, c)
            k = _exact_rows(st["k"][b, :n], st["w"][1], st["table"], pos, c)
            flat = st["tables"][b].long()[pos >> 6] * P + (pos & 63)
            for i, x in enumerate((k, st["v"][b, :n].double())):
                if fp8:  # codes: the quotient by the stored scale, before its rounding
                    s = x.abs().amax(-1) / 448
                    scales[i].view(-1, H)[flat] = s
                    x = x / s.half().double().clamp(min=1e-300).unsqueeze(-1)
                planes[i].view(-1, H, D)[flat] = x
        return [q_out] + [p.transpose(1, 2) for p in planes] + ([s.transpose(1, 2) for s in scales] if fp8 else [])
    if c["op"] == "shared":
        B, T, Hq, H, D = c["B"], c["T"], c["Hq"], c["H"], c["D"]
        out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=DEV)
        lse = torch.zeros((B, T, Hq), dtype=torch.float64, device=DEV)
        M = _pages(st)
        kinds = _kinds(c["profile"])
        for b, F in enumerate(_frontiers(c)):
            pages = st["tables"][b].long()
            for h in range(H):  # the row's tokens in order, one KV head
                k, v = (_values(kinds[s], st["planes"][s].view(M, H, P, -1)[pages, h],
                                None if kinds[s] == "bf16" else st["planes"][2 + s].view(M, H, P, -1)[pages, h], D,
                                torch.float64).reshape(-1, D)[:F] for s in (0, 1))
                for t in range(T):
                    see = F - T + t + 1
                    hs = slice(h * (Hq // H), (h + 1) * (Hq // H))
                    z = st["q"][b, t, hs].double() @ k[:see].T * st["scale"]
                    lse[b, t, hs] = z.logsumexp(-1)
                    out[b, t, hs] = z.softmax(-1) @ v[:see]
        return [out, lse]
    return _exact_verify(c, st)


def _exact_verify(c, st):
    K, V = c["K"], c["V"]
    ns, rows = [], []
    u, ln, drafts = st["u"].double().cpu(), st["len"].tolist(), st["tokens"].tolist()
    for b in range(c["B"]):
        p, n = st["target"][b].double(), 0
        q = st["draft"][b].double() if st["draft"] is not None else None
        while n < ln[b]:
            x = drafts[b][n]
            if not float(u[b, n]) * (1.0 if q is None else float(q[n, x])) < float(p[n, x]):
                break
            n += 1
        d = p[n].clone()
        if n < ln[b] and q is not None:
            d = torch.relu(d - q[n])
        elif n < ln[b]:
            d[drafts[b][n]] = 0
        s = d.cumsum(0)
        new = int(torch.searchsorted(s, float(u[b, K]) * s[-1], right=True))
        ns.append(n)
        rows.append(drafts[b][:n] + [min(new, V - 1)] + [-1] * (K - n))
    as_int = dict(dtype=torch.int32, device=DEV)
    n = torch.tensor(ns, **as_int)
    return [n, torch.tensor(rows, **as_int), st["frontiers"] - torch.tensor(ln, **as_int) + n]
