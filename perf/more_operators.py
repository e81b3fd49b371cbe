"""Measured cases of a differential-attention layer over the paged cache, with their plain forms.

Four operators of a serving step over the typed growing KV pool:

* ``grow``     block tables, frontiers, positions and slot maps of a step from
               the requests' lengths, pages taken from and returned to a stack
               of free pages (``Pool.grow``);
* ``decode``   differential attention of decode / verify tokens over the pages:
               per head the difference of two softmax maps over values of twice
               the head size, with its norm (``Pool.diff_decode``);
* ``prefill``  the same for chunks of prompts (``Pool.diff_prefill``);
* ``norm``     the norms before and after a block with its gate and the scales
               of the residual (``nk.residual_norm``).

``run`` computes the plain form in elementary torch operations, or calls the
library when ``own`` is true.  ``exact`` computes the definition in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
P = 64
EPS = 1e-5
PROFILES = ("bf16", "int8_g64", "fp8_row", "nvfp4_g16", "k8v4")
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
#: (query heads, KV heads, head_dim) of the workloads and tests of this library, heads of 64 and 128
HEADS = ((8, 2, 128), (32, 4, 128), (4, 4, 64), (12, 2, 64), (16, 4, 128), (20, 4, 128))
#: what a drawn case may cost at most: that of the largest listed one
DECODE_BYTES = 8 * 131072 * 4 * 202
PREFILL_PAIRS = 4 * (16384 * 2048 + 1024 * 2049) * 16 * 128


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one speculative step of a full compact batch: a page or none for each row, four slots a row
        dict(name="grow_step", op="grow", B=8, T=4, S=131072, fresh=False),
        # eight long prompts admitted at once: most of the pool's pages, a slot for every token
        dict(name="grow_prompts", op="grow", B=8, T=131072, S=131072, fresh=True),
        # one request, one token, a short context: latency
        dict(name="decode_one_bf16", op="decode", profile="bf16", B=1, T=1, Hq=8, H=2, D=128, context=1000),
        # a full batch of ordinary contexts, small heads, INT8 pages
        dict(name="decode_batch_int8", op="decode", profile="int8_g64", B=8, T=1, Hq=12, H=2, D=64, context=4096),
        # long contexts in FP8-row pages
        dict(name="decode_long_fp8", op="decode", profile="fp8_row", B=8, T=1, Hq=16, H=4, D=128, context=32768),
        # the long-document workload: 131072 tokens a row, 4-token verify, K8V4 pages
        dict(name="decode_verify_k8v4", op="decode", profile="k8v4", B=8, T=4, Hq=32, H=4, D=128, context=131072),
        # a short first prompt, odd length, heads without groups
        dict(name="prefill_short_bf16", op="prefill", profile="bf16", B=1, T=501, Hq=4, H=4, D=64, prefix=0),
        # a chunk of a long prompt into BF16 pages
        dict(name="prefill_chunk_bf16", op="prefill", profile="bf16", B=1, T=2048, Hq=16, H=4, D=128, prefix=8150),
        # ragged chunks of four rows deep into long prompts, K8V4 pages
        dict(name="prefill_batch_k8v4", op="prefill", profile="k8v4", B=4, T=2048, Hq=16, H=4, D=128, prefix=16384),
        # one decode step of a full compact batch
        dict(name="norm_step", op="norm", N=8, dim=4096, gate="none", act=False, post=False, wide=False),
        # a prefill chunk with a gate of its own for each token
        dict(name="norm_chunk", op="norm", N=2048, dim=4096, gate="token", act=True, post=True, wide=False),
        # a long prompt in one pass, odd length, the residual stream in fp32
        dict(name="norm_prompt", op="norm", N=32749, dim=2560, gate="channel", act=False, post=True, wide=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(("grow", "decode", "decode", "prefill", "prefill", "norm"))
    if op == "grow":
        S = 64 * _log_int(rng, 4, 2048) - rng.choice((0, 0, 7))
        return dict(op=op, B=rng.randint(1, 8), T=_log_int(rng, 1, S), S=S, fresh=rng.random() < 0.5)
    if op == "norm":
        dim = 8 * _log_int(rng, 8, 2048)
        return dict(op=op, N=_log_int(rng, 1, min(32749, 32749 * 2560 // dim)), dim=dim,
                    gate=rng.choice(("none", "token", "channel")), act=rng.random() < 0.5, post=rng.random() < 0.5,
                    wide=rng.random() < 0.5)
    Hq, H, D = rng.choice(HEADS)
    profile = rng.choice(PROFILES)
    if op == "decode":
        B, T = rng.randint(1, 8), rng.choice((1, 1, 2, 3, 4))
        top = DECODE_BYTES // (B * H * _row_bytes(profile, D))
        return dict(op=op, profile=profile, B=B, T=T, Hq=Hq, H=H, D=D, context=_log_int(rng, T, min(131072, top)))
    B, T = rng.randint(1, 4), _log_int(rng, 1, 2048)
    top = PREFILL_PAIRS // (B * T * Hq * D) - T
    return dict(op=op, profile=profile, B=B, T=T, Hq=Hq, H=H, D=D, prefix=_log_int(rng, 1, max(1, min(16384, top))) - 1)


# ------------------------------------------------ what a case fixes without a seed

def _contexts(c):
    """Valid tokens of each row of a decode call, its own new ones among them."""
    return [max(c["T"], c["context"] - (37 * b + b * c["context"] // 16) % max(1, c["context"] // 2))
            for b in range(c["B"])]


def _chunks(c):
    """(prefix, chunk) of each row of a prefill call."""
    return [(c["prefix"] - (41 * b) % (c["prefix"] // 2 + 1), max(1, c["T"] - (b * c["T"]) // 9)) for b in range(c["B"])]


def _lengths(c):
    """(committed tokens, new tokens, mapped pages) of each row of a growing step.

    Fresh rows start empty.  The others hold committed tokens, and every third
    of them still maps pages of a provisional lead that has to be returned."""
    out = []
    for b in range(c["B"]):
        new = max(1, c["T"] - (b * c["T"]) // (2 * c["B"]))
        if c["fresh"]:
            out.append((0, new, 0))
            continue
        room = c["S"] - new
        have = (room * (2 * b + 3)) // (2 * c["B"] + 4)
        mapped = -(-have // P)
        if b % 3 == 1:
            mapped = min(-(-c["S"] // P), mapped + 5)
        out.append((have, new, mapped))
    return out


def _row_bytes(profile, D):
    fp8, nv = D + 2, D // 2 + D // 16
    return {"bf16": 4 * D, "int8_g64": 2 * (D + 2 * (D // 64)), "fp8_row": 2 * fp8, "nvfp4_g16": 2 * nv,
            "k8v4": fp8 + nv}[profile]


def work(c):
    if c["op"] == "grow":
        moved = sum(abs(-(-(have + new) // P) - mapped) for have, new, mapped in _lengths(c))
        # a position (4 bytes) and a slot (8) for each token of the batch's rows, page ids read and written
        return {"bytes": 12 * c["B"] * c["T"] + 8 * moved + 24 * c["B"], "flops": 4 * c["B"] * c["T"]}
    if c["op"] == "norm":
        n = c["N"] * c["dim"]
        r = 4 if c["wide"] else 2
        gate = {"none": 0, "token": 2 * n, "channel": 2 * c["dim"]}[c["gate"]]
        return {"bytes": n * (4 + 2 * r) + gate, "flops": 12 * n}
    row = c["H"] * _row_bytes(c["profile"], c["D"])
    if c["op"] == "decode":
        tokens = sum(_contexts(c))
        q = c["B"] * c["T"] * c["Hq"]
        return {"bytes": tokens * row + q * (4 * c["D"] + 4), "flops": 6 * c["D"] * c["Hq"] * c["T"] * tokens}
    chunks = _chunks(c)
    pairs = sum(p * n + n * (n + 1) // 2 for p, n in chunks)
    return {"bytes": sum(p + n for p, n in chunks) * row + sum(n for _, n in chunks) * c["Hq"] * (4 * c["D"] + 4),
            "flops": 6 * c["D"] * c["Hq"] * pairs}


# ------------------------------------------------------------------ the inputs

def _gen(seed, stream):
    g = torch.Generator(device=DEV)
    g.manual_seed((seed * 1009 + stream) % (1 << 62))
    return g


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


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
    code = torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8) + 8 * (v < 0).to(torch.uint8)
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


def _attention_inputs(c, st, g, lengths):
    """A pool whose pages hold keys and values, tables over a random order of them, queries, lambda and the norm."""
    B, T, Hq, H, D = c["B"], c["T"], c["Hq"], c["H"], c["D"]
    L = -(-max(lengths) // P)
    M = B * L
    if own:
        from paged_kv_cache_append_gb300 import nk
        st["pool"] = nk.Pool(c["profile"], 1, H, D, L * P, B, M)
        st["planes"] = st["pool"].planes[0]
    else:
        st["planes"] = _planes(c["profile"], M, H, D)
    for side, kind in enumerate(_kinds(c["profile"])):
        for lo in range(0, M, 2048):  # by 2048 pages, to hold few of them in fp32 at once
            n = min(2048, M - lo)
            codes, scales = _stored(kind, _normal((n, H, P, D), g))
            for plane, x in ((st["planes"][side], codes), (st["planes"][2 + side] if scales is not None else None, scales)):
                if x is not None:
                    w = x.numel() // n
                    plane[lo * w:(lo + n) * w].copy_(x.reshape(-1))
    st["tables"] = torch.randperm(M, generator=g, device=DEV).to(torch.int32).view(B, L)
    st["rows"] = torch.arange(B, dtype=torch.int32, device=DEV)
    st["q"] = _normal((B, T, Hq, D), g)
    st["scale"] = 1 / math.sqrt(D)
    st["lam"] = 0.1 + 0.7 * torch.rand(Hq // 2, generator=g, device=DEV)
    st["weight"] = (1 + 0.2 * torch.randn(2 * D, generator=g, device=DEV)).to(torch.bfloat16)
    st["out_scale"] = 0.2
    st["out"] = torch.zeros((B, T, Hq // 2, 2 * D), dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.full((B, T, Hq), -math.inf, dtype=torch.float32, device=DEV)
    if own:
        from paged_kv_cache_append_gb300 import nk
        st["diff"] = nk.Diff(st["lam"], st["weight"], eps=EPS, out_scale=st["out_scale"])


def prepare(c, seed):
    g = _gen(seed, 0)
    st = {"c": c}
    if c["op"] == "grow":
        B, S = c["B"], c["S"]
        L = -(-S // P)
        lengths = _lengths(c)
        st["committed"], st["counts"], mapped = (_ints(list(x)) for x in zip(*lengths))
        used = [x[2] for x in lengths]
        perm = torch.randperm(B * L, generator=g, device=DEV).to(torch.int32)
        rows = torch.randperm(B, generator=g, device=DEV)
        st["rows"] = rows.to(torch.int32)
        st["tables"] = torch.full((B, L), -1, dtype=torch.int32, device=DEV)
        st["mapped"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        st["mapped"][rows] = mapped
        for b, (row, n) in enumerate(zip(rows.tolist(), used)):
            st["tables"][row, :n] = perm[sum(used[:b]):sum(used[:b + 1])]
        free = sum(used)
        st["free"] = torch.full((B * L,), -1, dtype=torch.int32, device=DEV)
        st["free"][:B * L - free] = perm[free:]
        st["n_free"] = _ints([B * L - free])
        if own:
            from paged_kv_cache_append_gb300 import nk
            st["pool"] = nk.Pool("nvfp4_g16", 1, 1, 64, S, B, B * L)
            st["after"] = (torch.zeros_like(st["mapped"]), torch.zeros_like(st["n_free"]))
            st["outs"] = (torch.zeros_like(st["committed"]),
                          torch.zeros((B, c["T"]), dtype=torch.int32, device=DEV),
                          torch.zeros((B, c["T"]), dtype=torch.int64, device=DEV))
    elif c["op"] == "decode":
        F = _contexts(c)
        _attention_inputs(c, st, g, F)
        st["frontiers"] = _ints(F)
        if own:
            st["ws"] = st["pool"].diff_decode_workspace(c["B"], c["T"], c["Hq"])
    elif c["op"] == "prefill":
        chunks = _chunks(c)
        _attention_inputs(c, st, g, [p + n for p, n in chunks])
        st["prefix"], st["chunk"] = (_ints(list(x)) for x in zip(*chunks))
        if own:
            st["ws"] = st["pool"].diff_prefill_workspace(c["B"], c["T"], c["Hq"])
    else:
        N, dim = c["N"], c["dim"]
        st["y"] = _normal((N, dim), g)
        st["res"] = torch.randn((N, dim), generator=g, device=DEV) * 3
        if not c["wide"]:
            st["res"] = st["res"].to(torch.bfloat16)
        st["gate"] = {"none": None, "token": (N, dim), "channel": (dim,)}[c["gate"]]
        if st["gate"] is not None:
            st["gate"] = _normal(st["gate"], g)
        st["w"] = (1 + 0.2 * torch.randn(dim, generator=g, device=DEV)).to(torch.bfloat16)
        st["post"] = (1 + 0.2 * torch.randn(dim, generator=g, device=DEV)).to(torch.bfloat16) if c["post"] else None
        st["scales"] = (0.7, 1.25)  # of the block's output, of the residual
        st["x_out"], st["res_out"] = torch.zeros_like(st["y"]), torch.zeros_like(st["res"])
        if own:
            from paged_kv_cache_append_gb300 import nk
            st["norm"] = nk.ResidualNorm(st["w"], post_weight=st["post"], eps=EPS, scale=st["scales"][0],
                                         residual_scale=st["scales"][1], sigmoid_gate=c["act"])
    return st


# ------------------------------------------------------------------ plain forms

def run(st):
    c = st["c"]
    if c["op"] == "grow":
        if own:
            out = st["pool"].grow(st["tables"], st["rows"], st["committed"], st["mapped"], st["free"], st["n_free"],
                                  c["T"], counts=st["counts"], mapped_out=st["after"][0], free_count_out=st["after"][1],
                                  frontiers=st["outs"][0], positions=st["outs"][1], slots=st["outs"][2])
            return [st["tables"], st["after"][0], st["free"], st["after"][1], *out]
        return _grow_plain(st)
    if c["op"] == "decode":
        if own:
            return st["pool"].diff_decode(0, st["q"], st["tables"], st["rows"], st["frontiers"], st["scale"], st["diff"],
                                          out=st["out"], lse=st["lse"], workspace=st["ws"])
        F = _contexts(c)
        rows = [_attend(st, b, f, f - c["T"], c["T"]) for b, f in enumerate(F)]
        return [torch.stack([r[i] for r in rows]) for i in (0, 1)]
    if c["op"] == "prefill":
        if own:
            return st["pool"].diff_prefill(0, st["q"], st["tables"], st["rows"], st["prefix"], st["chunk"], st["scale"],
                                           st["diff"], out=st["out"], lse=st["lse"], workspace=st["ws"])
        for b, (prefix, n) in enumerate(_chunks(c)):
            st["out"][b, :n], st["lse"][b, :n] = _attend(st, b, prefix + n, prefix, n)
        return [st["out"], st["lse"]]
    if own:
        from paged_kv_cache_append_gb300 import nk
        return nk.residual_norm(st["y"], st["res"], st["norm"], gate=st["gate"], out=st["x_out"],
                                residual_out=st["res_out"])
    return _norm_plain(st)


def _grow_plain(st):
    """Row by row over the batch: first what goes back to the stack, last row first, then what is taken, first row first."""
    c = st["c"]
    B, T = c["B"], c["T"]
    rows = st["rows"].long()
    frontiers = st["committed"] + st["counts"]
    need = (frontiers + (P - 1)) // P
    have = st["mapped"][rows]
    tables, free = st["tables"], st["free"]
    page = torch.arange(tables.shape[1], device=DEV)
    top = st["n_free"][0].long()
    for b in reversed(range(B)):
        gone = (page >= need[b]) & (page < have[b])
        at = top + (have[b] - 1 - page)
        pad = torch.cat((free, free[:1]))  # pages that stay are sent behind the stack
        free[:] = pad.scatter_(0, torch.where(gone, at, free.numel()), tables[rows[b]])[:-1]
        top = top + (have[b] - need[b]).clamp(min=0)
    for b in range(B):
        new = (page >= have[b]) & (page < need[b])
        at = (top - 1 - (page - have[b])).clamp(0, free.numel() - 1)
        tables[rows[b]] = torch.where(new, free[at], tables[rows[b]])
        top = top - (need[b] - have[b]).clamp(min=0)
    mapped = st["mapped"].clone()
    mapped[rows] = need
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    live = t < st["counts"][:, None]
    positions = torch.where(live, st["committed"][:, None] + t, -1)
    pages = tables[rows].long().gather(1, (positions // P).clamp(min=0).long())
    slots = torch.where(live, pages * P + positions % P, -1)
    return [tables, mapped, free, top.to(torch.int32).view(1), frontiers, positions, slots]


def _keys_values(st, b, F, dtype=torch.float32):
    """[H, F, D] keys and values of row b's first F tokens."""
    c = st["c"]
    H, D = c["H"], c["D"]
    M = st["tables"].numel()
    pages = st["tables"][b, :-(-F // P)].long()
    out = []
    for side, kind in enumerate(_kinds(c["profile"])):
        codes = st["planes"][side].view(M, H, P, -1)[pages]
        scales = st["planes"][2 + side].view(M, H, P, -1)[pages] if kind != "bf16" else None
        out.append(_values(kind, codes, scales, D, dtype).transpose(0, 1).reshape(H, -1, D)[:, :F])
    return out


def _attend(st, b, F, first, n):
    """Differential attention of row b's queries 0 .. n - 1, at positions from `first` on, over its F tokens."""
    c = st["c"]
    Hq, H, D = c["Hq"], c["H"], c["D"]
    heads, per = Hq // 2, Hq // H  # differential heads, heads that share a pair of KV heads
    k, v = _keys_values(st, b, F)
    v = v.unflatten(0, (H // 2, 2)).permute(0, 2, 1, 3).flatten(2)  # [pairs, F, 2D]
    q = st["q"][b, :n].float().view(n, heads, 2, D)
    hidden = torch.arange(F, device=DEV)[None] > first + torch.arange(n, device=DEV)[:, None]
    out = torch.empty((n, heads, 2 * D), device=DEV)
    lse = torch.empty((n, heads, 2), device=DEV)
    for pair in range(H // 2):
        hs = slice(pair * per, (pair + 1) * per)
        o = None
        for m in (0, 1):
            z = torch.matmul(q[:, hs, m].transpose(0, 1).reshape(-1, D) * st["scale"], k[2 * pair + m].T)
            z = z.view(per, n, F).masked_fill_(hidden, -math.inf)
            top = z.amax(-1, keepdim=True)
            z = (z - top).exp_()
            total = z.sum(-1, keepdim=True)
            x = torch.matmul(z.view(-1, F), v[pair]).view(per, n, 2 * D) / total
            lse[:, hs, m] = (top + total.log()).squeeze(-1).T
            o = x if m == 0 else o - st["lam"][hs, None, None] * x
        o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS)
        out[:, hs] = (o * st["weight"].float() * st["out_scale"]).transpose(0, 1)
    return out.to(torch.bfloat16), lse.flatten(1)


def _norm_plain(st):
    c = st["c"]
    y = st["y"].float()
    if st["post"] is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * st["post"].float()
    if st["gate"] is not None:
        g = st["gate"].float()
        y = y * (1 / (1 + (-g).exp()) if c["act"] else g)
    h = st["res"].float() * st["scales"][1] + y * st["scales"][0]
    x = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * st["w"].float()
    return [x.to(torch.bfloat16), h.to(st["res"].dtype)]


# ------------------------------------------------------------------ definitions

def exact(c, seed):
    if c["op"] == "grow":
        return None  # whole numbers: the plain form's are the definition's
    st = prepare(c, seed)
    if c["op"] == "norm":
        scale, residual_scale = st["scales"]
        xs, hs = [], []
        for lo in range(0, c["N"], 4096):
            part = slice(lo, lo + 4096)
            u = st["y"][part].double()
            if c["post"]:
                u = u / (torch.linalg.vector_norm(u, dim=-1, keepdim=True) ** 2 / c["dim"] + EPS).sqrt() * st["post"].double()
            if c["gate"] != "none":
                gate = st["gate"][part].double() if c["gate"] == "token" else st["gate"].double()
                u = u * (torch.sigmoid(gate) if c["act"] else gate)
            h = torch.add(u * scale, st["res"][part].double(), alpha=residual_scale)
            hs.append(h)
            xs.append(h / (torch.linalg.vector_norm(h, dim=-1, keepdim=True) ** 2 / c["dim"] + EPS).sqrt() * st["w"].double())
        return [torch.cat(xs), torch.cat(hs)]
    B, T, Hq, H, D = c["B"], c["T"], c["Hq"], c["H"], c["D"]
    out = torch.zeros((B, T, Hq // 2, 2 * D), dtype=torch.float64, device=DEV)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    spans = [(f - T, T) for f in _contexts(c)] if c["op"] == "decode" else _chunks(c)
    for b, (first, n) in enumerate(spans):
        k, v = _keys_values(st, b, first + n, torch.float64)
        for i in range(Hq // 2):  # differential head i: query heads 2i, 2i + 1 and the pair of KV heads it shares
            j = i // (Hq // H)
            wide = torch.cat((v[2 * j], v[2 * j + 1]), -1)
            for lo in range(0, n, 512):
                hi = min(n, lo + 512)
                see = torch.ones((hi - lo, first + n), dtype=torch.bool, device=DEV).tril(first + lo)
                o = 0
                for m, sign in ((0, 1.0), (1, -float(st["lam"][i]))):
                    z = (st["q"][b, lo:hi, 2 * i + m].double() @ k[2 * j + m].T * st["scale"]).masked_fill(~see, -math.inf)
                    lse[b, lo:hi, 2 * i + m] = z.logsumexp(-1)
                    o = o + sign * (z.softmax(-1) @ wide)
                rms = (torch.linalg.vector_norm(o, dim=-1, keepdim=True) ** 2 / (2 * D) + EPS).sqrt()
                out[b, lo:hi, i] = o / rms * st["weight"].double() * st["out_scale"]
    return [out, lse]
