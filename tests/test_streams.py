"""Calls with ``stream=``: what they allocate belongs to that stream.

A block of torch's allocator is handed out in the order of the stream that was
current when it was allocated.  A tensor that a call allocates on one stream and
writes on another may lie over a block that queued work still uses.
"""

import contextlib

import numpy as np
import pytest
import torch

from paged_kv_cache_append_gb300 import nk


class Stream:
    device_index, cuda_stream = 0, 77


@pytest.fixture
def recorded(monkeypatch):
    """Every allocation as (current stream, what), every launch as (its stream, call); nothing runs."""
    seen, current = [], [None]

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def allocate(name):
        make = getattr(torch, name)

        def f(*a, device=None, **kw):
            seen.append((current[-1], name))
            return make(*a, **kw)
        return f

    class Args:
        def __getattr__(self, name):
            return lambda *a: seen.append((a[-1], name)) or 0

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((a[-1], name)) or 0

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for name in ("empty", "empty_like", "zeros", "zeros_like", "full"):
        monkeypatch.setattr(torch, name, allocate(name))
    monkeypatch.setattr(nk, "_pyargs", Args())
    monkeypatch.setattr(nk, "_lib", Lib())
    monkeypatch.setattr(nk, "_current_stream", lambda dev: 11)
    for f in ("nk_decode_workspace_bytes", "nk_prefill_workspace_bytes", "nk_shared_decode_workspace_bytes"):
        monkeypatch.setattr(nk, f, lambda *a: 32)
    return seen


def cpu(*shape, dtype=torch.bfloat16):
    t = torch.from_numpy(np.zeros(shape, np.float32)).to(dtype)
    return t


class OnDevice:
    """A tensor of device 0 as far as the binding looks before it hands on."""

    def __init__(self, *shape):
        self.shape, self.device, self.dtype = torch.Size(shape), "cpu", torch.float32

    def get_device(self):
        return 0


def pool():
    p = nk.Pool.__new__(nk.Pool)
    p.handle, p.H, p.D, p.C, p.L, p.device, p._ws = 0, 2, 64, 2, 4, 0, None
    p.planes = [[cpu(1)]]
    return p


def rope():
    r = nk.Rope.__new__(nk.Rope)
    r.device, r.address, r.head_dim = 0, 0, 0
    return r


Q, KV, I = cpu(2, 1, 8, 64), cpu(2, 1, 2, 64), cpu(2, dtype=torch.int32)
CALLS = {
    "norm_rope": (lambda s: nk.qk_norm_rope(Q, KV, I, rope(), stream=s), 2),
    "append_rope": (lambda s: pool().append_rope(0, I, I, I, KV, KV, rope(), q=Q, stream=s), 1),
    "shared_decode": (lambda s: pool().shared_decode(0, Q, I, I, I, I, 1.0, stream=s), 3),
    "verify": (lambda s: nk.verify_drafts(OnDevice(2, 3, 5), I, I, frontiers=I, stream=s), 3),
    "nk_paged_decode_attention": (lambda s: pool().decode(0, Q, I, I, I, 1.0, stream=s), 3),
    "nk_paged_append_decode_attention": (lambda s: pool().append_decode(0, Q, KV, KV, I, I, I, 1.0, stream=s), 3),
    "nk_paged_prefill_attention": (lambda s: pool().prefill(0, Q, I, I, I, I, 1.0, stream=s), 3),
}


@pytest.mark.parametrize("name", CALLS)
def test_allocations_are_in_the_order_of_the_calls_stream(recorded, name):
    call, made = CALLS[name]
    s = Stream()
    call(s)
    assert recorded == [(s, n) for _, n in recorded[:made]] + [(77, name)]
    recorded.clear()
    if name.startswith("nk_"):
        return
    call(None)
    assert recorded == [(None, n) for _, n in recorded[:made]] + [(11, name)]


@pytest.mark.parametrize("name", [n for n in CALLS if not n.startswith("nk_")])
def test_a_stream_of_another_device_is_refused(recorded, name):
    s = Stream()
    s.device_index = 1
    with pytest.raises(ValueError):
        CALLS[name][0](s)
    assert not recorded


# ---------------------------------------------------------------- on the GPU

def filled(profile, D, H, B, pages, own, seed):
    """A pool whose B rows share `pages` pages: (pool, tables, rows, frontiers)."""
    L = pages + -(-own // 64)
    M = pages + B * (L - pages)
    p = nk.Pool(profile, 1, H, D, 64 * L, B, M)
    t = torch.arange(M, dtype=torch.int32, device="cuda")
    tables = torch.cat([t[:pages].expand(B, pages), t[pages:].view(B, L - pages)], 1).contiguous()
    rows = torch.arange(B, dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(seed)
    kv = [torch.randn((B, 64 * L, H, D), generator=g, device="cuda").bfloat16() for _ in range(2)]
    p.append(0, tables, rows, torch.zeros_like(rows), *kv)
    return p, tables, rows, torch.full_like(rows, 64 * pages + own), g


@pytest.mark.gpu
def test_two_streams_without_workspaces():
    """Calls in turn on the current stream and on `stream=`, every tensor of the
    library's own making: the bits of calls one at a time."""
    D, H, G, B, pages = 128, 2, 8, 8, 40
    shared = torch.tensor([pages], dtype=torch.int32, device="cuda")
    batch = []
    for seed in (1, 2):
        p, t, r, F, g = filled("k8v4", D, H, B, pages, 100, seed)
        batch.append((p, t, r, F, torch.randn((B, 1, H * G, D), generator=g, device="cuda").bfloat16()))

    def call(b, s):
        p, t, r, F, q = b
        return p.shared_decode(0, q, t, r, F, shared, D ** -0.5, share_from=0, stream=s)

    refs = []
    for b in batch:
        refs.append([x.clone() for x in call(b, None)])
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    bad = 0
    for _ in range(50):
        got = [call(b, s) for b, s in zip(batch, (None, side))]
        torch.cuda.synchronize()
        bad += sum(not torch.equal(x, y) for a, c in zip(got, refs) for x, y in zip(a, c))
        del got
        for b, s in zip(batch, (None, side)):      # results dropped while their kernels run
            call(b, s)
    assert bad == 0


@pytest.mark.gpu
def test_small_calls_on_a_given_stream():
    """Norm + rotation, append, verification and the older calls with `stream=`: the results of the current stream."""
    D, H, G, B = 64, 2, 4, 4
    p, t, r, F, g = filled("bf16", D, H, B, 2, 90, 3)
    new = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    q, k, v = new(B, 1, H * G, D).bfloat16(), new(B, 1, H, D).bfloat16(), new(B, 1, H, D).bfloat16()
    table = nk.Rope(new(256, D).contiguous(), D, q_weight=new(D).bfloat16(), k_weight=new(D).bfloat16())
    prob, x = new(B, 3, 1000).softmax(-1), torch.randint(0, 1000, (B, 2), dtype=torch.int32, device="cuda")
    u, one = torch.rand((B, 3), generator=g, device="cuda"), torch.ones_like(r)
    side = torch.cuda.Stream()
    at, pos = F - 1, F[:, None].contiguous()

    def results(s):
        out = [*nk.qk_norm_rope(q, k, pos, table, stream=s)]
        out.append(p.append_rope(0, t, r, at, k, v, table, q=q, stream=s))
        out += nk.verify_drafts(prob, x, u, frontiers=F, stream=s)
        out += p.decode(0, q, t, r, F, 0.125, stream=s)
        out += p.append_decode(0, q, k, v, t, r, F, 0.125, stream=s)
        out += p.prefill(0, q, t, r, at, one, 0.125, stream=s)
        torch.cuda.synchronize()
        return out

    torch.cuda.synchronize()
    for a, b in zip(results(None), results(side)):
        assert torch.equal(a, b)
