"""The differential attentions', the norms' and the pages' calls without a GPU: what they allocate belongs to the
call's stream, and their kernels are granted shared memory on every device."""

import pytest
import torch

from paged_kv_cache_append_gb300 import nk
from tests.test_streams import I, Q, Stream, cpu, pool, recorded  # noqa: F401
from tests.test_two_devices import fake, fake_path  # noqa: F401


def diff():
    d = nk.Diff.__new__(nk.Diff)
    d.device, d.address, d.heads, d.tokens, d.width = 0, 0, 4, 1, 128
    return d


def norm():
    n = nk.ResidualNorm.__new__(nk.ResidualNorm)
    n.device, n.address, n.dim = 0, 0, 64
    return n


CALLS = {
    "diff_decode": (lambda s: pool().diff_decode(0, Q, I, I, I, 1.0, diff(), stream=s), "diff", 3),
    "diff_prefill": (lambda s: pool().diff_prefill(0, Q, I, I, I, I, 1.0, diff(), stream=s), "diff", 3),
}


@pytest.mark.parametrize("name", CALLS)
def test_allocations_are_in_the_order_of_the_calls_stream(recorded, monkeypatch, name):  # noqa: F811
    for f in ("nk_diff_decode_workspace_bytes", "nk_diff_prefill_workspace_bytes"):
        monkeypatch.setattr(nk, f, lambda *a: 32)
    call, what, made = CALLS[name]
    s = Stream()
    call(s)
    assert recorded == [(s, n) for _, n in recorded[:made]] + [(77, what)]
    recorded.clear()
    call(None)
    assert recorded == [(None, n) for _, n in recorded[:made]] + [(11, what)]
    s.device_index = 1
    recorded.clear()
    with pytest.raises(ValueError):
        call(s)
    assert not recorded


@pytest.mark.parametrize("profile", list(nk.PROFILES))
@pytest.mark.parametrize("D", [64, 128])
def test_kernels_are_granted_their_shared_memory_on_every_device(fake, profile, D):  # noqa: F811
    p, ws, size = 4096, 1 << 20, 1 << 40
    d = nk.DiffDesc(p, 0, p, 1e-5, 1.0)
    for device in (0, 1, 0):
        fake.fake_reset(device)
        pool_desc = nk.make_desc(profile, 1, 2, D, 64 * 100, 8)
        n, _, _ = nk.nk_pool_plane_bytes(pool_desc, 800)
        handle = nk.nk_pool_create(pool_desc, 800, [4096] * n)
        for G, T in ((1, 1), (4, 1), (4, 2), (8, 4)):
            nk.nk_paged_diff_decode_attention(p, 2 * G, handle, 0, p, p, p, 8, T, 0.1, d, p, p, ws, size, None)
        nk.nk_paged_diff_prefill_attention(p, 8, handle, 0, p, p, p, p, 8, 200, 0.1, d, p, p, ws, size, None)
        nk.nk_pool_destroy(handle)
        assert fake.fake_launches() >= 10 and fake.fake_refused() == 0
