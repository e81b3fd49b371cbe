"""Two devices in one process, on a CUDA runtime that runs nothing (fake_cudart.c).

Kernels with more than 48 KB of shared memory have to be granted it on every
device; the grant of one device says nothing about another.
"""

import ctypes
import os
import subprocess

import pytest

from paged_kv_cache_append_gb300 import build, nk

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def fake_path(tmp_path_factory):
    """libnk's objects linked to the fake runtime (and to that one where torch has loaded the real one)."""
    at = tmp_path_factory.mktemp("fake")
    rt, so = str(at / "cudart.o"), str(at / "libnk_fake.so")
    subprocess.run(["gcc", "-O1", "-Wall", "-fPIC", "-c", os.path.join(HERE, "fake_cudart.c"), "-o", rt], check=True)
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", so, rt, *build.objects()], check=True)
    return so


@pytest.fixture
def fake(fake_path, monkeypatch):
    monkeypatch.setattr(nk, "_lib", None)
    return nk.load(fake_path)


def calls(profile, D, device):
    """Every launch of one pool's attention calls."""
    H, C = 2, 8
    desc = nk.make_desc(profile, 1, H, D, 64 * 100, C)
    n, _, _ = nk.nk_pool_plane_bytes(desc, 800)
    pool = nk.nk_pool_create(desc, 800, [4096] * n)
    p, ws, size = 4096, 1 << 20, 1 << 40
    for G, T in ((1, 1), (8, 1), (8, 2), (8, 4)):
        if G * T > 16 and D == 256 and profile in ("bf16", "int8_g64"):
            continue
        nk.nk_paged_shared_decode_attention(p, G * H, pool, 0, p, p, p, p, C, T, 0.1, p, p, 0, ws, size, None)
        nk.nk_paged_decode_attention(p, G * H, pool, 0, p, p, p, C, T, 0.1, p, p, ws, size, None)
    nk.nk_paged_prefill_attention(p, 8 * H, pool, 0, p, p, p, p, C, 200, 0.1, p, p, ws, size, None)
    nk.nk_pool_destroy(pool)


@pytest.mark.parametrize("profile", list(nk.PROFILES))
@pytest.mark.parametrize("D", [64, 128, 256])
def test_kernels_are_granted_their_shared_memory_on_every_device(fake, profile, D):
    for device in (0, 1, 0):
        fake.fake_reset(device)
        calls(profile, D, device)
        assert fake.fake_launches() > 0 and fake.fake_refused() == 0


@pytest.mark.parametrize("profile", list(nk.PROFILES))
def test_the_split_plan_is_the_devices_own(fake, profile):
    """Occupancy is asked on each device: the same workspace on two alike."""
    got = []
    for device in (0, 1):
        fake.fake_reset(device)
        desc = nk.make_desc(profile, 1, 2, 64, 6400, 8)
        n, _, _ = nk.nk_pool_plane_bytes(desc, 800)
        pool = nk.nk_pool_create(desc, 800, [4096] * n)
        got.append(nk.nk_decode_workspace_bytes(pool, 8, 1, 16))
        nk.nk_pool_destroy(pool)
    assert got[0] == got[1]
