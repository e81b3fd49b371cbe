"""The trimmed frontiers of the draft verification, read by the very next kernel."""

import pytest
import torch

from paged_kv_cache_append_gb300 import nk
from tests.test_streams import filled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("profile,D,G,T", [("bf16", 128, 4, 1), ("k8v4", 128, 8, 4), ("fp8_row", 256, 8, 4)])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_fused_append_decode_right_behind(profile, D, G, T, in_place, graph):
    """The fused append + decode starts before the kernel ahead of it ends and
    reads its frontiers at once: they are the verification's, not those of the
    round before, in every launch of a chain.  A large vocabulary keeps the
    verification busy long after the lengths are known."""
    H, B, K, V, rounds = 2, 8, 3, 131072, 12
    pool, tables, rows, F, g = filled(profile, D, H, B, 2, 900, 5)
    new = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    q, k, v = new(B, T, H * G, D).bfloat16(), new(B, T, H, D).bfloat16(), new(B, T, H, D).bfloat16()
    p = new(B, K + 1, V).softmax(-1)
    x = torch.randint(0, V, (B, K), dtype=torch.int32, device="cuda")
    px = p[:, :K].gather(-1, x.long()[..., None])[..., 0]
    draft = torch.zeros((B, K, V), device="cuda").scatter_(2, x.long()[..., None], 2 * px[..., None])
    u = [torch.rand((B, K + 1), generator=g, device="cuda") for _ in range(rounds)]     # a draft stands iff u < 1/2
    start = F - 600
    after = [start.clone() if in_place else torch.full_like(F, 64 * (i + 1)) for i in range(rounds)]
    ints = [torch.empty((B, n), dtype=torch.int32, device="cuda") for n in (1, K + 1)]
    ws = torch.empty(nk.nk_decode_workspace_bytes(pool.handle, B, T, H * G), dtype=torch.uint8, device="cuda")
    outs = [(torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")) for _ in range(rounds)]
    at = after if in_place else [start] * rounds

    def chain(wait):
        s = torch.cuda.current_stream().cuda_stream
        for i in range(rounds):
            nk.nk_verify_drafts(p.data_ptr(), V, draft.data_ptr(), V, x.data_ptr(), None, u[i].data_ptr(),
                                at[i].data_ptr(), B, K, V, ints[0].data_ptr(), ints[1].data_ptr(), after[i].data_ptr(), s)
            if wait:
                torch.cuda.synchronize()
            pool.append_decode(0, q, k, v, tables, rows, after[i], D ** -0.5, out=outs[i][0], lse=outs[i][1],
                               workspace=ws)
        return [t.clone() for t in after] + [t.clone() for o in outs for t in o]

    planes = [t.clone() for t in pool.planes[0]]
    kept = [t.clone() for t in after]

    def again():
        for a, b in zip(pool.planes[0] + after, planes + kept):
            a.copy_(b)
        torch.cuda.synchronize()

    want = chain(True)
    assert len({tuple(t.tolist()) for t in want[:rounds]}) > 1
    if graph:
        c = torch.cuda.CUDAGraph()
        with torch.cuda.graph(c):
            got = chain(False)
        for _ in range(3):
            again()
            c.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    else:
        for _ in range(3):
            again()
            got = chain(False)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
