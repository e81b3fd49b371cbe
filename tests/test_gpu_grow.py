"""GPU parity of the page growth against the oracle, entry by entry (whole numbers)."""

import numpy as np
import pytest
import torch

from oracle import pages as OP
from paged_kv_cache_append_gb300 import nk
from tests.test_oracle_diff import state

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


class Case:
    def __init__(self, C, L, M, used, rows, committed, T, counts=None, keep=None, n_free=None, seed=0):
        self.tables, self.mapped, self.free, self.n = state(C, L, M, used, seed)
        self.n = self.n if n_free is None else n_free
        self.rows, self.committed, self.T, self.M = rows, np.asarray(committed), T, M
        self.counts, self.keep = counts, keep
        self.pool = nk.Pool("nvfp4_g16", 1, 1, 64, 64 * L, C, M)
        self.d = dict(tables=dev(self.tables), mapped=dev(self.mapped), free=dev(self.free), n=dev([self.n]))

    def oracle(self):
        return OP.grow(self.tables, self.rows, self.committed, self.mapped, self.free, self.n, self.T, self.M,
                       self.counts, self.keep)

    def gpu(self, **kw):
        d, opt = self.d, lambda x: None if x is None else dev(x)  # noqa: E731
        return self.pool.grow(d["tables"], dev(self.rows), dev(self.committed), d["mapped"], d["free"], d["n"], self.T,
                              counts=opt(self.counts), keep=opt(self.keep), **kw)

    def check(self):
        want = self.oracle()
        nk.nk_status_read(True)
        f, p, s = self.gpu()
        torch.cuda.synchronize()
        assert nk.nk_status_read(True) == want["status"]
        for name, got in (("tables", self.d["tables"]), ("mapped", self.d["mapped"]), ("free", self.d["free"]),
                          ("n_free", self.d["n"]), ("frontiers", f), ("positions", p), ("slots", s)):
            assert np.array_equal(got.cpu().numpy().reshape(-1), np.asarray(want[name]).reshape(-1)), name


def test_one_row_one_page():
    Case(1, 1, 1, [0], [0], [0], 1).check()
    Case(1, 1, 1, [1], [0], [63], 1).check()
    Case(1, 1, 1, [1], [0], [0], 0).check()


@pytest.mark.parametrize("T", [0, 1, 4, 63, 64, 65, 513, 1300])
def test_lengths_at_page_edges(T):
    """Rows that stay on their page, cross into the next, fill it exactly, return pages, in an odd order; 513 tokens
    are the first whose slots a second kernel writes at 8 rows."""
    used = [1, 2, 3, 4, 9, 0, 7, 30]
    committed = [0, 1, 63, 64, 65, 127, 128, 400]
    Case(8, 64, 8 * 64, used, [3, 1, 7, 0, 2, 6, 5, 4], committed, T).check()
    Case(8, 64, 8 * 64, used, [3, 1, 7, 0, 2, 6, 5, 4], committed, T, counts=[T, 0, T // 2, T, min(T, 1), 0, T, T]).check()


def test_pages_returned_in_a_call_are_taken_in_it():
    """An empty stack: every page that a row takes is one that another returned."""
    Case(4, 8, 16, [8, 0, 8, 0], [0, 1, 2, 3], [10, 0, 70, 0], 300, counts=[0, 300, 0, 200]).check()


def test_too_few_pages():
    """A row takes all or nothing, and the next one is tried."""
    c = Case(3, 8, 8, [2, 0, 0], [1, 0, 2], [0, 100, 0], 450, counts=[450, 28, 60])
    assert c.oracle()["status"] == OP.PAGES and list(c.oracle()["frontiers"]) == [0, 128, 60]
    c.check()


def test_keep_protects_leading_pages():
    Case(2, 8, 12, [6, 6], [0, 1], [10, 200], 5, keep=[4, 0]).check()
    Case(2, 8, 12, [6, 6], [0, 1], [10, 200], 5, keep=[9, -3]).check()


@pytest.mark.parametrize("bad", [
    dict(rows=[0, 9, 2]), dict(rows=[0, -1, 2]), dict(rows=[0, 2, 2]), dict(committed=[10, -1, 20]),
    dict(counts=[1, -1, 2]), dict(counts=[1, 5, 2]), dict(committed=[10, 509, 20]), dict(committed=[10, 2 ** 31 - 1, 20]),
    dict(n_free=-1), dict(n_free=25), dict(n_free=23)])
def test_refused_on_the_device(bad):
    """A broken row is left as it was, the others get their pages; a broken stack counts as empty."""
    kw = dict(rows=[0, 1, 2], committed=[10, 30, 20], counts=[4, 4, 4])
    kw.update(bad)
    Case(3, 8, 24, [3, 2, 0], T=4, **kw).check()


def test_mapped_counts_out_of_range():
    for n in (-1, 9):
        c = Case(3, 8, 24, [1, 2, 0], [0, 1, 2], [10, 30, 20], 4)
        c.mapped[1] = n
        c.d["mapped"] = dev(c.mapped)
        c.check()


@pytest.mark.parametrize("seed", range(30))
def test_random_batches(seed):
    g = np.random.default_rng(seed)
    C, L = int(g.integers(1, 9)), int(g.integers(1, 200))
    M = int(g.integers(max(L, C), C * L + 1))
    used = np.zeros(C, int)
    for row in g.permutation(C):
        used[row] = g.integers(0, min(L, M - used.sum()) + 1)
    B = int(g.integers(1, C + 1))
    T = int(g.choice([0, 1, 3, 100, 700, 64 * L]))
    rows = g.permutation(C)[:B]
    committed = [int(g.integers(0, 64 * L + 1)) for _ in rows]
    counts = g.integers(0, T + 1, B) if g.random() < 0.7 else None
    keep = g.integers(0, L + 1, C) if g.random() < 0.3 else None
    Case(C, L, M, used, rows, committed, T, counts=counts, keep=keep, seed=seed).check()


def test_given_outputs_and_frontiers_in_place():
    c = Case(4, 16, 64, [3, 2, 0, 5], [2, 0, 3], [0, 180, 300], 70)
    want = c.oracle()
    f = dev(c.committed)
    mapped_out, n_out = dev([-5] * 4), dev([-5])
    before = {k: v.clone() for k, v in c.d.items()}
    got = c.pool.grow(c.d["tables"], dev(c.rows), f, c.d["mapped"], c.d["free"], c.d["n"], 70, frontiers=f,
                      mapped_out=mapped_out, free_count_out=n_out, positions=False)
    torch.cuda.synchronize()
    assert got[0] is f and got[1] is None and np.array_equal(f.cpu(), want["frontiers"])
    assert np.array_equal(got[2].cpu(), want["slots"]) and np.array_equal(mapped_out.cpu(), want["mapped"])
    assert int(n_out) == want["n_free"]
    assert torch.equal(c.d["mapped"], before["mapped"]) and torch.equal(c.d["n"], before["n"])


def test_captured_steps_grow_and_trim():
    """One graph: a step of 4 tokens, two of which stand, replayed over page edges; the host only reads at the end."""
    C, L, M = 4, 8, 20
    pool = nk.Pool("nvfp4_g16", 1, 1, 64, 64 * L, C, M)
    tables, mapped, free, n = pool.free_pages()
    assert int(n) == M and torch.equal(free.cpu(), torch.arange(M - 1, -1, -1, dtype=torch.int32))
    rows = dev([2, 0, 3])
    done = dev([0, 61, 120])
    out = [torch.empty(3, dtype=torch.int32, device=DEV), torch.empty((3, 4), dtype=torch.int32, device=DEV),
           torch.empty((3, 4), dtype=torch.int64, device=DEV)]
    trimmed = torch.empty(3, dtype=torch.int32, device=DEV)

    def step():
        pool.grow(tables, rows, done, mapped, free, n, 4, frontiers=out[0], positions=out[1], slots=out[2])
        done.add_(2)
        pool.grow(tables, rows, done, mapped, free, n, 0, frontiers=trimmed, positions=False, slots=False)

    ref = dict(tables=tables.cpu().numpy(), mapped=mapped.cpu().numpy(), free=free.cpu().numpy(), n_free=int(n))
    length = done.cpu().numpy().copy()

    def oracle():
        nonlocal ref, length
        a = OP.grow(ref["tables"], rows.cpu().numpy(), length, ref["mapped"], ref["free"], ref["n_free"], 4, M)
        length = length + 2
        ref = OP.grow(a["tables"], rows.cpu().numpy(), length, a["mapped"], a["free"], a["n_free"], 0, M)
        return a

    step()
    oracle()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(70):
        g.replay()
        a = oracle()
    torch.cuda.synchronize()
    assert np.array_equal(tables.cpu(), ref["tables"]) and np.array_equal(mapped.cpu(), ref["mapped"])
    assert int(n) == ref["n_free"] and np.array_equal(free.cpu(), ref["free"])
    assert np.array_equal(out[0].cpu(), a["frontiers"]) and np.array_equal(out[2].cpu(), a["slots"])
    assert np.array_equal(trimmed.cpu(), length)


@pytest.mark.parametrize("B,T", [(8, 256), (8, 257), (1, 2048), (1, 2049), (3, 682), (3, 683)])
def test_tokens_beside_the_tables_and_in_a_launch_of_their_own(B, T):
    """Up to 2048 tokens of a batch get their positions and slots from the CTA of the tables, more from a second kernel."""
    used = [1, 2, 3, 4, 9, 0, 7, 30][:B]
    committed = [0, 1, 63, 64, 65, 127, 128, 400][:B]
    Case(B, 64, B * 64, used, list(range(B))[::-1], committed, T).check()
    Case(B, 64, B * 64, used, list(range(B)), committed, T, counts=[max(0, T - 5 * i) for i in range(B)]).check()
