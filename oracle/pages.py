"""Pages of a step from the requests' lengths, page by page (test infrastructure only).

A list is the stack of free pages (its end is the top).  Rows from the last to
the first return the pages behind max(need, keep), last page first; then rows
from the first to the last take what they need, or nothing where too few are
free.  Refused rows are left as they were.  Pinned by hand-worked cases and by
invariants: no page is lost or held twice; a step and its trim undo one another.
"""

from __future__ import annotations

import numpy as np

P = 64
FRONTIER, PAGE_RANGE, PAGES = 2, 1, 32


def grow(tables, table_rows, committed, mapped, free, n_free, T, M, counts=None, keep=None):
    """All arrays are copied.  Returns a dict of tables, mapped, free, n_free, frontiers, positions, slots, status."""
    tables, mapped, free = tables.copy(), mapped.copy(), free.copy()
    C, L = tables.shape
    B = len(table_rows)
    status = 0
    stack_ok = 0 <= n_free <= M
    if not stack_ok:
        status |= PAGE_RANGE
    top = n_free if stack_ok else 0
    rows = []
    for b in range(B):
        row, n = int(table_rows[b]), T if counts is None else int(counts[b])
        F = int(committed[b]) + n
        ok = (0 <= row < C and row not in [int(x) for x in table_rows[:b]] and committed[b] >= 0 and 0 <= n <= T
              and F <= 64 * L and 0 <= mapped[row] <= L)
        if not ok:
            status |= FRONTIER
        rows.append([ok, row, n, F])
    for ok, row, n, F in reversed(rows):
        if not ok:
            continue
        least = max(-(-F // P), 0 if keep is None else int(keep[row]))
        gone = int(mapped[row]) - least
        if gone > 0 and (not stack_ok or top + gone > M):
            status |= PAGE_RANGE
            continue
        while mapped[row] > least:
            mapped[row] -= 1
            free[top] = tables[row, mapped[row]]
            top += 1
    frontiers = np.zeros(B, np.int32)
    positions = np.full((B, T), -1, np.int32)
    slots = np.full((B, T), -1, np.int64)
    for b, (ok, row, n, F) in enumerate(rows):
        if not ok:
            continue
        need = -(-F // P)
        if need - mapped[row] > top:
            status |= PAGES
            continue
        while mapped[row] < need:
            top -= 1
            tables[row, mapped[row]] = free[top]
            mapped[row] += 1
        frontiers[b] = F
        for t in range(n):
            pos = F - n + t
            positions[b, t] = pos
            slots[b, t] = int(tables[row, pos // P]) * P + pos % P
    return dict(tables=tables, mapped=mapped, free=free, n_free=top if stack_ok else n_free, frontiers=frontiers,
                positions=positions, slots=slots, status=status)
