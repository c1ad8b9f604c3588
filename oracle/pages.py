"""Oracle of the page operations (TEST INFRASTRUCTURE; see the package doc):
reference counts from tables, block copies and compaction, one block at a time."""
from __future__ import annotations

import numpy as np


def used_entries(table_row, seq_len: int, block_size: int = 16):
    """A row's used part: its first ceil(seq_len / block_size) entries."""
    n = -(-max(0, int(seq_len)) // block_size)
    return list(map(int, table_row[:min(n, len(table_row))]))


def ref_blocks(refcounts, tables, seq_lens, delta: int):
    out = np.array(refcounts, dtype=np.int64)
    for row, n in zip(tables, seq_lens):
        for i in used_entries(row, n):
            if 0 <= i < len(out):
                out[i] += delta
    return out


def copy_blocks(pool: np.ndarray, src, dst):
    """All sources are read before any destination is written."""
    out = pool.copy()
    for s, d in zip(src, dst):
        if 0 <= s < len(pool) and 0 <= d < len(pool):
            out[d] = pool[s]
    return out


def compact(refcounts, tables, seq_lens):
    """(moves [(old, new)], live, remap, new counts, new tables): the highest
    live block goes to the lowest hole until no live block is above a hole."""
    refs = [max(0, int(r)) for r in refcounts]
    n = len(refs)
    live = sum(r > 0 for r in refs)
    remap = [i if refs[i] > 0 else -1 for i in range(n)]
    moves = []
    lo, hi = 0, n - 1
    counts = list(refs)
    while True:
        while lo < n and counts[lo] > 0:
            lo += 1
        while hi >= 0 and counts[hi] <= 0:
            hi -= 1
        if lo >= hi:
            break
        moves.append((hi, lo))
        counts[lo], counts[hi] = counts[hi], 0
        remap[hi] = lo
    new_tables = np.array(tables, copy=True)
    for b, (row, ln) in enumerate(zip(tables, seq_lens)):
        for j, i in enumerate(used_entries(row, ln)):
            if 0 <= i < n:
                new_tables[b][j] = remap[i]
    return moves, live, np.array(remap), np.array(counts), new_tables
