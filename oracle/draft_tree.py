"""Oracle of the draft trees (TEST INFRASTRUCTURE; see the package doc): a
step's masks, positions and slots, the attention of drafted tokens, and the
walk that accepts them, one token at a time."""
from __future__ import annotations

import numpy as np


def ancestors(parents):
    """For each token of a tree the set of itself and its ancestors."""
    seen = []
    for i, p in enumerate(parents):
        seen.append({i} | (seen[p] if 0 <= p < i else set()))
    return seen


def tree_plan(parents, query_start_loc, seq_lens, tables, total_lens=None, block_size: int = 16):
    """(masks as Python integers, positions, slots) of all rows; rows of no
    request get (0, 0, -1)."""
    rows = len(parents)
    masks, positions, slots = [0] * rows, [0] * rows, [-1] * rows
    totals = seq_lens if total_lens is None else total_lens
    for b, (L, T) in enumerate(zip(seq_lens, totals)):
        lo, hi = query_start_loc[b], query_start_loc[b + 1]
        n = hi - lo
        for i, up in enumerate(ancestors(parents[lo:hi])):
            t = L - n + i
            masks[lo + i] = sum(1 << j for j in up)
            positions[lo + i] = T - n + len(up) - 1
            slots[lo + i] = int(tables[b][t // block_size]) * block_size + t % block_size
    return masks, positions, slots


def tree_visible(masks, L: int, window: int):
    """[n][L]: whether drafted token i (mask an integer, bit j: token j) sees key t."""
    n = len(masks)
    masks = [m & ((1 << n) - 1) for m in masks]
    deep = [bin(m).count("1") for m in masks]
    base = L - n
    sees = np.zeros((n, L), dtype=bool)
    for i in range(n):
        p = base + max(deep[i], 1) - 1
        for t in range(base):
            sees[i, t] = window <= 0 or t > p - window
        for j in range(n):
            sees[i, base + j] = (masks[i] >> j & 1) and (window <= 0 or deep[i] - deep[j] < window)
    return sees


def tree_attention(q, k_pool, v_pool, tables, query_start_loc, masks, seq_lens, scale,
                   softcap=0.0, window=0, weight_of=None):
    """fp64 [total_q][Hq][D]: attention of drafted tokens; rows of no request are
    NaN.  ``weight_of``: a function of V applied before the sum (abs, for bounds)."""
    q = np.asarray(q, dtype=np.float64)
    rows, Hq, D = q.shape
    Hkv, bs = k_pool.shape[1], k_pool.shape[2]
    G = Hq // Hkv
    out = np.full((rows, Hq, D), np.nan)
    for b, L in enumerate(map(int, seq_lens)):
        lo, hi = int(query_start_loc[b]), int(query_start_loc[b + 1])
        if hi <= lo:
            continue
        sees = tree_visible([int(m) for m in masks[lo:hi]], L, window)
        t = np.flatnonzero(sees.any(0))
        blk = np.asarray(tables[b])[t // bs]
        K, V = k_pool[blk, :, t % bs, :], v_pool[blk, :, t % bs, :]
        if weight_of is not None:
            V = weight_of(V)
        for i in range(hi - lo):
            mine = sees[i, t]
            for h in range(Hq):
                if not mine.any():
                    out[lo + i, h] = 0.0
                    continue
                s = scale * (K[mine, h // G] @ q[lo + i, h])
                if 0 < softcap < np.inf:  # (an infinite cap is none)
                    s = softcap * np.tanh(s / softcap)
                with np.errstate(invalid="ignore"):
                    p = np.exp(s - np.max(s))
                    out[lo + i, h] = (p / p.sum()) @ V[mine, h // G]
    return out


def tree_accept(parents, tokens, targets, query_start_loc, seq_lens, width: int):
    """(paths [B][width], accepted, next tokens, new lengths)."""
    paths, counts, nexts, lens = [], [], [], []
    for b, L in enumerate(map(int, seq_lens)):
        lo, hi = query_start_loc[b], query_start_loc[b + 1]
        n, path, nxt = hi - lo, [], -1
        if n > 0:
            path = [0]
            while True:
                cur = path[-1]
                nxt = int(targets[lo + cur])
                child = [c for c in range(cur + 1, n)
                         if parents[lo + c] == cur and tokens[lo + c] == nxt]
                if not child:
                    break
                path.append(child[0])
        paths.append(path + [-1] * (width - len(path)))
        counts.append(len(path))
        nexts.append(nxt)
        lens.append(L - n + len(path))
    return paths, counts, nexts, lens


def tree_move(pool: np.ndarray, slots, query_start_loc, paths):
    """The pool after the accepted tokens' rows moved to their trees' first slots."""
    out = pool.copy()
    bs = pool.shape[2]
    for b, path in enumerate(paths):
        mine = slots[query_start_loc[b]:query_start_loc[b + 1]]
        for k, p in enumerate(x for x in path if x >= 0):
            if mine[p] >= 0 and mine[k] >= 0:
                out[mine[k] // bs, :, mine[k] % bs] = pool[mine[p] // bs, :, mine[p] % bs]
    return out
