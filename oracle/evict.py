"""Oracle of the eviction by attention mass (TEST INFRASTRUCTURE; see the
package doc): one (request, KV head) at a time, keys as Python tuples."""
from __future__ import annotations

import math

import numpy as np


def evict_plan(mass, pos, L: int, T: int, budget: int, sinks: int, recent: int):
    """(keys that stay, moves [(from, to)], positions of the L keys)."""
    where = [int(pos[t]) if pos[t] >= 0 else T - L + t for t in range(L)]
    n = min(L, budget)

    def order(t):
        if where[t] < sinks or where[t] >= T - recent:
            return (0, 0.0, t)
        m = float(mass[t])
        return (2, 0.0, t) if math.isnan(m) else (1, -m, t)

    stay = set(sorted(range(L), key=order)[:n])
    holes = [t for t in range(n) if t not in stay]
    movers = sorted((t for t in stay if t >= n), reverse=True)
    return stay, list(zip(movers, holes)), where


def evict(pools, mass, pos, tables, seq_lens, total_lens, budget, sinks, recent, new_mass, new_pos,
          whole=()):
    """The pools (K and V of each layer), masses, positions and lengths after an
    eviction; new_mass and new_pos: what the outputs held before.  ``whole``:
    requests that are left as they are."""
    pools = [p.copy() for p in pools]
    was = [p.copy() for p in pools]
    new_mass, new_pos = np.array(new_mass, copy=True), np.array(new_pos, copy=True)
    layers, B, Hkv, _ = mass.shape
    new_lens = []
    for b in range(B):
        L = int(seq_lens[b])
        T = L if total_lens is None else int(total_lens[b])
        n = L if b in whole else min(L, budget)
        new_lens.append(n)
        for layer in range(layers):
            for h in range(Hkv):
                m, p = mass[layer, b, h], pos[layer, b, h]
                _, moves, where = evict_plan(m, p, L, T, n, sinks, recent)
                nm, np_ = new_mass[layer, b, h], new_pos[layer, b, h]
                nm[:L], np_[:L] = 0.0, -1
                nm[:n] = m[:n]
                np_[:n] = where[:n]
                for src, dst in moves:
                    nm[dst], np_[dst] = m[src], where[src]
                    sb, db = tables[b][src // 16], tables[b][dst // 16]
                    for i in (2 * layer, 2 * layer + 1):
                        pools[i][db, h, dst % 16] = was[i][sb, h, src % 16]
    return pools, new_mass, new_pos, new_lens
