"""Pins of the oracles of the draft trees and of the eviction (CPU)."""
import numpy as np
import pytest

import oracle


def problem(lens, ns, *, hq=4, hkv=2, D=8, seed=0):
    rng = np.random.default_rng(seed)
    nbs = [-(-x // 16) for x in lens]
    blocks = sum(nbs) + 2
    perm = rng.permutation(blocks)
    table, at = np.full((len(lens), max(nbs)), -1), 0
    for b, nb in enumerate(nbs):
        table[b, :nb] = perm[at:at + nb]
        at += nb
    first = np.concatenate([[0], np.cumsum(ns)])
    k, v = rng.standard_normal((2, blocks, hkv, 16, D))
    return rng.standard_normal((first[-1], hq, D)), k, v, table, first


@pytest.mark.parametrize("window,softcap", [(0, 0.0), (5, 0.0), (0, 3.0), (20, 3.0)])
def test_a_chain_is_causal_prefill(window, softcap):
    lens, ns = [40, 17, 9], [12, 1, 9]
    q, k, v, table, first = problem(lens, ns)
    masks = oracle.tree_plan([i - 1 for n in ns for i in range(n)], first, lens, table)[0]
    got = oracle.tree_attention(q, k, v, table, first, masks, lens, 0.3, softcap, window)
    want, _ = oracle.paged_attention(q, k, v, table, lens, first, 0.3, softcap, window)
    assert np.allclose(got, want, rtol=0, atol=1e-12)


@pytest.mark.parametrize("window", [0, 3, 30])
def test_a_branch_is_its_own_sequence(window):
    """A leaf's row equals the last row of a cache that holds only its path."""
    parents = [-1, 0, 0, 1, 2, 2, 4]
    L, n = 50, 7
    q, k, v, table, first = problem([L], [n], seed=1)
    masks, positions, slots = oracle.tree_plan(parents, first, [L], table)
    got = oracle.tree_attention(q, k, v, table, first, masks, [L], 0.3, 0.0, window)
    for leaf in (3, 5, 6):
        path = sorted(oracle.ancestors(parents)[leaf])
        short = L - n + len(path)
        assert positions[leaf] == short - 1
        k2, v2 = k.copy(), v.copy()
        for i, p in enumerate(path):
            for pool, was in ((k2, k), (v2, v)):
                pool[slots[i] // 16, :, slots[i] % 16] = was[slots[p] // 16, :, slots[p] % 16]
        want, _ = oracle.paged_attention(q[leaf:leaf + 1], k2, v2, table, [short], [0, 1], 0.3, 0.0,
                                         window)
        assert np.allclose(got[leaf], want[0], rtol=0, atol=1e-12)
        # the same move by the acceptance of that path
        targets = [0] * n
        for p, c in zip(path, path[1:]):
            targets[p] = 10 + c
        paths, count, _, lens = oracle.tree_accept(parents, [10 + i for i in range(n)], targets,
                                                   first, [L], n)
        assert paths[0][:count[0]] == path and lens == [short]
        assert np.array_equal(oracle.tree_move(k, slots, first, paths), k2)


def test_plan_by_hand():
    masks, pos, slots = oracle.tree_plan([-1, 0, 0, 1], [0, 4], [18], [[3, 5]], [100])
    assert masks == [1, 3, 5, 11] and pos == [96, 97, 97, 98]
    assert slots == [3 * 16 + 14, 3 * 16 + 15, 5 * 16, 5 * 16 + 1]


def test_accept_takes_the_first_of_twins_and_stops():
    parents, tokens = [-1, 0, 0, 2, 1], [9, 7, 7, 4, 5]
    paths, count, nxt, lens = oracle.tree_accept(parents, tokens, [7, 5, 4, 0, 6], [0, 5], [30], 5)
    assert paths == [[0, 1, 4, -1, -1]] and (count, nxt, lens) == ([3], [6], [28])
    assert oracle.tree_accept(parents, tokens, [8] * 5, [0, 5], [30], 5)[:3] == ([[0] + [-1] * 4],
                                                                              [1], [8])
    assert oracle.tree_accept([], [], [], [0, 0], [30], 2) == ([[-1, -1]], [0], [-1], [30])


def test_evict_by_hand():
    mass = [5.0, 1.0, 9.0, 9.0, 0.0, 7.0, 2.0, float("nan")]
    stay, moves, where = oracle.evict_plan(mass, [-1] * 8, 8, 8, 4, 1, 1)
    assert stay == {0, 2, 3, 7} and moves == [(7, 1)] and where == list(range(8))
    # keys of an earlier eviction bring their positions; the rest are the latest
    stay, moves, where = oracle.evict_plan(mass, [0, 40, 7, -1, -1, -1, -1, -1], 8, 50, 4, 1, 1)
    assert where == [0, 40, 7, 45, 46, 47, 48, 49] and stay == {0, 2, 3, 7}


def test_evicted_attention_is_attention_over_the_kept_keys():
    rng = np.random.default_rng(3)
    L, budget = 60, 20
    q, k, v, table, _ = problem([L], [1], seed=4)
    mass, pos = rng.random((1, 1, 2, 64)).astype(np.float32), np.full((1, 1, 2, 64), -1)
    pools, new_mass, new_pos, lens = oracle.evict([k, v], mass, pos, table, [L], None, budget, 3, 5,
                                                  mass, pos)
    assert lens == [budget]
    got, _ = oracle.paged_decode(q, *pools, table, lens, 0.3)
    for h in range(4):
        kept = new_pos[0, 0, h // 2, :budget]
        assert len(set(kept)) == budget and set(range(3)) <= set(kept) and set(range(55, 60)) <= set(kept)
        assert np.array_equal(new_mass[0, 0, h // 2, :budget], mass[0, 0, h // 2, kept])
        keys = k[table[0][kept // 16], h // 2, kept % 16]
        vals = v[table[0][kept // 16], h // 2, kept % 16]
        p = np.exp(0.3 * keys @ q[0, h])
        assert np.allclose(got[0, h], (p / p.sum()) @ vals, atol=1e-12)
    assert np.all(new_pos[..., budget:L] == -1) and np.all(new_mass[..., budget:L] == 0)


@pytest.mark.parametrize("wrong", ["sibling", "window", "twin", "order"])
def test_planted_mistakes_are_seen(wrong):
    """The properties above tell the oracle from near misses of it."""
    parents = [-1, 0, 0, 1]
    masks = oracle.tree_plan(parents, [0, 4], [20], [[0, 1]])[0]
    if wrong == "sibling":
        assert (1 << 1) & masks[2] == 0 and oracle.tree_visible(masks, 20, 0)[2, 17] == 0
    elif wrong == "window":
        seen = oracle.tree_visible(masks, 20, 4)
        # token 3 at position 18 sees keys 15 and, of the tree, 0, 1 and itself
        assert np.flatnonzero(seen[3]).tolist() == [15, 16, 17, 19]
        assert np.flatnonzero(oracle.tree_visible(masks, 20, 2)[3]).tolist() == [17, 19]
    elif wrong == "twin":
        assert oracle.tree_accept([-1, 0, 0], [0, 1, 1], [1, 2, 3], [0, 3], [9], 3)[0] == [[0, 1, -1]]
    else:
        _, moves, _ = oracle.evict_plan([0, 0, 0, 1, 2, 3], [-1] * 6, 6, 6, 3, 0, 0)
        assert moves == [(5, 0), (4, 1), (3, 2)]
