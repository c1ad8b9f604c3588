"""Pins of the 4-bit cache's and the page operations' oracles: the formats'
levels, hand-worked roundings, the unit layout, and brute-force invariants."""
import numpy as np
import pytest
import torch

import oracle
from oracle.kv4 import E2M1, E4M3, nearest


def test_level_tables():
    # e4m3's values as torch decodes them; e2m1 has one mantissa bit, bias 1
    want = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(E4M3, want) and E4M3[-1] == 448
    assert E2M1.tolist() == [m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
                             for e in range(4) for m in range(2)]


def test_nearest_ties_go_to_the_even_code():
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert nearest(E2M1, mids).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert nearest(E2M1, mids + 1e-9).tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert nearest(E2M1, mids - 1e-9).tolist() == [0, 1, 2, 3, 4, 5, 6]
    assert nearest(E2M1, np.array([6.0, 7.0, 1e30])).tolist() == [7, 7, 7]
    x = torch.linspace(0, 460, 9001)
    got = E4M3[nearest(E4M3, x.double().numpy())]
    assert np.array_equal(got, x.clamp(max=448).to(torch.float8_e4m3fn).double().numpy())


def test_hand_worked_group():
    """A group with maximum 12 and pool scale 1: e4m3(12 / 6) = 2, steps of 2."""
    x = np.zeros(128)
    x[:16] = [12, -12, 1, 0.5, -0.5, 0.51, 3, -3, 5, 7, 8.9, 9, 11, -0.1, 4, 2]
    codes, sb = oracle.kv4_quantise(x, 1.0)
    assert E4M3[sb[0]] == 2 and sb[1:].tolist() == [0] * 7
    sign = np.where(codes[:16] >= 8, -1, 1)
    held = (sign * E2M1[codes[:16] & 7] * 2).tolist()
    # 0.5 / 2 = 0.25 ties to 0; 5 / 2 = 2.5 ties to 2; 7 / 2 = 3.5 ties to 4
    assert held == [12, -12, 1, 0, 0, 1, 3, -3, 4, 8, 8, 8, 12, 0, 4, 2]
    assert codes[4] == 8 and codes[13] == 8  # zeros keep their sign


def test_non_finite_groups_and_saturation():
    x = np.ones((1, 128))
    x[0, 3], x[0, 20] = np.nan, np.inf
    x[0, 40] = 1e30                                  # past 6 * 448
    pool = oracle.kv4_append(np.zeros((1, 1, 1, 1152), np.uint8), x[:, None], [5], 1.0, False)
    row = oracle.kv4_decode(pool, 1.0, False)[0, 0, 5]
    assert np.isnan(row[:32]).all() and np.isfinite(row[32:]).all()
    assert row[40] == 6 * 448 and row[32] == 0
    # 1 / 6 lies nearest to the e4m3 value 11 / 64
    assert (row[48:] == 6 * 11 / 64).all()


@pytest.mark.parametrize("is_v", [False, True])
def test_layout_is_a_bijection(is_v):
    nibbles = {oracle.kv4_place(t, c, is_v)[:2] for t in range(16) for c in range(128)}
    assert len(nibbles) == 2048 and {b for b, _ in nibbles} == set(range(1024))
    scales = {(t, c // 16): oracle.kv4_place(t, c, is_v)[2] for t in range(16) for c in range(128)}
    assert set(scales.values()) == set(range(1024, 1152))


@pytest.mark.parametrize("is_v,D,scale", [(False, 128, 0.01), (True, 256, 0.37)])
def test_append_reads_back_within_half_a_step(is_v, D, scale):
    rng = np.random.default_rng(3)
    pool = rng.integers(0, 127, (3, 2, D // 128, 1152)).astype(np.uint8)
    rows = rng.standard_normal((4, 2, D)) * np.exp(rng.standard_normal(D))
    slots = [17, -1, 40, 48]                         # a padding token and one past the pool
    out = oracle.kv4_append(pool, rows, slots, scale, is_v)
    old, new = (oracle.kv4_decode(p, scale, is_v) for p in (pool, out))
    keep = np.ones((3, 16), bool)
    keep[1, 1] = keep[2, 8] = False
    assert np.array_equal(new.transpose(0, 2, 1, 3)[keep], old.transpose(0, 2, 1, 3)[keep])
    for t, (b, o) in ((0, (1, 1)), (2, (2, 8))):
        held, x = new[b, :, o], rows[t]
        top = np.abs(x).reshape(2, -1, 16).max(-1).repeat(16, -1)
        # the widest gap of the levels is 2 of 6, the scale is within 2^-4 of top / 6
        assert (np.abs(held - x) <= top / 6 * (1 + 2 ** -4) + 1e-12).all()


def test_compaction_by_brute_force():
    rng = np.random.default_rng(1)
    for n in (1, 2, 5, 33):
        for _ in range(20):
            refs = rng.integers(-1, 3, n)
            tables = rng.integers(-1, n, (3, 4))
            lens = rng.integers(0, 65, 3)
            moves, live, remap, counts, new = oracle.compact(refs, tables, lens)
            assert live == (refs > 0).sum() and (counts[:live] > 0).all() and (counts[live:] == 0).all()
            assert all(s >= live > d for s, d in moves)
            assert [s for s, _ in moves] == sorted((s for s, _ in moves), reverse=True)
            assert [d for _, d in moves] == sorted(d for _, d in moves)
            for i in range(n):
                assert (remap[i] == -1) == (refs[i] <= 0)
                if refs[i] > 0:
                    assert counts[remap[i]] == refs[i]
            for b in range(3):
                for j in range(4):
                    used = j < -(-int(lens[b]) // 16) and tables[b, j] >= 0
                    assert new[b, j] == (remap[tables[b, j]] if used else tables[b, j])


def test_ref_and_copy_hand_worked():
    assert oracle.ref_blocks([0, 1, 2, 0], [[1, 2, 3], [2, -1, 9]], [33, 40], 1).tolist() == \
        [0, 2, 4, 1]
    pool = np.arange(4)[:, None]
    assert oracle.copy_blocks(pool, [0, 0, 5], [2, 3, 1]).ravel().tolist() == [0, 1, 0, 0]
