"""GPU checks of the eviction by attention mass: every result is exact."""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_kv_attention_12_gb300 import _build, binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    binding.lib()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def bits(t):
    return t.cpu().view(torch.int16).numpy()


def make(lens, *, layers=1, hkv=2, D=128, seed=0, mass="ties", evicted=(), width=None, spare=2):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    B = len(lens)
    nbs = [-(-x // 16) for x in lens]
    width = width or max(nbs + [1])
    blocks = sum(nbs) + spare
    perm = rng.permutation(blocks)
    table, at = np.full((B, width), -1), 0
    for b, nb in enumerate(nbs):
        table[b, :nb] = perm[at:at + nb]
        at += nb
    shape = (layers, B, hkv, 16 * width)
    m = rng.exponential(1.0, shape).astype(np.float32)
    if mass == "ties":
        m = np.round(m * 4) / 4
    elif mass == "same":
        m[:] = 2.5
    elif mass == "wild":
        for value in (math.nan, math.inf, -math.inf, -1.0, -0.0, 0.0, 1e-42, 3e38):
            m[rng.random(shape) < 0.1] = value
    m = m.astype(np.float32)
    pos = np.full(shape, -1)
    total = list(lens)
    for b in evicted:
        total[b] = lens[b] + int(rng.integers(1, 500))
        old = int(rng.integers(0, lens[b] + 1))
        for layer in range(layers):
            for h in range(hkv):
                pos[layer, b, h, :old] = rng.permutation(total[b] - lens[b] + old)[:old]
    pools = [torch.randn((blocks, hkv, 16, D), generator=g, device=DEV).to(torch.bfloat16)
             for _ in range(2 * layers)]
    return dict(pools=pools, mass=m, pos=pos, table=table, lens=list(lens), total=total)


def run(c, budget, sinks, recent, *, in_place=False, total=True, refcounts=None, err=None):
    mass, pos, lens = torch.tensor(c["mass"], device=DEV), i32(c["pos"]), i32(c["lens"])
    outs = (mass, pos, lens) if in_place else \
        (torch.full_like(mass, 3.0), torch.full_like(pos, 3), torch.full_like(lens, 3))
    layers, B, hkv, keys = c["mass"].shape
    n = binding.paged_kv_evict_ws_bytes(layers, B, hkv, keys // 16, budget)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device=DEV)
    pools = [p.clone() for p in c["pools"]]
    binding.paged_kv_evict(pools, mass, pos, i32(c["table"]), lens,
                           i32(c["total"]) if total else None, budget, sinks, recent, *outs, ws,
                           refcounts=refcounts, err=err)
    torch.cuda.synchronize()
    return pools, outs


def check(c, budget, sinks, recent, *, in_place=False, total=True, whole=(), refcounts=None):
    err = i32([0])
    pools, (mass, pos, lens) = run(c, budget, sinks, recent, in_place=in_place, total=total,
                                   refcounts=refcounts, err=err)
    assert err.item() == 0
    held = (c["mass"], c["pos"]) if in_place else (np.full_like(c["mass"], 3), np.full_like(c["pos"], 3))
    want = oracle.evict([bits(p) for p in c["pools"]], c["mass"], c["pos"], c["table"], c["lens"],
                        c["total"] if total else None, budget, sinks, recent, *held, whole=whole)
    assert lens.tolist() == want[3]
    assert np.array_equal(pos.cpu().numpy(), want[2])
    assert np.array_equal(mass.cpu().numpy(), want[1].astype(np.float32), equal_nan=True)
    for p, w in zip(pools, want[0]):
        assert np.array_equal(bits(p), w)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("mass", ["ties", "same", "wild", "random"])
@pytest.mark.parametrize("lens,budget,sinks,recent", [
    ([1], 1, 0, 0), ([2, 1, 0], 1, 0, 1), ([33, 100, 16], 16, 4, 4), ([400, 17, 255], 31, 0, 31),
    ([700, 650], 600, 600, 0), ([700, 650], 600, 4, 100), ([1000, 31, 32, 33], 32, 1, 0)])
def test_evict(lens, budget, sinks, recent, mass, in_place):
    c = make(lens, mass=mass, seed=budget, evicted=range(0, len(lens), 2))
    check(c, budget, sinks, recent, in_place=in_place)


@pytest.mark.parametrize("layers,hkv,D", [(1, 1, 256), (3, 2, 128), (2, 4, 256), (130, 1, 128)])
def test_layers_heads_and_head_dims(layers, hkv, D):
    c = make([120, 75, 300], layers=layers, hkv=hkv, D=D, seed=layers, evicted=[1])
    check(c, 70, 2, 20)
    check(c, 70, 2, 20, in_place=True)


@pytest.mark.parametrize("L,width", [
    (16384, 1024), (16385, 1025), (40000, 2500), (40000, 5000), (65536, 4096), (65537, 4097),
    (131072, 8192), (140000, 8750), (5000, 9000), (300, 9000)])
@pytest.mark.parametrize("mass", ["ties", "random", "same"])
def test_long_rows(L, width, mass):
    """One to eight CTAs a segment, keys past those that stay in registers."""
    c = make([L], hkv=1, width=width, seed=L, mass=mass, evicted=[0])
    for budget in (1, 257, L // 2 + 3, L - 1):
        check(c, budget, min(4, budget - 1), (budget - 1) // 3, in_place=budget == 257)


@pytest.mark.parametrize("D,budget", [(128, 255), (128, 256), (128, 257), (256, 127), (256, 128),
                                      (256, 129)])
@pytest.mark.parametrize("heaviest", ["first", "last"])
def test_moves_with_the_selection_and_behind_it(D, budget, heaviest):
    """On both sides of the bytes that a selection moves itself: as many moves as there
    can be, and none; lengths in place and beside, masses in place and lengths not."""
    c = make([600, 300, 40, 0, 600], hkv=3, layers=2, D=D, seed=budget, mass="random")
    order = np.arange(c["mass"].shape[-1], dtype=np.float32)
    c["mass"][:] = order if heaviest == "last" else -order
    for in_place in (False, True):
        check(c, budget, 0, 0, in_place=in_place)
    mass, pos, lens = torch.tensor(c["mass"], device=DEV), i32(c["pos"]), i32(c["lens"])
    new_lens, ws = i32([7] * 5), torch.full((binding.paged_kv_evict_ws_bytes(
        2, 5, 3, c["mass"].shape[-1] // 16, budget),), 0xff, dtype=torch.uint8, device=DEV)
    pools = [p.clone() for p in c["pools"]]
    binding.paged_kv_evict(pools, mass, pos, i32(c["table"]), lens, None, budget, 0, 0, mass, pos,
                           new_lens, ws)
    torch.cuda.synchronize()
    want, outs = run(c, budget, 0, 0, in_place=True, total=False)
    assert all(torch.equal(x, y) for x, y in zip((*pools, mass, pos, new_lens), (*want, *outs)))
    assert lens.tolist() == c["lens"]


def test_without_total_lengths():
    check(make([100, 300], seed=3), 64, 4, 16, total=False)


def test_more_held_keys_than_the_budget():
    """Positions that occur twice hold more keys than sinks and recent say."""
    c = make([200], seed=6)
    c["pos"][..., :120] = 190
    check(c, 50, 4, 30)


def test_shared_blocks_leave_a_request_whole():
    c = make([200, 200, 90], seed=8)
    refs = np.ones(len(c["pools"][0]), dtype=np.int64)
    refs[c["table"][0][3]] = 2          # below its budget of 5 blocks
    refs[c["table"][1][5]] = 2          # past it
    check(c, 80, 4, 16, whole=[0], refcounts=i32(refs))
    check(c, 80, 4, 16, whole=[0], refcounts=i32(refs), in_place=True)


def test_bad_data_is_reported():
    c = make([200, 100], seed=9)
    for key, value in (("lens", [-3, 100]), ("lens", [10 ** 6, 100]), ("total", [100, 100])):
        err = i32([0])
        run(dict(c, **{key: value}), 64, 4, 16, err=err)
        assert err.item() & binding.DEVERR_SEQ_LEN
    d = dict(c, table=c["table"].copy())
    d["table"][0, :] = [10 ** 9, -7] * 6 + [500]
    err = i32([0])
    pools, (mass, pos, lens) = run(d, 64, 4, 16, err=err)
    assert err.item() == binding.DEVERR_BAD_TABLE and lens.tolist() == [64, 64]
    good, _ = run(c, 64, 4, 16)
    mine = c["table"][1][:7]
    for p, q, was in zip(pools, good, c["pools"]):
        assert torch.equal(p[mine], q[mine])
        assert torch.equal(p[c["table"][0][:13]], was[c["table"][0][:13]])


def test_a_graph_evicts_again_and_again():
    c = make([500, 300], seed=10)
    mass, pos, lens, total = torch.tensor(c["mass"], device=DEV), i32(c["pos"]), i32(c["lens"]), \
        i32(c["total"])
    table = i32(c["table"])
    n = binding.paged_kv_evict_ws_bytes(1, 2, 2, mass.shape[3] // 16, 200)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    pools = [p.clone() for p in c["pools"]]
    args = (pools, mass, pos, table, lens, total, 200, 4, 50, mass, pos, lens, ws)
    snap = [x.clone() for x in (*pools, mass, pos, lens)]
    binding.paged_kv_evict(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.paged_kv_evict(*args)
    for x, was in zip((*pools, mass, pos, lens), snap):
        x.copy_(was)
    d = dict(c, pools=[bits(p) for p in c["pools"]])
    grown = 0
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = oracle.evict(d["pools"], d["mass"], d["pos"], c["table"], d["lens"], d["total"], 200,
                            4, 50, d["mass"], d["pos"])
        assert lens.tolist() == want[3] and np.array_equal(pos.cpu().numpy(), want[2])
        assert np.array_equal(mass.cpu().numpy(), want[1].astype(np.float32))
        for p, w in zip(pools, want[0]):
            assert np.array_equal(bits(p), w)
        # 40 new tokens each, and some mass
        grown += 40
        lens += 40
        total += 40
        mass += 0.25 * (torch.arange(mass.shape[3], device=DEV) % 7)
        torch.cuda.synchronize()
        d = dict(pools=want[0], mass=mass.cpu().numpy(), pos=pos.cpu().numpy(), lens=lens.tolist(),
                 total=total.tolist())
