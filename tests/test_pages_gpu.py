"""GPU checks of the page operations: every result is exact."""
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


@pytest.mark.parametrize("B,width,n", [(1, 1, 1), (5, 7, 40), (300, 33, 1000)])
def test_ref_blocks(B, width, n):
    rng = np.random.default_rng(B)
    tables = rng.integers(-1, n, (B, width))
    lens = rng.integers(0, 16 * width + 1, B)
    refs = rng.integers(0, 5, n) + 10000
    got, err = i32(refs), i32([0])
    for delta in (1, -1, -1, 3):
        binding.paged_kv_ref_blocks(i32(tables), i32(lens), got, delta, err)
        refs = oracle.ref_blocks(refs, tables, lens, delta)
    torch.cuda.synchronize()
    assert err.item() == 0 and np.array_equal(got.cpu().numpy(), refs)


def test_ref_blocks_reports():
    refs, err = i32([1, 0, 2]), i32([0])
    binding.paged_kv_ref_blocks(i32([[0, 1, 9]]), i32([20]), refs, -1, err)  # 9 is not used
    torch.cuda.synchronize()
    assert err.item() == binding.DEVERR_REFCOUNT and refs.tolist() == [0, -1, 2]
    err.zero_()
    binding.paged_kv_ref_blocks(i32([[0, 2, 9], [2, 2, 2]]), i32([48, -5]), refs, 1, err)
    torch.cuda.synchronize()
    assert err.item() == binding.DEVERR_BAD_TABLE | binding.DEVERR_SEQ_LEN
    assert refs.tolist() == [1, -1, 3]


@pytest.mark.parametrize("shape,dtype,pools,pairs", [
    ((9, 16), torch.uint8, 1, 1), ((40, 2, 1, 1152), torch.uint8, 3, 11),
    ((64, 2, 16, 128), torch.bfloat16, 2, 30), ((30, 1, 16, 256), torch.bfloat16, 4, 15),
    ((50, 2064), torch.uint8, 300, 20)])
def test_copy_blocks(shape, dtype, pools, pairs):
    g = torch.Generator(device=DEV).manual_seed(pairs)
    ps = [torch.randint(0, 200, shape, generator=g, device=DEV).to(dtype) for _ in range(pools)]
    rng = np.random.default_rng(pairs)
    ids = rng.permutation(shape[0])
    dst = ids[:pairs]
    src = rng.choice(ids[pairs:], pairs)               # one source may have several copies
    want = [oracle.copy_blocks(p.float().cpu().numpy(), src, dst) for p in ps]
    err = i32([0])
    binding.paged_kv_copy_blocks(ps, i32(src), i32(dst), err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for p, w in zip(ps, want):
        assert np.array_equal(p.float().cpu().numpy(), w)


def test_copy_blocks_bad_and_equal_ids():
    p = torch.arange(64, dtype=torch.uint8, device=DEV).repeat_interleave(16).view(64, 16)
    want, err = p.clone(), i32([0])
    binding.paged_kv_copy_blocks([p], i32([5, 64, -1, 3, 7]), i32([5, 1, 2, -9, 8]), err)
    want[8] = want[7]
    torch.cuda.synchronize()
    assert err.item() == binding.DEVERR_BAD_TABLE and torch.equal(p, want)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,share,B,width", [
    (1, 1.0, 1, 1), (1, 0.0, 2, 3), (2, 0.5, 1, 2), (31, 0.5, 3, 5), (32, 0.9, 3, 5),
    (33, 0.1, 2, 9), (255, 0.5, 4, 20), (257, 0.99, 4, 20), (8192, 0.6, 40, 100),
    (8191, 0.0, 3, 3), (8193, 1.0, 3, 3), (70001, 0.3, 17, 260)])
def test_compact(n, share, B, width, in_place):
    rng = np.random.default_rng(n + int(10 * share))
    refs = np.where(rng.random(n) < share, rng.integers(1, 9, n), rng.integers(-1, 1, n))
    tables = rng.integers(-1, n, (B, width))
    lens = rng.integers(0, 16 * width + 1, B)
    moves, live, remap, counts, new_tables = oracle.compact(refs, tables, lens)
    pools = [torch.randint(0, 255, (n, 48), dtype=torch.uint8, device=DEV),
             torch.randint(0, 255, (n, 48), dtype=torch.uint8, device=DEV)]
    want = [oracle.copy_blocks(p.cpu().numpy(), [m[0] for m in moves], [m[1] for m in moves])
            for p in pools]
    r, t = i32(refs), i32(tables)
    nr, nt = (r, t) if in_place else (torch.full_like(r, 9), torch.full_like(t, 9))
    rm, mv, err = torch.full_like(r, 9), torch.full((n + 2,), 9, dtype=torch.int32, device=DEV), i32([0])
    binding.paged_kv_compact(pools, r, t, i32(lens), nr, nt, rm, mv, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert np.array_equal(rm.cpu().numpy(), remap)
    assert np.array_equal(nr.cpu().numpy(), counts)
    assert np.array_equal(nt.cpu().numpy(), new_tables)
    flat = [x for m in moves for x in m]
    assert mv.tolist() == [len(moves), live] + flat + [-1] * (n - len(flat))
    for p, w in zip(pools, want):
        assert np.array_equal(p.cpu().numpy(), w)


def test_compact_reports_and_replays():
    """A table entry past the pool is reported and kept; a captured compaction
    does its work again on new counts."""
    n = 300
    pool = torch.arange(n, dtype=torch.int32, device=DEV).repeat_interleave(4).view(n, 4)
    refs = torch.zeros(n, dtype=torch.int32, device=DEV)
    t, lens = i32([[299, 300, 299]]), i32([33])
    nr, nt, rm = torch.zeros_like(refs), torch.zeros_like(t), torch.zeros_like(refs)
    mv, err = torch.zeros(n + 2, dtype=torch.int32, device=DEV), i32([0])
    args = ([pool], refs, t, lens, nr, nt, rm, mv, err)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.paged_kv_compact(*args)
    for live in ([299], [299, 3, 200], []):
        refs.zero_()
        refs[live] = 1
        err.zero_()
        pool.copy_(torch.arange(n, dtype=torch.int32, device=DEV).repeat_interleave(4).view(n, 4))
        graph.replay()
        torch.cuda.synchronize()
        moves, k, remap, counts, tables = oracle.compact(refs.tolist(), t.tolist(), [33])
        assert err.item() == binding.DEVERR_BAD_TABLE
        assert mv[:2].tolist() == [len(moves), k] and np.array_equal(rm.cpu().numpy(), remap)
        assert nt.tolist() == tables.tolist() and np.array_equal(nr.cpu().numpy(), counts)
        for s, d in moves:
            assert (pool[d] == s).all()


def test_plan_alone():
    """No pools: the plan and the tables only."""
    L = binding.lib()
    n = 100
    refs = torch.zeros(n, dtype=torch.int32, device=DEV)
    refs[40:] = 1
    out, remap = torch.zeros_like(refs), torch.zeros_like(refs)
    mv = torch.zeros(n + 2, dtype=torch.int32, device=DEV)
    s = torch.cuda.current_stream().cuda_stream
    st = L.paged_kv_compact(None, 0, n, 0, refs.data_ptr(), out.data_ptr(), None, None, 0, None, 0,
                            remap.data_ptr(), mv.data_ptr(), None, s)
    torch.cuda.synchronize()
    assert st == 0 and mv[:4].tolist() == [40, 60, 99, 0] and out.sum().item() == 60
    t, nt, lens = i32([[99, 60, 40]]), i32([[9, 9, 9]]), i32([48])
    st = L.paged_kv_compact(None, 0, n, 0, refs.data_ptr(), out.data_ptr(), t.data_ptr(),
                            nt.data_ptr(), 3, lens.data_ptr(), 1, remap.data_ptr(), mv.data_ptr(),
                            None, s)
    torch.cuda.synchronize()
    assert st == 0 and nt.tolist() == [[0, 39, 40]]


def test_no_pools_in_python():
    """The binding with an empty list: a copy does nothing, a compaction plans."""
    n = 70
    refs = torch.zeros(n, dtype=torch.int32, device=DEV)
    refs[50:] = 2
    t, lens = i32([[69, 50, -1]]), i32([20])
    nr, nt, rm = torch.zeros_like(refs), torch.zeros_like(t), torch.zeros_like(refs)
    mv = torch.zeros(n + 2, dtype=torch.int32, device=DEV)
    binding.paged_kv_copy_blocks([], i32([0]), i32([1]))
    binding.paged_kv_compact([], refs, t, lens, nr, nt, rm, mv)
    moves, k, remap, counts, tables = oracle.compact(refs.tolist(), t.tolist(), [20])
    assert mv[:2].tolist() == [len(moves), k] == [20, 20]
    assert np.array_equal(rm.cpu().numpy(), remap) and np.array_equal(nr.cpu().numpy(), counts)
    assert nt.tolist() == tables.tolist()


def test_pools_past_32_bits():
    """Blocks beyond 4 GiB of a pool are copied and moved where they are."""
    nbytes = 1 << 20
    n = 4 * 1024 + 24
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GiB of free device memory")
    pool = torch.zeros((n, nbytes), dtype=torch.uint8, device=DEV)
    pool[n - 1] = 7
    pool[3] = 5
    binding.paged_kv_copy_blocks([pool], i32([n - 1, 3]), i32([n - 9, n - 2]))
    assert (pool[n - 9] == 7).all() and (pool[n - 2] == 5).all() and not pool[n - 8:n - 2].any()
    refs = torch.zeros(n, dtype=torch.int32, device=DEV)
    refs[[n - 9, n - 2]] = 1
    nr, rm = torch.zeros_like(refs), torch.zeros_like(refs)
    mv = torch.zeros(n + 2, dtype=torch.int32, device=DEV)
    none = torch.zeros((0, 1), dtype=torch.int32, device=DEV)
    binding.paged_kv_compact([pool], refs, none, i32([]), nr, none, rm, mv)
    assert mv[:6].tolist() == [2, 2, n - 2, 0, n - 9, 1]
    assert (pool[0] == 5).all() and (pool[1] == 7).all() and not pool[2].any()


def test_captured_beside_another_stream():
    """A graph in which the operations follow events of another stream and
    kernels of other programs: every replay sees what they wrote before it."""
    n, B = 500, 3
    pool = torch.zeros((n, 64), dtype=torch.int32, device=DEV)
    base = torch.arange(n, dtype=torch.int32, device=DEV)[:, None].expand(n, 64)
    step, refs = i32([0]), torch.zeros(n, dtype=torch.int32, device=DEV)
    t, lens = i32(np.arange(B * 4).reshape(B, 4) * 40 + 20), i32([64, 0, 50])
    nr, nt, rm = torch.zeros_like(refs), torch.zeros_like(t), torch.zeros_like(refs)
    mv, err = torch.zeros(n + 2, dtype=torch.int32, device=DEV), i32([0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        step.add_(1)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.add(base, step, out=pool)
            binding.paged_kv_copy_blocks([pool], t[0, :1].contiguous(), t[1, :1].contiguous())
        refs.zero_()
        binding.paged_kv_ref_blocks(t, lens, refs, 1, err)
        main.wait_stream(side)
        binding.paged_kv_compact([pool], refs, t, lens, nr, nt, rm, mv, err)
        binding.paged_kv_ref_blocks(nt, lens, nr, -1, err)
    for k in range(1, 5):
        graph.replay()
        torch.cuda.synchronize()
        ids = t.tolist()
        live = sorted(ids[0] + ids[2])
        holes = [i for i in range(8) if i not in live]
        where = {i: i for i in live}
        where.update(zip(sorted(live)[::-1], holes))
        assert err.item() == 0 and not nr.any() and mv[:2].tolist() == [len(holes), 8]
        assert nt.tolist() == [[where[i] for i in ids[0]], ids[1], [where[i] for i in ids[2]]]
        for i in live:
            assert (pool[where[i]] == i + k).all()
        assert (pool[ids[1][0]] == ids[0][0] + k).all()
