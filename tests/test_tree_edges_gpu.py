"""GPU checks of the draft-tree calls at the edges of what they take."""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_attention_12_gb300 import _build, binding
from tests.test_tree_gpu import check, f64, i32, i64, make, run, workspace

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    binding.lib()


@pytest.mark.parametrize("lens,hkv", [([600] * 8, 2), ([3000, 2500, 4000], 2), ([500] * 100, 1)])
def test_first_loads_out_of_cold_memory(lens, hkv):
    """D = 256: V's first loads come behind K's first tile, whatever the caches hold.
    Pairs of CTAs, cut segments and whole ones; no wait runs out."""
    c = make(lens, [9] * len(lens), D=256, hq=4 * hkv, hkv=hkv, seed=len(lens))
    want = run(c)
    check(c, want)
    args = (c["k"], c["v"], i32(c["table"]), i32(c["first"]), i64(c["masks"]), i32(c["lens"]))
    out, ws, err = torch.full_like(want, 7.0), workspace(c), i32([0])
    cold = torch.zeros(1 << 28, dtype=torch.uint8, device=DEV)      # past the L2
    for i in range(50):
        if i % 2:
            cold.fill_(i)
        binding.paged_tree_attn_ws(c["q"], out, *args, c["most"], max(lens), ws, scale=c["scale"],
                                   err=err)
        if i % 2:
            assert torch.equal(out, want)
    torch.cuda.synchronize()
    assert err.item() == 0 and torch.equal(out, want)


def test_plan_of_sequences_shorter_than_their_trees():
    """A sequence's length below its tokens would give negative positions."""
    err, masks = i32([0]), torch.full((9,), 9, dtype=torch.int64, device=DEV)
    pos, slots = i32([9] * 9), i32([9] * 9)
    binding.paged_tree_plan(i32([-1, 0, 0] * 3), i32([0, 3, 6, 9]), i32([20, 20, 20]),
                            i32([[0, 1], [2, 3], [4, 5]]), 6, 3, masks, pos, slots,
                            total_lens=i32([2, 3, -5]), err=err)
    torch.cuda.synchronize()
    assert err.item() == binding.DEVERR_SEQ_LEN
    assert masks.tolist() == [0] * 3 + [1, 3, 5] + [0] * 3
    assert pos.tolist() == [0] * 3 + [0, 1, 1] + [0] * 3
    assert slots.tolist() == [-1] * 3 + [49, 50, 51] + [-1] * 3


def accept(first, lens, parents=(-1, 0, 1), tokens=(5, 6, 7), targets=(6, 7, 8), sizes=(0, 0, 0, 0),
           in_place=False):
    """The walk alone, through the C entry point: (status, path, accepted, next tokens, new
    lengths, error word)."""
    B, n, width = len(lens), len(parents), 3
    ins = [i32(x) for x in (parents, tokens, targets, first, lens)]
    par, tok, tar, dfirst, dlens = (x.data_ptr() for x in ins)
    outs = [i32(np.full((B, width), 9)), i32([9] * B), i32([9] * B),
            ins[4] if in_place else i32([9] * B), i32([0])]
    st = binding.lib().paged_tree_accept(None, 0, *sizes, par, tok, tar, None, dfirst, dlens, B, n,
                                         width, *(x.data_ptr() for x in outs),
                                         torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return (st, *(x.tolist() for x in outs))


@pytest.mark.parametrize("sizes", [(0, 0, 0, 0), (-1, 5000, 7, 100), (8, 1025, 16, 128),
                                   (2 ** 30, 2 ** 31 - 1, 16, 256)])
def test_the_walk_alone_looks_at_no_sizes(sizes):
    """(num_blocks, num_kv_heads, block_size, head_dim) of no pools."""
    assert accept([0, 3], [30], sizes=sizes) == (0, [[0, 1, 2]], [3], [8], [30], [0])


@pytest.mark.parametrize("in_place", [False, True])
def test_more_tokens_than_keys_accept_none(in_place):
    """A length below the tree's tokens: nothing is accepted, the length stays, and the
    error word says so; as many keys as tokens are fine."""
    got = accept([0, 3, 5, 5, 8], [3, 1, -4, 2], parents=[-1, 0, 1, -1, 0, -1, 0, 1],
                 tokens=[5, 6, 7, 0, 1, 0, 1, 2], targets=[6, 7, 8, 1, 2, 1, 2, 3], in_place=in_place)
    assert got == (0, [[0, 1, 2], [-1] * 3, [-1] * 3, [-1] * 3], [3, 0, 0, 0], [8, -1, -1, -1],
                   [3, 1, -4, 2], [binding.DEVERR_SEQ_LEN])
    assert accept([0, 3], [3], in_place=in_place)[5] == [0]


def test_a_step_of_more_tokens_than_keys_leaves_the_pools():
    """Plan and acceptance of such a request beside one that is fine."""
    pools = [torch.randn((6, 2, 16, 128), device=DEV).to(torch.bfloat16) for _ in range(2)]
    was = [p.clone() for p in pools]
    parents, first, table = i32([-1, 0, 0, -1, 0, 0]), i32([0, 3, 6]), i32([[0, 1], [2, 3]])
    lens, err = i32([2, 20]), i32([0])
    masks = torch.ones(6, dtype=torch.int64, device=DEV)
    pos, slots = i32([9] * 6), i32([9] * 6)
    binding.paged_tree_plan(parents, first, lens, table, 6, 3, masks, pos, slots, err=err)
    path, count, nxt = i32([[9] * 3] * 2), i32([9, 9]), i32([9, 9])
    binding.paged_tree_accept(pools, parents, i32([1, 2, 3] * 2), i32([3, 0, 7] * 2), slots, first, lens,
                              path, count, nxt, lens, err)
    torch.cuda.synchronize()
    assert err.item() == binding.DEVERR_SEQ_LEN and lens.tolist() == [2, 19]
    assert path.tolist() == [[-1] * 3, [0, 2, -1]] and count.tolist() == [0, 2]
    assert nxt.tolist() == [-1, 7]
    for p, w in zip(pools, was):
        w[3, :, 2] = w[3, :, 3]         # token 2 (position 19) to the place of token 1
        assert torch.equal(p, w)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window", [62, 63, 64, 65])
def test_windows_as_long_as_the_widest_mask(D, window):
    """Masks that are no tree: a row of all 64 bits is 64 deeper than one of none, and a
    window of 64 hides that key from it."""
    rng = np.random.default_rng(5)
    ns = [20, 64, 9]
    masks = [int(x) for x in rng.integers(0, 1 << 63, sum(ns))] + [1] * 3
    masks[30], masks[31], masks[40] = 0, (1 << 64) - 1, 1 << 63
    c = make([100, 64, 400], ns, D=D, masks=masks, window=window, seed=window)
    assert (oracle.tree_visible(masks[20:84], 64, window)[11, 10]) == (window > 64)
    check(c, run(c))


@pytest.mark.parametrize("B", [255, 256, 257, 512, 513])
@pytest.mark.parametrize("last", [4, 900])
def test_as_many_requests_as_threads(B, last):
    """The work is summed by 256 threads, then in rounds of them: batches around whole
    rounds, whose last request has rows, on a line of work that is cut and on one that
    is not."""
    rng = np.random.default_rng(B)
    ns = [int(x) for x in rng.choice([0, 1, 2], B)]
    ns[-1] = ns[0] = 3
    lens = [max(n, int(x)) for n, x in zip(ns, rng.integers(0, 40, B))]
    lens[-1] = last
    c = make(lens, ns, hq=4, seed=B)
    err = i32([0])
    out = run(c, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    check(c, out)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (8, 1)])
def test_promises_wider_than_the_batch(D, hq, hkv):
    """Captured steps promise the widest tree and the longest row: 64 tokens over a batch
    of a few rows, of one, and all of the table's keys."""
    for lens, ns in (([40, 7, 200], [2, 1, 3]), ([1], [1]), ([33], [1])):
        c = dict(make(lens, ns, D=D, hq=hq, hkv=hkv, pad=0, seed=D), most=64)
        keys = 16 * c["table"].shape[1]
        check(c, run(c, max_len=keys))
        binding.paged_tree_plan(i32(c["parents"]), i32(c["first"]), i32(c["lens"]), i32(c["table"]),
                                len(c["k"]), 64, i64([0] * len(c["masks"])), None, None)
    torch.cuda.synchronize()


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("lens,first", [
    ([60], 0), ([500, 500], 0),                       # whole; pairs of CTAs
    ([3000], 0), ([3000], 2048), ([9000, 4000], 0),   # cut: the first pieces, the last, many
    ([24000], 0)])
@pytest.mark.parametrize("value", [NAN, float("inf")])
def test_what_v_holds_behind_logits_of_minus_infinity(D, lens, first, value):
    """A key whose logit is -infinity has no weight, and 0 times an infinity or NaN in its
    V is NaN: also where a whole piece of the keys is such, and however keys are cut."""
    c = make(lens, [5] * len(lens), D=D, hq=4, hkv=1, seed=len(lens))
    c["q"][:] = c["q"].abs() + 0.1
    for b, L in enumerate(lens):
        for t in range(first, max(first, 3 * L // 5 if first == 0 else L - 5)):
            c["k"][c["table"][b, t // 16], 0, t % 16, 0] = -float("inf")
    clean = run(c)
    at = first + 3
    d = dict(c, v=c["v"].clone())
    d["v"][c["table"][0, at // 16], 0, at % 16, 7] = value
    rows, got = c["first"][-1], run(d)
    with np.errstate(invalid="ignore"):
        want = oracle.tree_attention(f64(d["q"]), f64(d["k"]), f64(d["v"]), d["table"], d["first"],
                                     d["masks"], d["lens"], d["scale"])
    assert np.array_equal(np.isfinite(f64(got))[:rows], np.isfinite(want)[:rows])
    keep = torch.isfinite(got.float())
    assert torch.equal(got[keep], clean[keep]) and not keep[:5, :, 7].any()
    assert torch.isfinite(clean.float()).all()


def test_pools_past_four_gib():
    """Blocks whose bytes lie past 2^32 and whose elements past 2^31: attention,
    acceptance and eviction give what they give in a small pool."""
    hkv, D, blocks, small = 8, 256, 70000, 24
    if torch.cuda.mem_get_info()[0] < 3 * blocks * hkv * 16 * D * 2:
        pytest.skip("not enough free memory")
    near = [torch.randn((small, hkv, 16, D), device=DEV).to(torch.bfloat16) for _ in range(2)]
    far = [torch.empty((blocks, hkv, 16, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    assert far[0].numel() > 1 << 31 and 2 * far[0].numel() > 1 << 32
    up = blocks - small
    for f, n in zip(far, near):
        f[up:] = n
    parents, first, lens = [-1, 0, 0, 1, 2, -1, 0, 1], i32([0, 5, 8]), [192, 97]
    table = np.arange(24).reshape(2, 12)
    tokens, targets = i32([1, 2, 3, 4, 5, 1, 2, 3]), i32([3, 0, 5, 0, 0, 2, 9, 0])
    q = torch.randn((8, 8, D), device=DEV).to(torch.bfloat16)
    results = []
    for pools, base in ((near, 0), (far, up)):
        seq, tab, err = i32(lens), i32(table + base), i32([0])
        masks, slots = torch.zeros(8, dtype=torch.int64, device=DEV), i32([0] * 8)
        binding.paged_tree_plan(i32(parents), first, seq, tab, len(pools[0]), 5, masks, None, slots,
                                err=err)
        pools[1][base + 11, 3, 15, 9] = float("inf")         # request 0's last drafted key
        out = torch.zeros_like(q)
        ws = torch.zeros(binding.paged_tree_attn_ws_bytes(8, hkv, D, 5), dtype=torch.uint8, device=DEV)
        binding.paged_tree_attn_ws(q, out, *pools, tab, first, masks, seq, 5, 192, ws, scale=0.06,
                                   err=err)
        path, few = i32(np.zeros((2, 5))), [i32([0, 0]) for _ in range(2)]
        binding.paged_tree_accept(pools, i32(parents), tokens, targets, slots, first, seq, path, *few, seq,
                                  err)
        mass = torch.arange(2 * hkv * 192, device=DEV).float().view(1, 2, hkv, 192) % 37
        kpos = torch.full(mass.shape, -1, dtype=torch.int32, device=DEV)
        n = binding.paged_kv_evict_ws_bytes(1, 2, hkv, 12, 60)
        binding.paged_kv_evict(pools, mass, kpos, tab, seq, None, 60, 4, 16, mass, kpos, seq,
                               torch.zeros(n, dtype=torch.uint8, device=DEV), err=err)
        torch.cuda.synchronize()
        assert err.item() == 0
        results.append([out, slots - 16 * base, path, *few, seq, mass, kpos, *(p[base:base + small] for p in pools)])
    for x, y in zip(*results):
        assert torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x,
                           y.view(torch.int16) if y.dtype == torch.bfloat16 else y)


def test_two_streams_at_once():
    """Steps on two streams, each with workspaces of its own, give what they give alone:
    shared and cut segments, acceptance and eviction beside one another."""
    cases = [make([600] * 6, [9] * 6, D=256, seed=1), make([5000, 300, 2200], [16, 3, 16], D=128, seed=2)]
    jobs = []
    for c in cases:
        B, keys = len(c["lens"]), 16 * c["table"].shape[1]
        rows = len(c["masks"])
        args = dict(c=c, B=B, keys=keys, tab=i32(c["table"]), first=i32(c["first"]), lens=i32(c["lens"]),
                    masks=i64(c["masks"]), parents=i32(c["parents"]), ws=workspace(c),
                    tokens=i32([1] * rows), slots=i32([0] * rows),
                    mass=torch.rand((1, B, 2, keys), device=DEV),
                    kpos=torch.full((1, B, 2, keys), -1, dtype=torch.int32, device=DEV),
                    ews=torch.zeros(binding.paged_kv_evict_ws_bytes(1, B, 2, keys // 16, 256),
                                    dtype=torch.uint8, device=DEV))
        jobs.append(args)

    def step(j):
        c, B = j["c"], j["B"]
        pools = [c["k"].clone(), c["v"].clone()]
        out, lens = torch.zeros_like(c["q"]), j["lens"].clone()
        mass, kpos = j["mass"].clone(), j["kpos"].clone()
        path, few = torch.zeros((B, c["most"]), dtype=torch.int32, device=DEV), \
            [torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(2)]
        for _ in range(3):
            binding.paged_tree_attn_ws(c["q"], out, *pools, j["tab"], j["first"], j["masks"], lens,
                                       c["most"], max(c["lens"]), j["ws"], scale=c["scale"])
        binding.paged_tree_plan(j["parents"], j["first"], lens, j["tab"], len(pools[0]), c["most"], None,
                                None, j["slots"])
        binding.paged_tree_accept(pools, j["parents"], j["tokens"], j["tokens"], j["slots"], j["first"],
                                  lens, path, *few, lens)
        binding.paged_kv_evict(pools, mass, kpos, j["tab"], lens, None, 256, 4, 16, mass, kpos, lens,
                               j["ews"])
        return [out, path, *few, lens, mass, kpos, *pools]

    alone = [step(j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for i, (j, s) in enumerate(zip(jobs, streams)):
            with torch.cuda.stream(s):
                got[i].append(step(j))
    torch.cuda.synchronize()
    for want, runs in zip(alone, got):
        for r in runs:
            for x, y in zip(r, want):
                assert torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x,
                                   y.view(torch.int16) if y.dtype == torch.bfloat16 else y)
