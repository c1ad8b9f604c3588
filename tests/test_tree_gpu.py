"""GPU checks of the draft-tree operators against the fp64 oracle.

Attention is held to an elementwise bound (``bound`` below): weights and
outputs are each rounded once to bf16 (half a step is 2^-8 of the value), and
logits are sums of D products in fp32.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_kv_attention_12_gb300 import _build, binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    binding.lib()


def i32(x, dev=DEV):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def i64(masks, dev=DEV):
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64,
                        device=dev)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def tree(n, rng, reach=6):
    return [-1] + [int(max(0, i - rng.integers(1, reach + 1))) for i in range(1, n)]


def make(lens, ns, *, hq=8, hkv=2, D=128, window=0, softcap=0.0, scale=None, seed=0, pad=3,
         drop=True, masks=None, spare=3, poison=NAN):
    """A batch of trees.  What no query may read holds ``poison``: slots behind a
    sequence, blocks of no table, and (drop) blocks before every window, whose ids
    are -1."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    nbs = [-(-x // 16) for x in lens]
    blocks = sum(nbs) + spare
    k, v = (torch.full((blocks, hkv, 16, D), poison) for _ in range(2))
    perm = rng.permutation(blocks)
    table, at = np.full((len(lens), max(nbs + [1]) + 1), -1), 0
    for b, (L, n, nb) in enumerate(zip(lens, ns, nbs)):
        ids = perm[at:at + nb]
        at += nb
        first = max(0, L - n - window + 1) // 16 if window > 0 and drop else 0
        table[b, first:nb] = ids[first:]
        for p in (k, v):
            rows = torch.randn((L, hkv, D), generator=g)
            t = np.arange(16 * first, L)
            p[ids[t // 16], :, t % 16] = rows[t]
    first = np.concatenate([[0], np.cumsum(ns)]).astype(int)
    parents = sum((tree(n, rng) for n in ns), []) + [-1] * pad
    rows = len(parents)
    if masks is None:
        masks = oracle.tree_plan(parents, first, lens, table)[0]
    q = torch.randn((rows, hq, D), generator=g)
    c = dict(k=k, v=v, q=q)
    c = {name: x.to(torch.bfloat16).to(DEV) for name, x in c.items()}
    return dict(c, table=table, first=first, parents=parents, masks=masks, lens=list(lens),
                ns=list(ns), window=window, softcap=softcap, hkv=hkv,
                scale=1 / math.sqrt(D) if scale is None else scale, most=max(ns), pad=pad)


def workspace(c):
    hq, D = c["q"].shape[1:]
    n = binding.paged_tree_attn_ws_bytes(hq, c["hkv"], D, c["most"])
    return torch.full((n,), 0xff, dtype=torch.uint8, device=DEV)


def run(c, err=None, ws=None, out=None, max_len=None, stream=None):
    out = torch.full_like(c["q"], 7.0) if out is None else out
    binding.paged_tree_attn_ws(c["q"], out, c["k"], c["v"], i32(c["table"]), i32(c["first"]),
                               i64(c["masks"]), i32(c["lens"]), c["most"],
                               max(c["lens"]) if max_len is None else max_len,
                               workspace(c) if ws is None else ws, scale=c["scale"],
                               softcap=c["softcap"], window=c["window"], err=err, stream=stream)
    return out


def expected(c):
    args = (f64(c["q"]), f64(c["k"]), f64(c["v"]), c["table"], c["first"], c["masks"], c["lens"],
            c["scale"], c["softcap"], c["window"])
    return oracle.tree_attention(*args), oracle.tree_attention(*args, weight_of=np.abs)


def bound(c, ref, spread):
    """|out - ref| at most: the output's rounding, 2^-8 |ref|; the weights', 2^-8 sum
    p |v|; and what logits off by e do to the weights, 2 e sum p |v|: D products and
    sums of fp32 (2^-23 of the sum of their sizes each, truncation allowed), and a
    cap's forms, each off by less than 7e-7 of the cap and 2e-6 of the logit: the
    short series below an argument of 1/8 (17/315 y^6 of it and a few roundings), the
    long one below 1/2 (4.5e-7 / 0.46), exp2 above (7e-7 / 0.46)."""
    D = c["q"].shape[2]
    q, k = f64(c["q"]), f64(c["k"])
    size = abs(c["scale"]) * np.abs(q).sum(-1).max() * np.nanmax(np.abs(k))
    e = D * 2.0 ** -23 * size + max(0.0, min(2e-6 * size, 7e-7 * c["softcap"]))
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * e + 2.0 ** -14) * spread + 1e-30


def check(c, out):
    ref, spread = expected(c)
    got = f64(out)
    own = ~np.isnan(ref).all((1, 2))
    assert np.array_equal(own, np.arange(len(got)) < c["first"][-1])
    assert np.all(got[~own] == 7.0), "rows of no request were written"
    assert np.all(np.isfinite(got[own])), "a NaN that no query may see"
    off = np.abs(got[own] - ref[own]) / bound(c, ref[own], spread[own])
    assert off.max() <= 1.0, (off.max(), np.argwhere(off == off.max())[:3])


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (8, 1), (24, 3)])
def test_groups_and_head_dims(D, hq, hkv):
    c = make([40, 7, 200, 1], [8, 7, 5, 1], hq=hq, hkv=hkv, D=D, seed=D + hq)
    err = i32([0])
    out = run(c, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    check(c, out)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("lens,ns", [
    ([1], [1]), ([64], [64]), ([65], [64]), ([16, 17, 15], [16, 16, 15]),
    ([300, 129, 64], [64, 33, 17]), ([2000], [3]), ([5000, 30], [64, 30]),
    ([128, 127, 130, 256, 255], [1, 2, 3, 4, 5])])
def test_lengths_and_tree_sizes(D, lens, ns):
    c = make(lens, ns, D=D, seed=sum(lens))
    check(c, run(c))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window", [1, 2, 5, 16, 17, 63, 64, 100, 1000, 2 ** 31 - 1])
def test_windows(D, window):
    c = make([40, 300, 70, 513], [33, 20, 64, 1], D=D, window=window, seed=window)
    err = i32([0])
    out = run(c, err)
    torch.cuda.synchronize()
    assert err.item() == 0      # blocks before every window are not looked at
    check(c, out)


@pytest.mark.parametrize("softcap,scale", [(50.0, None), (2.0, None), (0.5, 1.0), (50.0, -0.1),
                                           (0.0, -0.1), (0.0, 0.0), (1000.0, 0.5),
                                           (1e-38, None), (1e-3, -2.0), (1e20, None), (1e37, 0.3),
                                           (3e38, None), (math.inf, -0.2), (-1.0, 0.1)])
def test_caps_and_scales(softcap, scale):
    for D in (128, 256):
        c = make([150, 90], [20, 31], D=D, softcap=softcap, scale=scale, seed=D)
        check(c, run(c))


@pytest.mark.parametrize("poison", [math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("softcap", [0.0, 50.0, 1e6])
def test_what_lies_beside_the_keys_has_no_say(softcap, poison):
    """Stale slots and rows of no token pick no form of the logits: the bits are
    those beside NaN, and a cap of 1e6 keeps its small logits."""
    for D in (128, 256):
        args = dict(D=D, hq=4, softcap=softcap, seed=3)
        c = make([150, 90, 21], [20, 9, 3], poison=poison, **args)
        d = make([150, 90, 21], [20, 9, 3], **args)
        out = run(c)
        assert torch.equal(out, run(d))
        check(d, out)


@pytest.mark.parametrize("D", [128, 256])
def test_one_row_far_out_under_a_large_cap(D):
    """A row whose logits reach the cap does not cost its neighbours their accuracy."""
    c = make([300, 40], [16, 8], D=D, softcap=1e5, scale=1.0, seed=7)
    c["q"][3] *= 4096
    ref, _ = expected(c)
    got = f64(run(c))
    rest = [r for r in range(24) if r != 3]
    calm = make([300, 40], [16, 8], D=D, softcap=1e5, scale=1.0, seed=7)
    want, spread = expected(calm)
    off = np.abs(got[rest] - want[rest]) / bound(dict(calm, softcap=0.0), want[rest], spread[rest])
    assert off.max() <= 1.0, off.max()
    assert np.all(np.isfinite(got[:24]))


@pytest.mark.parametrize("D", [128, 256])
def test_masks_that_are_no_tree(D):
    rng = np.random.default_rng(5)
    ns = [20, 64, 9, 3, 2]
    masks = [int(x) for x in rng.integers(0, 1 << 63, sum(ns))]
    masks[0] = masks[30] = 0
    masks[31] = (1 << 64) - 1
    masks[-2:] = [0, 0]                      # request 4: two keys, and nothing is seen
    masks += [1] * 3
    for window in (0, 7, 200):
        c = make([100, 64, 400, 3, 2], ns, D=D, masks=masks, window=window, seed=window)
        out = run(c)
        check(c, out)
        assert torch.all(out[sum(ns) - 2:sum(ns)] == 0)


@pytest.mark.parametrize("D,lens,ns,hkv", [
    (256, [4000, 10, 700, 3000, 1500], [64, 3, 40, 16, 1], 2),   # cut, whole and double tiles
    (128, [20000], [7], 1), (256, [9000], [64], 1), (128, [6000, 5999, 100], [64, 30, 64], 3)])
def test_cut_segments(D, lens, ns, hkv):
    """Segments over several CTAs and their merge, against the oracle and twice alike."""
    c = make(lens, ns, D=D, hq=4 * hkv, hkv=hkv, seed=len(lens))
    ws = workspace(c)
    out = run(c, ws=ws)
    check(c, out)
    for _ in range(3):
        assert torch.equal(out, run(c, ws=ws))


@pytest.mark.parametrize("B", [192, 193, 400, 1000])
def test_many_requests(B):
    """More requests than the threads that sum the work, and empty ones."""
    rng = np.random.default_rng(B)
    ns = [int(x) for x in rng.choice([0, 1, 2, 5], B)]
    ns[-1] = 3
    lens = [max(n, int(x)) for n, x in zip(ns, rng.integers(0, 60, B))]
    lens[B // 2], ns[B // 2] = 900, 5
    c = make(lens, ns, hq=4, seed=B)
    check(c, run(c))
    # one key head and short requests: segments stay whole, a CTA each
    c = make([20] * 140, [2] * 140, hq=4, hkv=1, seed=B)
    check(c, run(c))


@pytest.mark.parametrize("D,hq,hkv,most", [(128, 8, 2, 16), (256, 8, 2, 16), (128, 8, 2, 40),
                                           (256, 8, 1, 64), (128, 2, 2, 64), (256, 4, 4, 5)])
@pytest.mark.parametrize("window", [0, 200])
def test_segments_shared_by_two(D, hq, hkv, most, window):
    """Few segments of a few hundred keys: two CTAs take half of the tiles each.
    Rows of one tile (which the first takes alone), of two, odd and even numbers of
    tiles, short last ones, and none."""
    lens = [1, 64, 65, 128, 129, 200, 256, 300, 385, 511, 576, 0]
    ns = [min(L, 1 + (7 * i) % most) for i, L in enumerate(lens)]
    c = make(lens, ns, D=D, hq=hq, hkv=hkv, window=window, softcap=30.0 if hkv == 2 else 0.0,
             seed=D + most)
    out = run(c)
    check(c, out)
    assert torch.equal(run(c), out)


@pytest.mark.parametrize("D", [128, 256])
def test_halves_without_weight_and_with_infinities(D):
    """Keys whose logits are -infinity fill one half of a segment, or both, for one
    head; V's infinities and NaN lie in either half."""
    c = make([512, 512, 512, 300], [9, 9, 16, 9], D=D, seed=1)
    c["q"][:] = c["q"].abs() + 0.1
    for b, (lo, hi) in enumerate(((0, 256), (256, 512), (0, 512))):
        for t in range(lo, hi):
            c["k"][c["table"][b, t // 16], 1, t % 16, 0] = -math.inf
    n0 = 512 - 9
    for b, t, x in ((0, n0 + 3, math.inf), (1, n0 + 8, NAN), (3, 300 - 4, -math.inf)):
        c["v"][c["table"][b, t // 16], 0, t % 16, 5] = x
    rows = c["first"][-1]
    out = f64(run(c))[:rows]
    with np.errstate(invalid="ignore"):
        ref = expected(c)[0][:rows]
    args = dict(c, v=torch.where(torch.isfinite(c["v"]), c["v"], torch.zeros_like(c["v"])))
    with np.errstate(invalid="ignore"):
        fine, spread = (x[:rows] for x in expected(args))
    assert np.array_equal(np.isnan(out), np.isnan(ref))
    assert np.array_equal(np.isinf(out), np.isinf(ref))
    assert np.array_equal(np.sign(out[np.isinf(ref)]), np.sign(ref[np.isinf(ref)]))
    keep = np.isfinite(ref)
    # (the -infinities of K add nothing to the logits that have weight)
    args["k"] = torch.where(torch.isfinite(c["k"]), c["k"], torch.zeros_like(c["k"]))
    assert np.all(np.abs(out - fine)[keep] <= bound(args, fine, spread)[keep])


def test_lengths_past_the_promise():
    c = make([700, 90, 333], [6, 9, 12])
    for max_len in (0, 16, 100, 700):
        check(c, run(c, max_len=max_len))


@pytest.mark.parametrize("D", [128, 256])
def test_infinities_and_nan_reach_only_who_sees_them(D):
    # two branches under the root: {0, 1, 3} and {0, 2, 4}
    c = make([40, 500], [5, 5], D=D, seed=1)
    c["parents"][:10] = [-1, 0, 0, 1, 2] * 2
    c["masks"] = oracle.tree_plan(c["parents"], c["first"], c["lens"], c["table"])[0]
    plain = run(c)
    for pool, value in (("v", math.inf), ("v", NAN), ("k", NAN), ("k", -math.inf), ("v", -math.inf)):
        d = dict(c, k=c["k"].clone(), v=c["v"].clone())
        for b in (0, 1):
            t = c["lens"][b] - 5 + 3                       # token 3 of each tree
            d[pool][c["table"][b][t // 16], 1, t % 16, 7] = value
        out = run(d)
        torch.cuda.synchronize()
        seen = [3, 8]
        rest = [r for r in range(13) if r not in seen]
        assert torch.equal(out[rest], plain[rest])
        assert torch.equal(out[seen][:, :4], plain[seen][:, :4])    # KV head 0
        hit = out[seen][:, 4:].float()
        if pool == "v":
            assert torch.equal(hit[..., 8:], plain[seen][:, 4:, 8:].float())
            col = hit[..., 7]
            assert torch.all(torch.isnan(col)) if math.isnan(value) else torch.all(col == value)
        elif math.isnan(value):
            assert torch.all(torch.isnan(hit))
    # and in a prefix, from where a window cuts it
    c = make([600], [4], D=D, window=40, seed=2)
    c["parents"][:4] = [-1, 0, 1, 2]
    c["masks"] = oracle.tree_plan(c["parents"], c["first"], c["lens"], c["table"])[0]
    plain = run(c)
    t = 600 - 4 - 40 + 1                                    # the root's oldest key
    for value in (math.inf, NAN):
        d = dict(c, v=c["v"].clone())
        d["v"][c["table"][0][t // 16], 0, t % 16, 100] = value
        out = run(d)
        assert torch.equal(out[1:], plain[1:])
        assert not torch.isfinite(out[0, :4, 100]).any()
        out[0, :4, 100] = plain[0, :4, 100]
        assert torch.equal(out, plain)


def test_logits_that_are_all_minus_infinity():
    c = make([40, 3000], [3, 3], seed=4)
    c["q"][0] = 0
    c["q"][0, 0, 0] = math.inf
    c["q"][3, 0, 0] = math.inf
    c["k"][..., 0] = -c["k"][..., 0].abs().clamp(min=0.1)
    out = run(c)
    torch.cuda.synchronize()
    assert torch.isnan(out[[0, 3], 0].float()).all()
    assert torch.isfinite(out[[0, 3], 1:].float()).all() and torch.isfinite(out[[1, 2, 4, 5]].float()).all()


def test_bad_data_is_reported():
    c = make([40, 60, 30, 50], [5, 6, 4, 3], pad=9)
    err = i32([0])
    good = run(c, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    # a table id outside the pool reads as zeros
    d = dict(c, table=c["table"].copy())
    d["table"][1, 1] = 10 ** 9
    out = run(d, err)
    torch.cuda.synchronize()
    assert err.item() == binding.DEVERR_BAD_TABLE
    z = dict(c, k=c["k"].clone(), v=c["v"].clone())
    for p in (z["k"], z["v"]):
        p[c["table"][1, 1]] = 0
    check(z, out)
    # more tokens than keys, a length past the table, a bad span
    err.zero_()
    out = run(dict(c, lens=[40, 5, 30, 50]), err, max_len=60)
    torch.cuda.synchronize()
    assert err.item() == binding.DEVERR_SEQ_LEN
    assert torch.all(out[5:11] == 7) and torch.equal(out[:5], good[:5])
    for first, want in (([0, 5, 11, 4, 18], [2, 3]), ([0, 5, 11, 15, 99], [3]),
                        ([-1, 5, 11, 15, 18], [0]), ([0, 5, 11, 15, 22], [3])):
        err.zero_()
        out = run(dict(c, first=np.array(first)), err)
        torch.cuda.synchronize()
        assert err.item() & binding.DEVERR_QUERY_LOC
    d = dict(c, lens=[40, 60, 30, 10 ** 6])
    err.zero_()
    out = run(d, err, max_len=60)
    torch.cuda.synchronize()
    assert err.item() & binding.DEVERR_SEQ_LEN
    assert torch.equal(out[:15], good[:15])


def test_streams_graphs_and_unaligned_neighbours():
    c = make([1000, 400, 77], [12, 64, 5], D=256, seed=9)
    want = run(c)
    q, first, masks, lens, table = c["q"], i32(c["first"]), i64(c["masks"]), i32(c["lens"]), \
        i32(c["table"])
    side = torch.cuda.Stream()
    outs = [torch.zeros_like(q) for _ in range(2)]
    spaces = [workspace(c) for _ in range(2)]
    torch.cuda.synchronize()

    def call(i, stream=None):
        binding.paged_tree_attn_ws(q, outs[i], c["k"], c["v"], table, first, masks, lens, 64, 1000,
                                   spaces[i], scale=c["scale"], stream=stream)

    call(0, side)
    call(1)
    torch.cuda.synchronize()
    n = c["first"][-1]
    assert torch.equal(outs[0][:n], want[:n]) and torch.equal(outs[1][:n], want[:n])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
        call(0)
    outs[0].zero_()
    lens -= 16                      # the graph reads the lengths when it runs
    graph.replay()
    torch.cuda.synchronize()
    d = dict(c, lens=[x - 16 for x in c["lens"]])
    got = outs[0].clone()
    got[n:] = 7
    d["masks"] = c["masks"]
    ref = run(d)
    assert torch.equal(got[:n], ref[:n])


@pytest.mark.parametrize("D", [128, 256])
def test_shared_segments_in_a_graph_behind_one_another(D):
    """Launches of pairs that follow one another at once, of full and of sliding
    layers in turn, replayed with other lengths; some of a row's segments then fit one
    CTA, and one is longer than was promised."""
    c = make([520, 300, 150], [12, 9, 5], D=D, seed=3)
    table, first, masks, lens = i32(c["table"]), i32(c["first"]), i64(c["masks"]), i32(c["lens"])
    ws, outs = workspace(c), [torch.zeros_like(c["q"]) for _ in range(6)]

    def step():
        for i, o in enumerate(outs):
            binding.paged_tree_attn_ws(c["q"], o, c["k"], c["v"], table, first, masks, lens, 12, 500,
                                       ws, scale=c["scale"], window=(0, 300)[i % 2])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rows = c["first"][-1]
    for shift in (0, 100, 140):
        lens.copy_(i32([x - shift for x in c["lens"]]))
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, window in enumerate((0, 300)):
            d = dict(c, lens=[x - shift for x in c["lens"]], window=window)
            ref, spread = expected(d)
            got = f64(outs[i])
            assert np.all(np.abs(got - ref)[:rows] <= bound(d, ref, spread)[:rows])
            assert not outs[i][rows:].any()
            assert all(torch.equal(outs[j], outs[i]) for j in range(i, 6, 2))


# ----------------------------------------------------------------- the plan
@pytest.mark.parametrize("B,most", [(1, 1), (1, 64), (3, 7), (4, 33), (130, 64)])
@pytest.mark.parametrize("evicted", [False, True])
def test_plan(B, most, evicted):
    rng = np.random.default_rng(B + most)
    ns = [int(x) for x in rng.integers(0, most + 1, B)]
    ns[0] = most
    lens = [n + int(x) for n, x in zip(ns, rng.integers(0, 200, B))]
    total = [x + 1000 for x in lens] if evicted else None
    width = max(lens) // 16 + 2
    table = rng.permutation(B * width).reshape(B, width)
    first = np.concatenate([[0], np.cumsum(ns)])
    # chains, stars, forests and ordinary trees
    parents = []
    for b, n in enumerate(ns):
        kind = b % 4
        parents += [i - 1 for i in range(n)] if kind == 0 else \
            [-1 if i == 0 else 0 for i in range(n)] if kind == 1 else \
            [int(rng.integers(-1, i)) if i else -1 for i in range(n)] if kind == 2 else \
            tree(n, rng) if n else []
    rows = len(parents) + 5
    parents += [63] * 5
    err = i32([0])
    masks = torch.full((rows,), 9, dtype=torch.int64, device=DEV)
    pos, slots = i32(np.full(rows, 9)), i32(np.full(rows, 9))
    args = (i32(parents), i32(first), i32(lens), i32(table), B * width, 64)
    kw = dict(total_lens=None if total is None else i32(total), err=err)
    binding.paged_tree_plan(*args, masks, pos, slots, **kw)
    torch.cuda.synchronize()
    want = oracle.tree_plan(parents, first, lens, table, total)
    assert err.item() == 0
    assert torch.equal(masks, i64(want[0]))
    assert pos.tolist() == want[1] and slots.tolist() == want[2]
    only = i32(np.full(rows, 9))
    binding.paged_tree_plan(*args, None, None, only, **kw)
    assert torch.equal(only, slots)


def test_plan_reports():
    parents, first = i32([-1, 0, 5, -2, 0, 0, 3, 3]), i32([0, 3, 6, 8, 8])
    err = i32([0])
    masks = torch.zeros(8, dtype=torch.int64, device=DEV)
    pos, slots = i32([0] * 8), i32([7] * 8)
    table = i32([[0, 1], [2, 99], [4, 5], [-1, -1]])
    args = (parents, first, i32([20, 20, 1, 0]), table, 10, 64, masks, pos, slots)
    binding.paged_tree_plan(*args, err=err)
    torch.cuda.synchronize()
    assert err.item() == binding.DEVERR_TREE | binding.DEVERR_BAD_TABLE | binding.DEVERR_SEQ_LEN
    assert masks.tolist() == [1, 3, 4, 1, 3, 5, 0, 0]
    assert pos.tolist() == [17, 18, 17, 17, 18, 18, 0, 0]
    assert slots.tolist() == [17, 18, 19, -1, -1, -1, -1, -1]
    for first in ([0, 9, 6, 8, 8], [0, 3, 2, 8, 8], [-4, 3, 6, 8, 8]):
        err.zero_()
        binding.paged_tree_plan(args[0], i32(first), *args[2:], err=err)
        torch.cuda.synchronize()
        assert err.item() & binding.DEVERR_QUERY_LOC
    err.zero_()
    binding.paged_tree_plan(*args[:5], 2, masks, pos, slots, err=err)   # trees of 3 tokens
    torch.cuda.synchronize()
    assert err.item() & binding.DEVERR_QUERY_LOC


# ------------------------------------------------------------ the acceptance
@pytest.mark.parametrize("D,hkv,pools", [(128, 2, 2), (256, 1, 4), (128, 3, 6), (256, 2, 0),
                                         (128, 1, 260)])
@pytest.mark.parametrize("B,most", [(1, 1), (5, 9), (40, 64)])
def test_accept(D, hkv, pools, B, most):
    if pools == 260 and B == 40:
        B, most = 3, 20
    rng = np.random.default_rng(D + B)
    ns = [int(x) for x in rng.integers(0, most + 1, B)]
    ns[-1] = most
    lens = [n + int(x) for n, x in zip(ns, rng.integers(0, 40, B))]
    width = max(lens) // 16 + 1
    blocks = B * width + 2
    table = rng.permutation(blocks)[:B * width].reshape(B, width)
    first = np.concatenate([[0], np.cumsum(ns)])
    parents, tokens, targets = [], [], []
    for b, n in enumerate(ns):
        # chains are accepted far, bushy trees less far; tokens of few kinds, so
        # that siblings are alike at times
        p = [i - 1 for i in range(n)] if b % 3 == 0 else tree(n, rng) if n else []
        t = [int(x) for x in rng.integers(0, 3, n)]
        want = [int(x) for x in rng.integers(0, 3, n)]
        for i in range(1, n):
            if rng.random() < 0.7:
                want[p[i]] = t[i]
        parents, tokens, targets = parents + p, tokens + t, targets + want
    pad = [0] * 4
    parents, tokens, targets = parents + pad, tokens + pad, targets + pad
    slots = oracle.tree_plan(parents, first, lens, table)[2]
    g = torch.Generator(device=DEV).manual_seed(B)
    ps = [torch.randn((blocks, hkv, 16, D), generator=g, device=DEV).to(torch.bfloat16)
          for _ in range(pools)]
    path = i32(np.full((B, most), 5))
    count, nxt, err = i32([9] * B), i32([9] * B), i32([0])
    want = oracle.tree_accept(parents, tokens, targets, first, lens, most)
    moved = [oracle.tree_move(f64(p), slots, first, want[0]) for p in ps]
    new_lens = i32(lens)                                        # in place
    binding.paged_tree_accept(ps, i32(parents), i32(tokens), i32(targets),
                              i32(slots) if pools else None, i32(first), new_lens, path, count,
                              nxt, new_lens, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert path.tolist() == want[0] and count.tolist() == want[1]
    assert nxt.tolist() == want[2] and new_lens.tolist() == want[3]
    for p, m in zip(ps, moved):
        assert np.array_equal(f64(p), m)


def test_accept_whole_long_chain_in_one_block_order():
    """64 tokens, every second one accepted: rows overtake one another."""
    n, D = 64, 128
    parents = [-1, 0] + [i - 2 for i in range(2, n)]
    tokens, targets = list(range(n)), [i + 2 for i in range(n)]
    targets[0] = 2
    table = np.arange(5)[None]
    slots = oracle.tree_plan(parents, [0, n], [70], table)[2]
    pool = torch.randn((5, 2, 16, D), device=DEV).to(torch.bfloat16)
    want = oracle.tree_accept(parents, tokens, targets, [0, n], [70], n)
    assert want[1] == [32]
    moved = oracle.tree_move(f64(pool), slots, [0, n], want[0])
    path, count, nxt, lens = i32([[0] * n]), i32([0]), i32([0]), i32([0])
    binding.paged_tree_accept([pool], i32(parents), i32(tokens), i32(targets), i32(slots),
                              i32([0, n]), i32([70]), path, count, nxt, lens)
    torch.cuda.synchronize()
    assert path.tolist() == want[0] and lens.tolist() == want[3]
    assert np.array_equal(f64(pool), moved)


def test_accept_reports():
    pool = torch.randn((4, 1, 16, 128), device=DEV).to(torch.bfloat16)
    was = pool.clone()
    parents, tokens, targets = [-1, 0, 0, 9, -1, 0, 1], [0, 1, 2, 3, 0, 1, 2], [2, 0, 7, 0, 1, 2, 9]
    err = i32([0])
    path, count, nxt, lens = i32(np.zeros((3, 4))), i32([0] * 3), i32([0] * 3), i32([0] * 3)
    # request 0: token 2 at a slot past the pool; request 1: a bad span; request 2: a slot to skip
    slots = [0, 1, 64, 3, 16, -1, 18]
    binding.paged_tree_accept([pool], i32(parents), i32(tokens), i32(targets), i32(slots),
                              i32([0, 4, 3, 7]), i32([30, 20, 10]), path, count, nxt, lens, err)
    torch.cuda.synchronize()
    assert err.item() & binding.DEVERR_BAD_TABLE and err.item() & binding.DEVERR_QUERY_LOC
    assert err.item() & binding.DEVERR_TREE
    assert path.tolist()[:2] == [[0, 2, -1, -1], [-1] * 4]
    assert count.tolist()[:2] == [2, 0] and nxt.tolist()[:2] == [7, -1]
    assert lens.tolist()[:2] == [28, 20]
    assert torch.equal(pool, was)


def test_batches_without_rows_and_rows_without_requests():
    """A step in which no request brings a token; a batch that is all padding."""
    none, first, lens, table = i32([]), i32([0, 0, 0]), i32([20, 0]), i32([[0, 1], [-1, -1]])
    pool = [torch.randn((4, 2, 16, 128), device=DEV).to(torch.bfloat16) for _ in range(2)]
    kept = [p.clone() for p in pool]
    binding.paged_tree_plan(none, first, lens, table, 4, 8, none.long(), none, none)
    for pools, slots, width in ((pool, none, 3), ([], None, 0), (pool, none, 0)):
        path, got, err = i32(np.full((2, width), 7)), [i32([9, 9]) for _ in range(3)], i32([0])
        binding.paged_tree_accept(pools, none, none, none, slots, first, lens, path, *got, err)
        torch.cuda.synchronize()
        assert [x.tolist() for x in got] == [[0, 0], [-1, -1], [20, 0]] and err.item() == 0
        assert path.tolist() == [[-1] * width] * 2
    assert all(torch.equal(p, k) for p, k in zip(pool, kept))
    masks, pos, slots = torch.ones(5, dtype=torch.int64, device=DEV), i32([3] * 5), i32([3] * 5)
    binding.paged_tree_plan(i32([-1] * 5), i32([0]), none, none.view(0, 4), 4, 8, masks, pos, slots)
    torch.cuda.synchronize()
    assert (masks.tolist(), pos.tolist(), slots.tolist()) == ([0] * 5, [0] * 5, [-1] * 5)
