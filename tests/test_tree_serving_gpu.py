"""The draft-tree and eviction calls in a row, as a serving loop makes them, and
beside the library's other calls on the same cache."""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_kv_attention_12_gb300 import _build, binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    binding.lib()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Model:
    """Token ids to q, k, v of ``layers`` layers: a table each; positions enter by
    the append's rotary embedding."""

    def __init__(self, layers, hq, hkv, D, vocab=50, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def table(h):
            return torch.randn((layers, vocab, h, D), generator=g, device=DEV).to(BF)
        self.q, self.k, self.v = table(hq), table(hkv), table(hkv)
        self.layers, self.hq, self.hkv, self.D = layers, hq, hkv, D


def pools_of(m, blocks, fill=0.0):
    return [torch.full((blocks, m.hkv, 16, m.D), fill, device=DEV, dtype=BF)
            for _ in range(2 * m.layers)]


def append(m, layer, pools, tokens, slots, positions):
    """q of the tokens after norms and rotation; their K and V go into the pools."""
    q = m.q[layer, tokens.long()].clone()
    binding.paged_kv_append_rope(q, m.k[layer, tokens.long()].clone(),
                                 m.v[layer, tokens.long()].clone(), pools[2 * layer],
                                 pools[2 * layer + 1], slots, positions,
                                 q_norm_weight=torch.ones(m.D, device=DEV),
                                 k_norm_weight=torch.ones(m.D, device=DEV), rope_theta=1e4)
    return q


def slots_of(table, b, t):
    return table[b][t // 16] * 16 + t % 16


@pytest.mark.parametrize("D,window", [(128, 0), (256, 40)])
def test_speculative_steps_leave_the_cache_of_plain_decoding(D, window):
    """Steps of plan, append, attention and acceptance over 3 requests: the cache
    holds, bit by bit, what appending the accepted tokens one by one gives, and
    the rows of accepted tokens agree with plain decode at their positions."""
    rng = np.random.default_rng(D)
    m = Model(2, 8, 2, D)
    B, steps, most = 3, 5, 12
    prompt = [30, 5, 77]
    truth = [rng.integers(0, 50, 300) for _ in range(B)]       # what the target would say
    width = 16
    table = rng.permutation(B * width + 5)[:B * width].reshape(B, width)
    blocks = B * width + 5
    pools = pools_of(m, blocks)
    lens = list(prompt)
    for layer in range(2):
        toks = i32(np.concatenate([truth[b][:lens[b]] for b in range(B)]))
        pos = np.concatenate([np.arange(x) for x in lens])
        slots = np.concatenate([slots_of(table, b, np.arange(lens[b])) for b in range(B)])
        append(m, layer, pools, toks, i32(slots), i32(pos))
    ws = torch.zeros(binding.paged_tree_attn_ws_bytes(8, 2, D, most), dtype=torch.uint8, device=DEV)
    dtable, scale = i32(table), 1 / math.sqrt(D)
    seq = i32(lens)
    err = i32([0])
    total_accepted = 0
    for step in range(steps):
        # trees whose tokens are right along a path of random length, else wrong
        ns = [int(x) for x in rng.integers(1, most + 1, B)]
        parents, tokens, targets = [], [], []
        for b, n in enumerate(ns):
            up = [-1] + [int(max(0, i - rng.integers(1, 4))) for i in range(1, n)]
            deep = [0] * n
            for i in range(1, n):
                deep[i] = deep[up[i]] + 1
            right = [True] + [bool(rng.random() < 0.7) for _ in range(n - 1)]
            at = [int(truth[b][lens[b] + d]) for d in deep]
            tokens += [x if ok else (x + 1) % 50 for x, ok in zip(at, right)]
            targets += [int(truth[b][lens[b] + d + 1]) for d in deep]
            parents += up
        first = np.concatenate([[0], np.cumsum(ns)])
        rows, pad = first[-1], 2
        parents, tokens, targets = (x + [0] * pad for x in (parents, tokens, targets))
        dfirst, dpar, dtok, dtar = i32(first), i32(parents), i32(tokens), i32(targets)
        seq += i32(ns)
        masks = torch.zeros(rows + pad, dtype=torch.int64, device=DEV)
        pos, slots = i32([0] * (rows + pad)), i32([0] * (rows + pad))
        binding.paged_tree_plan(dpar, dfirst, seq, dtable, blocks, most, masks, pos, slots, err=err)
        outs = []
        for layer in range(2):
            q = append(m, layer, pools, dtok, slots, pos)
            out = torch.zeros_like(q)
            binding.paged_tree_attn_ws(q, out, pools[2 * layer], pools[2 * layer + 1], dtable,
                                       dfirst, masks, seq, most, 256, ws, scale=scale,
                                       window=window, err=err)
            outs.append((q, out))
        path, count, nxt = i32(np.zeros((B, most))), i32([0] * B), i32([0] * B)
        binding.paged_tree_accept(pools, dpar, dtok, dtar, slots, dfirst, seq, path, count, nxt,
                                  seq, err)
        torch.cuda.synchronize()
        assert err.item() == 0
        paths, counts = path.tolist(), count.tolist()
        assert seq.tolist() == [x + c for x, c in zip(lens, counts)]
        for b in range(B):
            got = [tokens[first[b] + i] for i in paths[b][:counts[b]]]
            assert got == truth[b][lens[b]:lens[b] + counts[b]].tolist()
            assert nxt[b].item() == truth[b][lens[b] + counts[b]]
            total_accepted += counts[b]
        # plain decode at every accepted position, over the cache as it is now
        # (a shorter length hides what comes after)
        for b in range(B):
            for k, i in enumerate(paths[b][:counts[b]]):
                for layer, (q, out) in enumerate(outs):
                    row = first[b] + i
                    plain = torch.zeros_like(q[row:row + 1])
                    binding.paged_decode_attn(q[row:row + 1].contiguous(), plain, pools[2 * layer],
                                              pools[2 * layer + 1], dtable[b:b + 1].contiguous(),
                                              i32([lens[b] + k + 1]), 256, scale=scale,
                                              window=window)
                    # two roundings of weights and outputs each: 4 half steps of 2^-8
                    # of values up to sum p |v| (rows of v are below 5)
                    assert (out[row].float() - plain[0].float()).abs().max() <= 4 * 2.0 ** -8 * 5
        lens = [x + c for x, c in zip(lens, counts)]
    assert total_accepted > B * steps          # some drafts were taken
    again = pools_of(m, blocks)
    for layer in range(2):
        toks = i32(np.concatenate([truth[b][:lens[b]] for b in range(B)]))
        pos = np.concatenate([np.arange(x) for x in lens])
        slots = np.concatenate([slots_of(table, b, np.arange(lens[b])) for b in range(B)])
        append(m, layer, again, toks, i32(slots), i32(pos))
    for p, w in zip(pools, again):
        for b in range(B):
            t = np.arange(lens[b])
            where = i32(table[b][t // 16]).long(), slice(None), i32(t % 16).long()
            assert torch.equal(p[where], w[where])


def test_decode_with_key_mass_and_eviction_and_then_a_tree():
    """A cache held to 48 keys a head over 60 decode steps: every eviction is the
    oracle's for the masses that decode gathered, what stays are the appended rows
    of the positions it names, and trees are verified on it."""
    D, hq, hkv, B, budget = 128, 8, 2, 2, 48
    m = Model(1, hq, hkv, D, seed=3)
    rng = np.random.default_rng(1)
    width, blocks = 8, 2 * 8 + 3
    table = rng.permutation(blocks)[:B * width].reshape(B, width)
    dtable, scale = i32(table), 1 / math.sqrt(D)
    pools = pools_of(m, blocks)
    shape = (1, B, hkv, width * 16)
    mass = torch.zeros(shape, device=DEV)
    kpos = torch.full(shape, -1, dtype=torch.int32, device=DEV)
    n = binding.paged_kv_evict_ws_bytes(1, B, hkv, width, budget)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    S, C = binding.paged_decode_splitk_plan(B, hkv, width * 16)
    po = torch.zeros((B, hq, S, D), device=DEV)
    pl = torch.zeros((B, hq, S), device=DEV)
    lse, logits = torch.zeros((B, hq), device=DEV), torch.zeros((B, hq, width * 16), device=DEV)
    lens, total, err = i32([0] * B), i32([0] * B), i32([0])
    kept_rows = [{}, {}]                       # (request) position -> (K, V) rows
    evictions = 0
    for step in range(60):
        toks = i32(rng.integers(0, 50, B))
        t = lens.tolist()
        slots = i32([slots_of(table, b, t[b]) for b in range(B)])
        q = append(m, 0, pools, toks, slots, total.clone())
        for b in range(B):
            s = slots[b].item()
            kept_rows[b][total[b].item()] = tuple(p[s // 16, :, s % 16].clone() for p in pools)
        lens += 1
        total += 1
        binding.paged_decode_splitk_logits(q, po, pl, logits, *pools, dtable, lens, width * 16, S, C,
                                           scale=scale, err=err)
        out = torch.zeros_like(q)
        binding.paged_decode_splitk_combine(po, pl, out, lse)
        binding.paged_decode_key_mass(logits, lse, lens, hkv, mass[0])
        if lens[0].item() >= budget + 16 or step == 59:
            evictions += 1
            torch.cuda.synchronize()
            bits = [p.cpu().view(torch.int16).numpy() for p in pools]
            want = oracle.evict(bits, mass.cpu().numpy(), kpos.cpu().numpy(), table, lens.tolist(),
                                total.tolist(), budget, 4, 10, mass.cpu().numpy(),
                                kpos.cpu().numpy())
            binding.paged_kv_evict(pools, mass, kpos, dtable, lens, total, budget, 4, 10, mass, kpos,
                                   lens, ws, err=err)
            torch.cuda.synchronize()
            for p, w in zip(pools, want[0]):
                assert np.array_equal(p.cpu().view(torch.int16).numpy(), w)
            assert np.array_equal(mass.cpu().numpy(), want[1].astype(np.float32))
            assert np.array_equal(kpos.cpu().numpy(), want[2]) and lens.tolist() == want[3]
    assert evictions >= 1 and err.item() == 0
    # every kept key is the row that was appended at the position it names
    for b in range(B):
        for h in range(hkv):
            for t in range(lens[b].item()):
                at = kpos[0, b, h, t].item()
                row = kept_rows[b][at]
                for p, r in zip(pools, row):
                    assert torch.equal(p[table[b][t // 16], h, t % 16], r[h])
    # a tree on the evicted cache: positions go on from the whole sequence's length
    ns, most = [5, 3], 5
    first = [0, 5, 8]
    parents = i32([-1, 0, 0, 1, 2, -1, 0, 1])
    toks = i32(rng.integers(0, 50, 8))
    base = lens.tolist()
    lens += i32(ns)
    total += i32(ns)
    masks = torch.zeros(8, dtype=torch.int64, device=DEV)
    pos, slots = i32([0] * 8), i32([0] * 8)
    binding.paged_tree_plan(parents, i32(first), lens, dtable, blocks, most, masks, pos, slots,
                            total_lens=total, err=err)
    torch.cuda.synchronize()
    want = oracle.tree_plan(parents.tolist(), first, lens.tolist(), table, total.tolist())
    assert pos.tolist() == want[1] and slots.tolist() == want[2]
    assert min(want[1]) == total.tolist()[0] - 5
    q = append(m, 0, pools, toks, slots, pos)
    out = torch.zeros_like(q)
    tws = torch.zeros(binding.paged_tree_attn_ws_bytes(hq, hkv, D, most), dtype=torch.uint8, device=DEV)
    binding.paged_tree_attn_ws(q, out, *pools, dtable, i32(first), masks, lens, most, width * 16, tws,
                               scale=scale, err=err)
    args = (f64(q), f64(pools[0]), f64(pools[1]), table, first, want[0], lens.tolist(), scale)
    ref, spread = oracle.tree_attention(*args), oracle.tree_attention(*args, weight_of=np.abs)
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * spread
    assert np.all(np.abs(f64(out) - ref) <= bound)
    path, count, nxt = i32(np.zeros((B, most))), i32([0] * B), i32([0] * B)
    targets = i32([toks[2].item(), 0, toks[4].item(), 0, 7, toks[6].item(), 99, 1])
    binding.paged_tree_accept(pools, parents, toks, targets, slots, i32(first), lens, path, count,
                              nxt, lens, err)
    torch.cuda.synchronize()
    walk = oracle.tree_accept(parents.tolist(), toks.tolist(), targets.tolist(), first,
                              [x + n for x, n in zip(base, ns)], most)
    assert path.tolist() == walk[0] and lens.tolist() == walk[3] and err.item() == 0


def test_freed_blocks_by_reference_counts():
    """What an eviction frees: counts taken back with the old lengths and given
    with the new ones leave the blocks behind the budget without a holder."""
    rng = np.random.default_rng(4)
    width, blocks = 20, 45
    table = rng.permutation(blocks)[:2 * width].reshape(2, width)
    refs, old = i32(np.zeros(blocks)), i32([320, 100])
    binding.paged_kv_ref_blocks(i32(table), old, refs, 1)
    pools = [torch.randn((blocks, 1, 16, 128), device=DEV).to(BF) for _ in range(2)]
    mass = torch.rand((1, 2, 1, width * 16), device=DEV)
    kpos = torch.full(mass.shape, -1, dtype=torch.int32, device=DEV)
    ws = torch.zeros(binding.paged_kv_evict_ws_bytes(1, 2, 1, width, 64), dtype=torch.uint8, device=DEV)
    new = i32([0, 0])
    binding.paged_kv_evict(pools, mass, kpos, i32(table), old, None, 64, 4, 16, mass, kpos, new, ws,
                           refcounts=refs)
    binding.paged_kv_ref_blocks(i32(table), old, refs, -1)
    binding.paged_kv_ref_blocks(i32(table), new, refs, 1)
    torch.cuda.synchronize()
    want = np.zeros(blocks)
    for b in range(2):
        want[table[b][:4]] = 1
    assert new.tolist() == [64, 64] and refs.tolist() == want.tolist()


def test_all_four_calls_in_one_graph():
    """Plan, attention, acceptance and eviction captured on one stream and replayed
    on new data give what the calls give one by one."""
    D, hq, hkv = 128, 4, 1
    g = torch.Generator(device=DEV).manual_seed(2)
    pools = [torch.randn((40, hkv, 16, D), generator=g, device=DEV).to(BF) for _ in range(2)]
    table, first = i32(np.arange(32).reshape(2, 16)), i32([0, 6, 9])
    parents = i32([-1, 0, 0, 1, 1, 2, -1, 0, 1])
    q = torch.randn((9, hq, D), generator=g, device=DEV).to(BF)
    state = dict(tokens=i32([1, 2, 3, 4, 5, 6, 1, 2, 3]), targets=i32([3, 0, 6, 0, 0, 9, 2, 3, 4]),
                 lens=i32([200, 90]), mass=torch.rand((1, 2, hkv, 256), generator=g, device=DEV),
                 kpos=torch.full((1, 2, hkv, 256), -1, dtype=torch.int32, device=DEV), k=pools[0],
                 v=pools[1])
    was = {name: x.clone() for name, x in state.items()}
    outs = dict(masks=torch.zeros(9, dtype=torch.int64, device=DEV), pos=i32([0] * 9),
                slots=i32([0] * 9), out=torch.zeros_like(q), path=i32(np.zeros((2, 6))),
                count=i32([0, 0]), nxt=i32([0, 0]))
    tws = torch.zeros(binding.paged_tree_attn_ws_bytes(hq, hkv, D, 6), dtype=torch.uint8, device=DEV)
    ews = torch.zeros(binding.paged_kv_evict_ws_bytes(1, 2, hkv, 16, 100), dtype=torch.uint8, device=DEV)

    def step():
        s, o = state, outs
        binding.paged_tree_plan(parents, first, s["lens"], table, 40, 6, o["masks"], o["pos"], o["slots"])
        binding.paged_tree_attn_ws(q, o["out"], *pools, table, first, o["masks"], s["lens"], 6, 256,
                                   tws, scale=0.1)
        binding.paged_tree_accept(pools, parents, s["tokens"], s["targets"], o["slots"], first,
                                  s["lens"], o["path"], o["count"], o["nxt"], s["lens"])
        binding.paged_kv_evict(pools, s["mass"], s["kpos"], table, s["lens"], None, 100, 4, 16,
                               s["mass"], s["kpos"], s["lens"], ews)

    def reset(shift):
        for name, x in was.items():
            state[name].copy_(x)
        state["lens"] -= shift
        state["targets"][0] = 3 if shift == 0 else 2

    results = {}
    for shift in (0, 17):
        reset(shift)
        step()
        torch.cuda.synchronize()
        results[shift] = [x.clone() for x in (*state.values(), *outs.values())]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for shift in (17, 0, 17):
        reset(shift)
        graph.replay()
        torch.cuda.synchronize()
        for x, w in zip((*state.values(), *outs.values()), results[shift]):
            assert torch.equal(x, w)


def _good():
    bf = dict(dtype=BF, device=DEV)
    k, v = torch.zeros((8, 2, 16, 128), **bf), torch.zeros((8, 2, 16, 128), **bf)
    table, first = i32(np.arange(4).reshape(1, 4)), i32([0, 3])
    return dict(k=k, v=v, table=table, first=first, lens=i32([20]), parents=i32([-1, 0, 0]),
                masks=torch.ones(3, dtype=torch.int64, device=DEV), pos=i32([0] * 3),
                slots=i32([0] * 3), q=torch.zeros((3, 8, 128), **bf), out=torch.zeros((3, 8, 128), **bf),
                ws=torch.zeros(binding.paged_tree_attn_ws_bytes(8, 2, 128, 3), dtype=torch.uint8,
                               device=DEV), path=i32([[0] * 3]), one=i32([0]),
                mass=torch.zeros((1, 1, 2, 64), device=DEV), kpos=i32(np.full((1, 1, 2, 64), -1)),
                err=i32([0]))


CALLS = dict(
    plan=lambda c: binding.paged_tree_plan(c["parents"], c["first"], c["lens"], c["table"], 8, 3,
                                           c["masks"], c["pos"], c["slots"], err=c["err"]),
    attn=lambda c: binding.paged_tree_attn_ws(c["q"], c["out"], c["k"], c["v"], c["table"], c["first"],
                                              c["masks"], c["lens"], 3, 64, c["ws"], scale=0.1,
                                              err=c["err"]),
    accept=lambda c: binding.paged_tree_accept([c["k"], c["v"]], c["parents"], c["pos"], c["pos"],
                                               c["slots"], c["first"], c["lens"], c["path"], c["one"],
                                               c["one"], c["one"], c["err"]),
    evict=lambda c: binding.paged_kv_evict([c["k"], c["v"]], c["mass"], c["kpos"], c["table"], c["lens"],
                                           None, 10, 1, 2, c["mass"], c["kpos"], c["one"], c["ws"],
                                           err=c["err"]))


@pytest.mark.parametrize("call,name", [
    ("plan", "parents"), ("plan", "first"), ("plan", "lens"), ("plan", "table"), ("plan", "masks"),
    ("plan", "pos"), ("plan", "slots"), ("plan", "err"), ("attn", "q"), ("attn", "out"), ("attn", "k"),
    ("attn", "v"), ("attn", "table"), ("attn", "first"), ("attn", "masks"), ("attn", "lens"),
    ("attn", "err"), ("accept", "k"), ("accept", "v"), ("accept", "parents"), ("accept", "pos"),
    ("accept", "slots"), ("accept", "first"), ("accept", "lens"), ("accept", "path"), ("accept", "one"),
    ("evict", "k"), ("evict", "v"), ("evict", "mass"), ("evict", "kpos"), ("evict", "table"),
    ("evict", "lens"), ("evict", "one"), ("evict", "err")])
def test_tensors_that_do_not_fit_are_refused(call, name):
    """Another type, a strided view, another shape, a host tensor, no tensor: each is
    refused before anything runs, and the right one is taken."""
    CALLS[call](_good())
    x = _good()[name]
    wider = torch.zeros((*x.shape[:-1], 2 * x.shape[-1]), dtype=x.dtype, device=DEV)[..., ::2]
    bad = [x.double(), x.cpu(), "no tensor"]
    if x.numel() > 1:
        bad.append(wider)
    if name not in ("err",):
        bad.append(torch.zeros((*x.shape[:-1], x.shape[-1] + 1), dtype=x.dtype, device=DEV))
        bad.append(x[None])
    for y in bad:
        # (a table or a path may be wider, and then a mass no longer fits it)
        if call != "evict" and name in ("table", "path") and y is not x and \
                getattr(y, "is_cuda", False) and y.dtype is x.dtype and y.is_contiguous() and y.dim() == 2:
            continue
        with pytest.raises(ValueError):
            CALLS[call](dict(_good(), **{name: y}))
    torch.cuda.synchronize()


def test_refusals_of_the_library_reach_python():
    c = _good()
    with pytest.raises(binding.PagedAttnError, match="PKA_ERR_WORKSPACE"):
        CALLS["attn"](dict(c, ws=c["ws"][:1000]))
    with pytest.raises(binding.PagedAttnError, match="PKA_ERR_ALIGN"):
        CALLS["attn"](dict(c, ws=c["ws"][8:]))
    with pytest.raises(binding.PagedAttnError, match="PKA_ERR_UNSUPPORTED"):
        binding.paged_tree_plan(c["parents"], c["first"], c["lens"], c["table"], 8, 65, None, None,
                                c["slots"])
    with pytest.raises(binding.PagedAttnError, match="PKA_ERR_SHAPE"):
        binding.paged_kv_evict([c["k"], c["v"]], c["mass"], c["kpos"], c["table"], c["lens"], None, 5,
                               4, 4, c["mass"], c["kpos"], c["one"], c["ws"])
    with pytest.raises(ValueError, match="pools"):
        binding.paged_kv_evict([c["k"]], c["mass"], c["kpos"], c["table"], c["lens"], None, 5, 1, 1,
                               c["mass"], c["kpos"], c["one"], c["ws"])
    with pytest.raises((ValueError, TypeError)):
        binding.paged_kv_evict([c["k"], c["v"]], c["mass"], c["kpos"], c["table"], c["lens"], None,
                               2 ** 40, 1, 1, c["mass"], c["kpos"], c["one"], c["ws"])
    # nothing to do: no rows, no requests
    none = i32([]).view(0, 4)
    binding.paged_tree_plan(i32([]), i32([0]), i32([]), none, 8, 3, None, None, i32([]))
    binding.paged_tree_attn_ws(c["q"][:0], c["out"][:0], c["k"], c["v"], none, i32([0]), c["masks"][:0],
                               i32([]), 3, 64, c["ws"], scale=0.1)
    binding.paged_tree_accept([], i32([]), i32([]), i32([]), None, i32([0]), i32([]), i32([]).view(0, 3),
                              i32([]), i32([]), i32([]))
    torch.cuda.synchronize()
