"""Cases of the draft-tree operators and of the eviction by attention mass.

A step of speculative decoding over a block-paged cache verifies a tree of
drafted tokens per request: ``plan`` gives the tokens' ancestor masks,
positions and cache slots, ``tree`` is the attention of one layer, ``accept``
walks the trees and moves the accepted tokens' K/V rows up.  ``evict`` holds a
cache to a budget of keys per request and KV head: the first keys, the most
recent ones and those that have drawn the most attention stay.

``own`` false: every operator in plain torch operations.  True: the
library's calls.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # two chats with small trees: launch latency
        dict(name="tree tiny", op="tree", b=2, lo=20, hi=250, nlo=4, nhi=7, hq=8, hkv=2, d=128,
             window=0, softcap=0.0, pool=64),
        # one layer of a serving step that verifies trees: full attention, logit cap
        dict(name="tree serving", op="tree", b=32, lo=512, hi=4096, nlo=8, nhi=16, hq=8, hkv=2,
             d=256, window=0, softcap=50.0, pool=16384),
        # its sliding layer
        dict(name="tree sliding", op="tree", b=32, lo=512, hi=4096, nlo=8, nhi=16, hq=8, hkv=2,
             d=256, window=512, softcap=50.0, pool=16384),
        # long documents, trees of up to 32 tokens
        dict(name="tree long", op="tree", b=4, lo=32768, hi=131072, nlo=17, nhi=32, hq=16, hkv=4,
             d=128, window=0, softcap=0.0, pool=32768),
        # the widest trees: 64 tokens of 4 heads, 256 rows for each KV head
        dict(name="tree wide", op="tree", b=8, lo=2001, hi=8003, nlo=49, nhi=64, hq=8, hkv=2,
             d=256, window=0, softcap=0.0, pool=8192),
        # the plan of a small and of a large step
        dict(name="plan few", op="plan", b=4, lo=20, hi=300, nlo=3, nhi=8, pool=128),
        dict(name="plan many", op="plan", b=256, lo=500, hi=4000, nlo=33, nhi=64, pool=65536),
        # acceptance in a small step, one layer's pools
        dict(name="accept few", op="accept", b=4, lo=20, hi=300, nlo=3, nhi=8, pool=128, layers=1,
             hkv=2, d=128),
        # acceptance of wide trees, four layers at once
        dict(name="accept many", op="accept", b=64, lo=100, hi=2000, nlo=33, nhi=64, pool=8192,
             layers=4, hkv=2, d=256),
        # one chat over its budget
        dict(name="evict chat", op="evict", b=1, lo=411, hi=411, budget=256, sinks=4, recent=64,
             layers=1, hkv=2, d=128, pool=64),
        # a serving batch cut to 1000 keys a head, two layers at once
        dict(name="evict serving", op="evict", b=32, lo=700, hi=4096, budget=1000, sinks=4,
             recent=256, layers=2, hkv=2, d=256, pool=8192),
        # long documents cut to 16384 keys
        dict(name="evict long", op="evict", b=4, lo=32768, hi=131072, budget=16384, sinks=16,
             recent=4096, layers=1, hkv=4, d=128, pool=32768),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "plan", "accept", "evict", "evict"])
    d = rng.choice([128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    nhi = _log(rng, 1, 64)
    nlo = rng.randint(1, nhi)
    if op == "tree":
        b = _log(rng, 1, 64)
        g = rng.choice([1, 2, 4, 8])
        # at most the keys, and the products, of the largest listed cases
        most = min(131072, 250000 * 512 // (b * hkv * d), 2 ** 31 // (b * hkv * g * nhi * d))
        hi = nhi + _log(rng, 1, max(1, most))
        lo = rng.randint(nlo, hi)
        window = rng.choice([0, 0, _log(rng, 1, 4096)])
        cap = rng.choice([0.0, 0.0, 30.0, 50.0])
        return dict(op=op, b=b, lo=lo, hi=hi, nlo=nlo, nhi=nhi, hq=g * hkv, hkv=hkv, d=d,
                    window=window, softcap=cap, pool=b * ((hi + 15) // 16) + rng.randint(1, 64))
    if op == "evict":
        layers = rng.randint(1, 3)
        b = _log(rng, 1, 32)
        hi = _log(rng, 16, max(17, min(131072, 131072 * 512 * 2 // (b * hkv * d * layers))))
        budget = _log(rng, 1, max(1, hi - 1))
        sinks = rng.randint(0, min(16, budget))
        recent = rng.randint(0, budget - sinks)
        return dict(op=op, b=b, lo=rng.randint(1, hi), hi=hi, budget=budget, sinks=sinks,
                    recent=recent, layers=layers, hkv=hkv, d=d,
                    pool=b * ((hi + 15) // 16) + rng.randint(1, 64))
    b = _log(rng, 1, 256 if op == "plan" else 64)
    hi = nhi + _log(rng, 1, 2000)
    case = dict(op=op, b=b, lo=rng.randint(nhi, hi), hi=hi, nlo=nlo, nhi=nhi,
                pool=b * ((hi + 15) // 16) + rng.randint(1, 64))
    if op == "accept":
        case.update(layers=rng.randint(1, 4), hkv=min(hkv, 2), d=d)
    return case


def _spread(lo, hi, b):
    """b values over the whole range, evenly."""
    return [hi] if b == 1 else [lo + (hi - lo) * i // (b - 1) for i in range(b)]


def _batch(case, host):
    """Lengths and tree sizes of the requests; which request has which is drawn."""
    b = case["b"]
    lens = torch.tensor(_spread(case["lo"], case["hi"], b))[torch.randperm(b, generator=host)]
    if "nhi" not in case:
        return lens, None
    n = torch.tensor(_spread(case["nlo"], case["nhi"], b))[torch.randperm(b, generator=host)]
    return torch.maximum(lens, n), n


def work(case):
    op = case["op"]
    b = case["b"]
    lens = _spread(case["lo"], case["hi"], b)
    if op == "evict":
        rows = case["hkv"] * case["layers"]
        # the keys past the budget that stay and have to move: the recent ones,
        # and of the others as many as a mass that knows no place gives
        moved = 0
        for x in lens:
            past, held = x - case["budget"], case["sinks"] + case["recent"]
            if past > 0:
                tail = min(past, case["recent"])
                moved += tail + (case["budget"] - held) * (past - tail) // max(1, x - held)
        return dict(bytes=rows * (sum(lens) * 16 + moved * 8 * case["d"]), flops=rows * sum(lens))
    n = _spread(case["nlo"], case["nhi"], b)
    if op == "plan":
        return dict(bytes=sum(n) * 24 + b * 12, flops=sum(n) * 4)
    if op == "accept":
        # tokens, parents, targets and slots of the trees, and a moved row for each request
        return dict(bytes=sum(n) * 16 + b * 20 + b * 4 * case["nhi"] +
                    b * case["layers"] * case["hkv"] * 8 * case["d"], flops=sum(n) * 4)
    w = case["window"]
    seen = [min(x, w + y) if w > 0 else x for x, y in zip(lens, n)]
    keys, rows = sum(seen), sum(n) * case["hq"]
    pairs = sum(y * min(x, w if w > 0 else x) for x, y in zip(lens, n)) * case["hq"]
    return dict(bytes=keys * case["hkv"] * 4 * case["d"] + rows * 4 * case["d"] + sum(n) * 8 +
                sum((x + 15) // 16 for x in seen) * 4, flops=4 * pairs * case["d"])


# ------------------------------------------------------------------ states
def _tables(lens, pool, width, host):
    table = torch.full((lens.numel(), width), -1, dtype=torch.int32)
    perm, at = torch.randperm(pool, generator=host), 0
    for i, n in enumerate(((lens + 15) // 16).tolist()):
        table[i, :n] = perm[at:at + n]
        at += n
    return table


def _trees(n, host):
    """Parents of every tree's tokens (-1: the root, its token 0), in request order."""
    own_index = torch.cat([torch.arange(x) for x in n.tolist()])
    back = torch.randint(1, 7, (own_index.numel(),), generator=host)
    return torch.where(own_index > 0, (own_index - back).clamp(min=0), torch.tensor(-1))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    op, b = case["op"], case["b"]
    i32 = dict(dtype=torch.int32, device=DEV)
    lens, n = _batch(case, host)
    width = max(1, (case["hi"] + 15) // 16)
    s = dict(op=op, b=b, lens=lens.to(**i32),
             tables=_tables(lens, case["pool"], width, host).to(**i32))

    def pool():
        return torch.randn((case["pool"], case["hkv"], 16, case["d"]), generator=gen, device=DEV,
                           dtype=torch.bfloat16)

    if op == "evict":
        shape = (case["layers"], b, case["hkv"], width * 16)
        # a few keys draw most of the attention; keys drawn less than once in
        # 2^-10 of a step share a mass
        mass = torch.exp(2.0 * torch.randn(shape, generator=gen, device=DEV))
        mass = torch.round(mass * 1024) / 1024
        # some requests were cut before: their first keys are out of order
        # and keep their positions, the keys since then have none yet
        total = lens + torch.randint(0, 500, (b,), generator=host)
        total = torch.where(torch.arange(b) % 2 == 0, lens, total)
        pos = torch.full(shape, -1, dtype=torch.int32, device=DEV)
        for i in range(1, b, 2):
            old = int(lens[i]) // 2
            older = torch.randperm(int(total[i] - lens[i]) + old, generator=host)[:old]
            pos[:, i, :, :old] = older.to(**i32)
        s.update(pools=[pool() for _ in range(2 * case["layers"])], mass=mass, pos=pos,
                 total=total.to(**i32), budget=case["budget"], sinks=case["sinks"],
                 recent=case["recent"], new_mass=torch.zeros(shape, device=DEV),
                 new_pos=torch.zeros(shape, **i32), new_lens=torch.zeros(b, **i32),
                 # room for every key's move, twice
                 workspace=torch.zeros(64 + 4 * shape[0] * b * shape[2] * (64 + 2 * shape[3]),
                                       dtype=torch.uint8, device=DEV))
        return s
    pad = 3  # rows behind the last request, as a batch of a fixed size has
    first = torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)])
    rows = int(first[-1]) + pad
    parents = torch.cat([_trees(n, host), torch.full((pad,), -1)])
    s.update(first=first.to(**i32), parents=parents.to(**i32), rows=rows, most=case["nhi"],
             max_len=max(case["hi"], case["nhi"]), blocks=case["pool"])
    if op == "plan":
        s.update(total=(lens + 7).to(**i32),
                 masks=torch.zeros(rows, dtype=torch.int64, device=DEV),
                 positions=torch.zeros(rows, **i32), slots=torch.zeros(rows, **i32))
        return s
    if op == "accept":
        # drafted tokens of a small vocabulary; the target agrees with a
        # drafted child of about three tokens in four
        tokens = torch.randint(0, 1000, (rows,), generator=host)
        targets = torch.randint(0, 1000, (rows,), generator=host)
        tree = torch.bucketize(torch.arange(rows), first[1:], right=True).clamp(max=b - 1)
        whose = first[tree] + parents.clamp(min=0)
        agree = (torch.rand(rows, generator=host) < 0.75) & (parents >= 0)
        targets[whose[agree]] = tokens[agree]
        slot_at = lens[tree] - n[tree] + torch.arange(rows) - first[tree]
        table = s["tables"].cpu().long()
        slots = table[tree, (slot_at // 16).clamp(max=width - 1)] * 16 + slot_at % 16
        slots[int(first[-1]):] = -1
        s.update(pools=[pool() for _ in range(2 * case["layers"])], tokens=tokens.to(**i32),
                 targets=targets.to(**i32), slots=slots.to(**i32),
                 path=torch.zeros((b, case["nhi"]), **i32), accepted=torch.zeros(b, **i32),
                 next_tokens=torch.zeros(b, **i32), new_lens=torch.zeros(b, **i32))
        return s
    d, hq = case["d"], case["hq"]
    masks = torch.zeros(rows, dtype=torch.int64)
    for lo, hi in zip(first[:-1].tolist(), first[1:].tolist()):
        up = parents[lo:hi].tolist()
        bits = []
        for i, p in enumerate(up):
            bits.append((1 << i) | (bits[p] if p >= 0 else 0))
        masks[lo:hi] = torch.tensor([x - (1 << 64) if x >> 63 else x for x in bits])
    s.update(k=pool(), v=pool(), masks=masks.to(DEV), hkv=case["hkv"], window=case["window"],
             softcap=case["softcap"], scale=1.0 / math.sqrt(d),
             q=torch.randn((rows, hq, d), generator=gen, device=DEV).to(torch.bfloat16),
             out=torch.zeros((rows, hq, d), dtype=torch.bfloat16, device=DEV),
             # room for two partial tiles of 128 rows on each SM
             workspace=torch.zeros(320 * 128 * (d + 1) * 4 + 65536, dtype=torch.uint8, device=DEV))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from paged_kv_attention_12_gb300 import binding
    op = s["op"]
    if op == "tree":
        binding.paged_tree_attn_ws(s["q"], s["out"], s["k"], s["v"], s["tables"], s["first"],
                                   s["masks"], s["lens"], s["most"], s["max_len"], s["workspace"],
                                   scale=s["scale"], softcap=s["softcap"], window=s["window"])
        return s["out"]
    if op == "plan":
        binding.paged_tree_plan(s["parents"], s["first"], s["lens"], s["tables"], s["blocks"],
                                s["most"], s["masks"], s["positions"], s["slots"],
                                total_lens=s["total"])
        return s["masks"], s["positions"], s["slots"]
    if op == "accept":
        binding.paged_tree_accept(s["pools"], s["parents"], s["tokens"], s["targets"], s["slots"],
                                  s["first"], s["lens"], s["path"], s["accepted"],
                                  s["next_tokens"], s["new_lens"])
        return s["path"], s["accepted"], s["next_tokens"], s["new_lens"], s["pools"]
    binding.paged_kv_evict(s["pools"], s["mass"], s["pos"], s["tables"], s["lens"], s["total"],
                           s["budget"], s["sinks"], s["recent"], s["new_mass"], s["new_pos"],
                           s["new_lens"], s["workspace"])
    return s["new_mass"], s["new_pos"], s["new_lens"], s["pools"]


def _grid(s):
    """Every request's tree, padded: rows [B][most] of the batch, which of them are its
    own, and for each row of the batch its request and index."""
    first = s["first"].long()
    i = torch.arange(s["most"], device=DEV)
    n = first[1:] - first[:-1]
    at = (first[:-1, None] + i).clamp(max=s["rows"] - 1)
    row = torch.arange(s["rows"], device=DEV)
    req = torch.searchsorted(first[1:].contiguous(), row, right=True).clamp(max=s["b"] - 1)
    return at, i < n[:, None], n, req, row - first[req], row < first[-1]


def _ancestors(s, at, mine):
    """[B][most][most]: whether token j is token i or one of its ancestors."""
    m = s["most"]
    i = torch.arange(m, device=DEV)
    a = ((s["parents"].long()[at][:, :, None] == i) | (i[:, None] == i)) & mine[:, :, None]

    def squared(x):
        return (torch.matmul(x.float(), x.float()) > 0)

    return squared(squared(squared(squared(squared(squared(a))))))


def _run_plain(s):
    op = s["op"]
    if op == "evict":
        return _plain_evict(s)
    at, mine, n, req, i_row, owned = _grid(s)
    base = s["lens"].long() - n
    if op == "plan":
        up = _ancestors(s, at, mine)
        i = torch.arange(s["most"], device=DEV)
        masks = (up.long() << i).sum(-1)[req, i_row.clamp(max=s["most"] - 1)]
        depth = (up.sum(-1) - 1)[req, i_row.clamp(max=s["most"] - 1)]
        t = base[req] + i_row
        slots = s["tables"].long()[req, (t // 16).clamp(max=s["tables"].shape[1] - 1)] * 16 + t % 16
        zero = torch.zeros_like(masks)
        s["masks"].copy_(torch.where(owned, masks, zero))
        s["positions"].copy_(torch.where(owned, (s["total"].long() - n)[req] + depth, zero))
        s["slots"].copy_(torch.where(owned, slots, zero - 1))
        return s["masks"], s["positions"], s["slots"]
    if op == "accept":
        up = _ancestors(s, at, mine)
        parent, token = s["parents"].long()[at], s["tokens"][at]
        i = torch.arange(s["most"], device=DEV)
        want = s["targets"][at].gather(1, parent.clamp(min=0))
        match = mine & (parent >= 0) & (token == want)
        twin = match[:, :, None] & match[:, None, :] & (parent[:, :, None] == parent[:, None, :])
        match = match & ~(twin & (i[None, :] < i[:, None])).any(-1)
        match[:, 0] = mine[:, 0]
        took = (match[:, None, :] | ~up).all(-1) & mine & up[:, :, 0]
        count = took.sum(-1)
        rank = torch.where(took, took.cumsum(-1) - 1, torch.full_like(at, s["most"]))
        path = torch.full((s["b"], s["most"] + 1), -1, device=DEV)
        path = path.scatter(1, rank, i.expand_as(rank))[:, :s["most"]]
        last = path.amax(-1).clamp(min=0)
        s["path"].copy_(path)
        s["accepted"].copy_(count)
        s["next_tokens"].copy_(s["targets"][at].gather(1, last[:, None])[:, 0])
        s["new_lens"].copy_(base + count)
        slots = s["slots"].long()[at]
        here, k = (path >= 0).nonzero(as_tuple=True)
        src, dst = slots[here, path[here, k]], slots[here, k]

        def move(p):
            p[dst // 16, :, dst % 16] = p[src // 16, :, src % 16]
            return p

        return s["path"], s["accepted"], s["next_tokens"], s["new_lens"], list(map(move, s["pools"]))
    # attention: the requests' keys side by side, padded to the longest
    b, hkv, (rows, hq, d) = s["b"], s["hkv"], s["q"].shape
    ids = s["tables"].clamp(min=0).long()
    keys = ids.shape[1] * 16
    key = torch.arange(keys, device=DEV)
    mask = s["masks"][at]
    bits = (mask[:, :, None] >> torch.arange(s["most"], device=DEV)) & 1        # [B][i][j]
    depth = bits.sum(-1) - 1
    seen = (key < base[:, None])[:, None].expand(b, s["most"], keys)
    j = key - base[:, None]                                                     # [B][keys]
    drafted = (j >= 0) & (j < n[:, None])
    tree = bits.bool()
    if s["window"] > 0:
        seen = seen & (key > (base[:, None] + depth)[:, :, None] - s["window"])
        tree = tree & (depth[:, :, None] - depth[:, None, :] < s["window"])
    jj = j.clamp(min=0, max=s["most"] - 1)[:, None].expand(b, s["most"], keys)
    seen = seen | (tree.gather(2, jj) & drafted[:, None])
    q = s["q"][at].float().view(b, -1, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    k = s["k"][ids.flatten()].float().view(b, -1, hkv, 16, d).transpose(1, 2).reshape(b, hkv, keys, d)
    x = torch.matmul(q.reshape(b, hkv, -1, d), k.transpose(2, 3)) * s["scale"]
    del k
    if s["softcap"] > 0:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    x = x.view(b, hkv, -1, s["most"], keys).masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    del x
    v = s["v"][ids.flatten()].float().view(b, -1, hkv, 16, d).transpose(1, 2).reshape(b, hkv, keys, d)
    v = torch.where((key < s["lens"][:, None])[:, None, :, None], v, torch.zeros_like(v[:1, :1]))
    y = torch.matmul(p.view(b, hkv, -1, keys), v).view(b, hkv, -1, s["most"], d)
    y = y / p.sum(-1, keepdim=True).clamp(min=1e-30)
    y = y.permute(0, 3, 1, 2, 4).reshape(b, s["most"], hq, d)[req, i_row.clamp(max=s["most"] - 1)]
    s["out"].copy_(torch.where(owned[:, None, None], y, s["out"].float()))
    return s["out"]


def _plain_evict(s):
    mass, lens = s["mass"], s["lens"].long()
    keys = mass.shape[-1]
    t = torch.arange(keys, device=DEV)
    total = s["total"].long()[:, None, None]
    L = lens[:, None, None]
    pos = torch.where(s["pos"] >= 0, s["pos"].long(), total - (L - t))
    valid = (t < L).expand_as(pos)
    held = valid & ((pos < s["sinks"]) | (pos >= total - s["recent"]))
    # the keys in the order in which they stay: held ones, then by mass, then by index
    order = torch.sort(torch.where(held, torch.zeros_like(mass), mass), dim=-1, descending=True,
                       stable=True).indices
    group = torch.where(held, 0, torch.where(valid, 1, 2)).gather(-1, order)
    order = order.gather(-1, torch.sort(group, dim=-1, stable=True).indices)
    rank = torch.empty_like(order).scatter(-1, order, t.expand_as(order))
    n = torch.clamp(L, max=s["budget"])
    keep = rank < n
    hole, mover = ~keep & (t < n), keep & (t >= n)
    place = torch.where(hole, hole.cumsum(-1) - 1, torch.full_like(order, keys))
    spots = torch.zeros((*order.shape[:-1], keys + 1), dtype=torch.long, device=DEV)
    spots = spots.scatter(-1, place, t.expand_as(place))
    from_top = mover.flip(-1).cumsum(-1).flip(-1) - 1
    layer, req, head, src = mover.nonzero(as_tuple=True)
    dst = spots[layer, req, head, from_top[layer, req, head, src]]
    kept = t < n
    new_mass = torch.where(kept, mass, torch.where(valid, torch.zeros_like(mass), s["new_mass"]))
    new_pos = torch.where(kept, pos.int(), torch.where(valid, torch.full_like(s["pos"], -1),
                                                      s["new_pos"]))
    new_mass[layer, req, head, dst] = mass[layer, req, head, src]
    new_pos[layer, req, head, dst] = pos[layer, req, head, src].int()
    s["new_mass"].copy_(new_mass)
    s["new_pos"].copy_(new_pos)
    s["new_lens"].copy_(n[:, 0, 0])
    table = s["tables"].long()
    pools = torch.arange(len(s["pools"]), device=DEV) // 2

    def move(item):
        which, p = item
        mine = layer == which // 2
        h, b = head[mine], req[mine]
        x, y = src[mine], dst[mine]
        p[table[b, y // 16], h, y % 16] = p[table[b, x // 16], h, x % 16]
        return p

    return s["new_mass"], s["new_pos"], s["new_lens"], list(map(move, enumerate(s["pools"])))


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    if case["op"] != "tree":
        # masks, slots, walks and moves: nothing is computed beyond whole numbers
        return None
    s = prepare(case, seed)
    hkv, (rows, hq, d) = case["hkv"], s["q"].shape
    out = torch.zeros((rows, hq, d), dtype=torch.float64, device=DEV)
    first = s["first"].tolist()
    for i, n_keys in enumerate(s["lens"].tolist()):
        lo, hi = first[i], first[i + 1]
        n = hi - lo
        base = n_keys - n
        # whether query a sees key t, from the parents and not from the masks
        up = s["parents"][lo:hi].tolist()
        depth, tree = [], torch.zeros((n, n), dtype=torch.bool)
        for a in range(n):
            tree[a, a] = True
            if up[a] >= 0:
                tree[a] |= tree[up[a]]
            depth.append(depth[up[a]] + 1 if up[a] >= 0 else 0)
        place = torch.tensor(list(range(base)) + [base + x for x in depth], device=DEV)
        sees = torch.cat([torch.ones((n, base), dtype=torch.bool), tree], 1).to(DEV)
        if s["window"] > 0:
            sees &= place[None] > place[base:, None] - s["window"]
        start = int(sees.any(0).int().argmax()) // 16 * 16
        ids = s["tables"][i, start // 16:(n_keys + 15) // 16].long()
        k = s["k"][ids].double().transpose(0, 1).flatten(1, 2)[:, :n_keys - start]
        q = s["q"][lo:hi].double().view(n, hkv, hq // hkv, d)
        x = torch.einsum("nhgd,htd->hgnt", q, k) * s["scale"]
        if s["softcap"] > 0:
            x = s["softcap"] * torch.tanh(x / s["softcap"])
        x = x.masked_fill(~sees[:, start:], -math.inf)
        p = torch.exp(x - x.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        v = s["v"][ids].double().transpose(0, 1).flatten(1, 2)[:, :n_keys - start]
        out[lo:hi] = torch.einsum("hgnt,htd->nhgd", p, v).reshape(n, hq, d)
    return out
