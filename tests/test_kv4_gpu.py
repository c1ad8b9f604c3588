"""GPU checks of the 4-bit cache: writing (bit by bit), expanding (bit by bit)
and decode attention against the fp64 oracle, at the sizes, masks and contents
where they can go wrong."""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_kv_attention_12_gb300 import _build, binding, workload

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KS, VS = 0.0047, 0.0019


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    binding.lib()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def rows(shape, seed, spread=0.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    mag = torch.exp(spread * torch.randn(shape[-1], generator=g, device=DEV))
    return (torch.randn(shape, generator=g, device=DEV) * mag).to(torch.bfloat16)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def random_pool(nb, hkv, D, seed, ks=KS, vs=VS):
    """A full pool, written by the oracle's rounding of random rows."""
    rng = np.random.default_rng(seed)
    out = []
    for is_v, s in ((False, ks), (True, vs)):
        x = rng.standard_normal((nb * 16, hkv, D)) * np.exp(0.5 * rng.standard_normal(D))
        p = oracle.kv4_append(np.zeros((nb, hkv, D // 128, 1152), np.uint8), x, range(nb * 16), s,
                              is_v)
        out.append(torch.from_numpy(p).to(DEV))
    return binding.Kv4Pool(out[0], out[1], ks, vs)


def byte_pool(nb, hkv, D, seed, ks=KS, vs=VS):
    """A full pool of random codes, with scales from 0.25 to 4: quick to make."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    out = []
    for _ in range(2):
        p = torch.randint(0, 256, (nb, hkv, D // 128, 1152), generator=g, device=DEV,
                          dtype=torch.uint8)
        p[..., 1024:] = p[..., 1024:] % 33 + 0x28
        out.append(p)
    return binding.Kv4Pool(out[0], out[1], ks, vs)


# ---------------------------------------------------------------- write
@pytest.mark.parametrize("D,hkv,T,wide", [(128, 1, 1, 0), (128, 3, 33, 5), (256, 2, 700, 0),
                                          (256, 8, 17, 3), (128, 4, 1025, 1)])
def test_append_bit_exact(D, hkv, T, wide):
    nb = (T + 15) // 16 + 5
    pool = random_pool(nb, hkv, D, T)
    # rows as slices of a wider projection (wide more heads)
    k_new = rows((T, hkv + wide, D), 1)[:, wide:]
    v_new = rows((T, hkv + wide, D), 2, 0.1)[:, :hkv]
    perm = torch.randperm(nb * 16, generator=torch.Generator().manual_seed(T))[:T].tolist()
    if T > 2:
        perm[1] = -1
    want = [oracle.kv4_append(p.cpu().numpy(), f64(x), perm, s, v) for p, x, s, v in
            ((pool.k, k_new, KS, False), (pool.v, v_new, VS, True))]
    err = i32([0])
    binding.paged_kv4_append(k_new, v_new, pool, i32(perm), err)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert np.array_equal(pool.k.cpu().numpy(), want[0])
    assert np.array_equal(pool.v.cpu().numpy(), want[1])


@pytest.mark.parametrize("scale", [2.0 ** -9, 0.0123, 1e-4, 1e-30, 3e37])
def test_append_borders_and_special_values(scale):
    """Values on and next to every rounding border, zeros of both signs,
    subnormals, the largest values, infinities and NaN."""
    x = []
    lv = oracle.kv4.E2M1
    mids = (lv[1:] + lv[:-1]) / 2
    for s in (1.0, 448.0, 2.0 ** -9, 0.171875, 2.0 ** -10, 1e-12):
        for sign in (1, -1):
            f = s * scale
            base = np.concatenate([[6.0], mids, mids * (1 + 2 ** -7), [0.0]])[:16]
            x.append(sign * base * f)
    r6 = oracle.kv4.E4M3[1:].astype(np.float64)
    tops = (r6[1:] + r6[:-1]) / 2 * 6 * scale            # maxima on the scales' borders
    for t in tops[:: 5]:
        x.append(np.concatenate([[t], np.linspace(-t, t, 15)]))
    x.append(np.array([np.nan] + [1.0] * 15))
    x.append(np.array([1.0] * 15 + [-np.inf]))
    x.append(np.array([-0.0, 0.0] * 8))
    x.append(np.array([1e-45, -1e-40, 9e-41] + [0.0] * 13))
    x.append(np.full(16, 3.3e38))
    x = np.concatenate(x)
    x = np.pad(x, (0, -len(x) % 256)).reshape(-1, 2, 128)
    t = torch.from_numpy(x).to(torch.bfloat16).to(DEV)
    T = t.shape[0]
    pool = binding.Kv4Pool.zeros((T + 15) // 16, 2, 128, scale, scale)
    binding.paged_kv4_append(t, t, pool, torch.arange(T, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    zero = np.zeros(pool.k.shape, np.uint8)
    for p, is_v in ((pool.k, False), (pool.v, True)):
        want = oracle.kv4_append(zero, f64(t), range(T), scale, is_v)
        assert np.array_equal(p.cpu().numpy(), want)


def test_append_slot_past_the_pool():
    pool = random_pool(4, 2, 128, 3)
    k0, v0 = pool.k.clone(), pool.v.clone()
    x = rows((3, 2, 128), 5)
    err = i32([0])
    binding.paged_kv4_append(x, x, pool, i32([64, -7, 2 ** 31 - 1]), err)
    torch.cuda.synchronize()
    assert err.item() == binding.DEVERR_BAD_TABLE
    assert torch.equal(pool.k, k0) and torch.equal(pool.v, v0)


# ---------------------------------------------------------------- expand
def bf16_bits(x32):
    return torch.from_numpy(np.ascontiguousarray(x32)).to(torch.bfloat16)


def test_append_more_heads_than_a_grid_has():
    """70000 heads of one block are the bytes of 70000 blocks of one head."""
    H, D, slots = 70000, 128, [5, 0, 9]
    k, v = rows((3, H, D), 1), rows((3, H, D), 2)
    a = binding.Kv4Pool.zeros(1, H, D, KS, VS, device=DEV)
    b = binding.Kv4Pool.zeros(H, 1, D, KS, VS, device=DEV)
    err = i32([0])
    binding.paged_kv4_append(k, v, a, i32(slots), err)
    one = torch.arange(H, device=DEV, dtype=torch.int32)[None] * 16 + i32(slots)[:, None]
    binding.paged_kv4_append(k.view(3 * H, 1, D), v.view(3 * H, 1, D), b, one.reshape(-1), err)
    assert err.item() == 0 and a.k[0, -1].any() and a.v[0, -1].any()
    assert torch.equal(a.k.view(-1), b.k.view(-1)) and torch.equal(a.v.view(-1), b.v.view(-1))
    binding.paged_kv4_append(k, v, a, i32([16, -1, 15]), err)
    assert err.item() == binding.DEVERR_BAD_TABLE


@pytest.mark.parametrize("D,hkv,n", [(128, 1, 1), (128, 3, 37), (256, 2, 90)])
def test_expand_bit_exact(D, hkv, n):
    pool = random_pool(n + 3, hkv, D, n)
    pool.k[0, 0, 0, 1024:] = 127                       # NaN scales read back as NaN
    ids = torch.randperm(n + 3, generator=torch.Generator().manual_seed(1))[:n].tolist()
    if n > 2:
        ids[1] = -1
    k16 = torch.full((n + 2, hkv, 16, D), 7.0, dtype=torch.bfloat16, device=DEV)
    v16 = k16.clone()
    to = torch.randperm(n + 2, generator=torch.Generator().manual_seed(2))[:n].tolist()
    for dst in (None, to):
        k16.fill_(7.0), v16.fill_(7.0)
        err = i32([0])
        binding.paged_kv4_expand(pool, k16, v16, i32(ids), None if dst is None else i32(dst), err)
        torch.cuda.synchronize()
        assert err.item() == 0
        for got, p, s, is_v in ((k16, pool.k, KS, False), (v16, pool.v, VS, True)):
            val = bf16_bits(oracle.kv4_decode(p.cpu().numpy(), s, is_v, exact=False))
            want = torch.full_like(got, 7.0).cpu()
            for i, b in enumerate(ids):
                if b >= 0:
                    want[i if dst is None else dst[i]] = val[b]
            assert torch.equal(got.cpu().nan_to_num(1e9), want.nan_to_num(1e9))


def test_expand_bad_ids():
    pool = random_pool(3, 1, 128, 9)
    k16 = torch.zeros((2, 1, 16, 128), dtype=torch.bfloat16, device=DEV)
    err = i32([0])
    binding.paged_kv4_expand(pool, k16, k16.clone(), i32([3, 0]), i32([0, 2]), err)
    torch.cuda.synchronize()
    assert err.item() == binding.DEVERR_BAD_TABLE and not k16.any()


# ---------------------------------------------------------------- decode
def make(lens, hq, hkv, D, *, seed=0, spare=5, qmag=1.0, scale=None, window=0, softcap=0.0,
         poison=True, pool_of=random_pool):
    """A decode call over a random pool; with poison, slots behind a row's end
    hold NaN scales and so do unused blocks."""
    rng = np.random.default_rng(seed + 77)
    nbs = [-(-n // 16) for n in lens]
    nb = sum(nbs) + spare
    pool = pool_of(nb, hkv, D, seed)
    perm = rng.permutation(nb)
    width = max(nbs + [1]) + 1
    table = np.full((len(lens), width), -1, np.int64)
    at = 0
    for b, n in enumerate(nbs):
        table[b, :n] = perm[at:at + n]
        at += n
    if poison:
        k, v = pool.k.cpu().numpy(), pool.v.cpu().numpy()
        for p, is_v in ((k, False), (v, True)):
            p[perm[at:], ..., 1024:] = 127
            for b, n in enumerate(lens):
                for tok in range(n % 16, 16) if n % 16 else ():
                    for grp in range(8):
                        p[table[b, n // 16], ..., oracle.kv4_place(tok, grp * 16, is_v)[2]] = 127
        pool.k.copy_(torch.from_numpy(k))
        pool.v.copy_(torch.from_numpy(v))
    q = (torch.randn((len(lens), hq, D), generator=torch.Generator().manual_seed(seed)) * qmag)
    return dict(pool=pool, table=table, lens=list(lens), q=q.to(torch.bfloat16).to(DEV),
                scale=scale if scale is not None else 1 / math.sqrt(D), window=window,
                softcap=softcap)


def workspace(c, max_len=None):
    B, hq, D = c["q"].shape
    n = binding.paged_kv4_decode_attn_ws_bytes(B, hq, c["pool"].num_kv_heads, D,
                                               max_len or max(c["lens"] + [1]), c["window"])
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=DEV)


def decode(c, ws=None, err=None, out=None, stream=None, table=None, max_len=None):
    if out is None:
        out = torch.full_like(c["q"], float("nan"))
    binding.paged_kv4_decode_attn_ws(c["q"], out, c["pool"],
                                     i32(c["table"]) if table is None else table, i32(c["lens"]),
                                     max_len or max(c["lens"] + [1]),
                                     workspace(c) if ws is None else ws, scale=c["scale"],
                                     softcap=c["softcap"], window=c["window"], err=err,
                                     stream=stream)
    return out


def check(c, out):
    """Against fp64 attention over the values the pool holds.  An output is
    rounded to bf16 (half a step: 2^-8 of it); the weights are rounded to f16
    (2^-11) and carry the logits' error, of numerator and sum: at most
    (D + 8) 2^-23 of the sum of |scale q_c k_c| for the fp32 sums (and their
    order), 2^-20 for the exponential and 2^-20 * cap * log2 e for the tanh.
    Weights below f16's normal range are rounded to multiples of 2^-24, an
    error of at most 2^-25 each, where the largest weight is at least 2^8: at
    most 2^-33 of every key's |v| (a peaked softmax leaves outputs that small)."""
    kp = oracle.kv4_decode(c["pool"].k.cpu().numpy(), KS, False)
    vp = oracle.kv4_decode(c["pool"].v.cpu().numpy(), VS, True)
    q, D = f64(c["q"]), c["q"].shape[2]
    args = (c["table"], c["lens"], c["scale"], c["softcap"], c["window"])
    ref, _ = oracle.paged_decode(q, kp, vp, *args)
    mag, _ = oracle.paged_decode(q, kp, np.abs(vp), *args)
    s, small = 0.0, np.zeros(mag.shape)
    hkv, G = kp.shape[1], q.shape[1] // kp.shape[1]
    for b, n in enumerate(c["lens"]):
        lo = max(0, n - c["window"]) if c["window"] > 0 else 0
        if n:
            key = oracle.gather_request_kv(kp, c["table"][b], n, 16)[lo:]
            a = np.einsum("hgd,thd->hgt", np.abs(q[b]).reshape(hkv, G, D), np.abs(key))
            s = max(s, abs(c["scale"]) * a.max())
            v = oracle.gather_request_kv(vp, c["table"][b], n, 16)[lo:]
            small[b] = 2.0 ** -33 * np.abs(v).sum(0).repeat(G, 0)
    delta = (D + 8) * 2.0 ** -23 * s + 2.0 ** -20 * (1 + 1.5 * max(0.0, c["softcap"]))
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * delta) * mag + small
    worst = float((np.abs(f64(out) - ref) - tol).max())
    assert worst <= 0, (worst, delta)                  # NaN fails too


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_decode_head_groups(D, G):
    hkv = 1 if G > 4 else 3
    c = make([1, 16, 17, 300, 0, 47], G * hkv, hkv, D, seed=G)
    err = i32([0])
    out = decode(c, err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    check(c, out)
    assert not out[4].any()                            # no key: zeros


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("lens", [[1], [2], [15], [31, 33], [4096], [5000, 1, 0, 900, 2500]])
def test_decode_lengths(D, lens):
    c = make(lens, 8, 2, D, seed=len(lens))
    check(c, decode(c))


@pytest.mark.parametrize("D,window,softcap", [(128, 1, 0.0), (128, 16, 30.0), (256, 17, 0.0),
                                              (256, 100, 50.0), (128, 700, 0.0), (256, 1, 5.0),
                                              (128, 0, 2.0), (256, 10 ** 6, 0.0)])
def test_decode_windows_and_caps(D, window, softcap):
    c = make([1, 15, 16, 17, 99, 100, 101, 700, 801, 0], 8, 2, D, seed=window, window=window,
             softcap=softcap, qmag=3.0)
    if window > 0:                                     # blocks no key is seen of may be gone
        for b, n in enumerate(c["lens"]):
            gone = max(0, n - window) // 16
            c["pool"].k[torch.tensor(c["table"][b, :gone])] = 255
            c["pool"].v[torch.tensor(c["table"][b, :gone])] = 255
    table = i32(c["table"])
    for b, n in enumerate(c["lens"]):
        if window > 0:
            table[b, :max(0, n - window) // 16] = -1
    err = i32([0])
    out = decode(c, err=err, table=table)
    torch.cuda.synchronize()
    assert err.item() == 0
    check(c, out)


def test_decode_many_short_requests():
    """More requests than lengths kept in shared memory, more segments than CTAs."""
    g = np.random.default_rng(0)
    c = make(g.integers(0, 70, 331).tolist(), 4, 2, 128, seed=5)
    check(c, decode(c))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("B,hkv,lo,hi", [
    (152, 1, 0, 900),      # as many segments as SMs
    (153, 1, 0, 1500),     # one more: two CTAs to an SM
    (60, 5, 700, 1400),    # 300 segments, some cut
    (77, 4, 0, 1300),      # 308: four to an SM
    (150, 8, 0, 700),      # 1200: more than run at once
    (760, 1, 0, 1000),     # more requests than a plan holds
    (40, 8, 1, 150)])      # short ones, whole
def test_decode_batches_of_many_segments(D, B, hkv, lo, hi):
    g = np.random.default_rng(B + hkv)
    lens = g.integers(lo, hi, B)
    lens[g.integers(0, B)] = 5 * hi                    # one long request among them
    c = make(lens.tolist(), hkv, hkv, D, seed=B, pool_of=byte_pool, poison=False)
    err = i32([0])
    out = decode(c, err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    check(c, out)
    assert torch.equal(decode(c), out)


@pytest.mark.parametrize("scale,qmag", [(0.0, 1.0), (-0.1, 1.0), (1.0, 4.0), (1e-3, 1e4),
                                        (3e4, 1e-6)])
def test_decode_scales_and_query_ranges(scale, qmag):
    c = make([40, 1000], 8, 2, 128, seed=8, scale=scale, qmag=qmag)
    check(c, decode(c))


def test_decode_rising_logits():
    """Each key's logit is above the last one's by several powers of two, so the
    running reference moves at every tile; and falling ones never move it."""
    for sign in (1.0, -1.0):
        L, D = 600, 128
        k = torch.zeros((L, 1, D), dtype=torch.bfloat16, device=DEV)
        k[:, 0, 0] = torch.arange(1, L + 1, device=DEV) * (12.0 / L)
        v = rows((L, 1, D), 3)
        c = make([L], 4, 1, D, poison=False)
        flat = i32(c["table"][0, :-1])
        slots = (flat[:, None] * 16 + torch.arange(16, device=DEV)).flatten()[:L].to(torch.int32)
        binding.paged_kv4_append(k, v, c["pool"], slots)
        c["q"].zero_()
        c["q"][:, :, 0] = sign * 64.0
        c["scale"] = 1.0
        torch.cuda.synchronize()
        check(c, decode(c))


def test_decode_visible_nan_reaches_its_head_only():
    c = make([100, 90], 8, 2, 128, seed=2)
    blk = int(c["table"][0, 3])
    c["pool"].k[blk, 1, 0, oracle.kv4_place(5, 0, False)[2]] = 127
    out = decode(c)
    assert torch.isnan(out[0, 4:]).all() and torch.isfinite(out[0, :4]).all()
    assert torch.isfinite(out[1]).all()
    long = make([9000], 8, 2, 128, seed=2)             # split: through the merge
    long["pool"].v[int(long["table"][0, 300]), 0, 0, oracle.kv4_place(5, 32, True)[2]] = 127
    out = decode(long)
    nan = torch.isnan(out[0, :4])
    assert nan[:, 32:48].all() and not nan[:, :32].any() and not nan[:, 48:].any()
    assert torch.isfinite(out[0, 4:]).all()
    long["pool"].k[:, 0, 0, 1024:] = 127               # every key of one head
    assert torch.isnan(decode(long)[0, :4]).all()


def test_decode_bad_tables_and_lengths_are_reported():
    c = make([64, 64, 64], 8, 2, 128, seed=4, poison=False)
    t = i32(c["table"])
    t[1, 2] = c["pool"].num_blocks                     # past the pool: reads as zeros
    t[2, 1] = -1
    err = i32([0])
    out = decode(c, err=err, table=t)
    torch.cuda.synchronize()
    assert err.item() == binding.DEVERR_BAD_TABLE
    assert torch.isfinite(out).all()
    c1 = dict(c, q=c["q"][:1], table=c["table"][:1], lens=[64])
    check(c1, out[:1])
    err.zero_()
    lens = i32([64, 10 ** 6, -3])                      # past the row, negative
    o2 = torch.full_like(out, float("nan"))
    binding.paged_kv4_decode_attn_ws(c["q"], o2, c["pool"], i32(np.maximum(c["table"], 0)), lens,
                                     64, workspace(c), scale=c["scale"], err=err)
    torch.cuda.synchronize()
    assert err.item() & binding.DEVERR_SEQ_LEN
    assert torch.equal(o2[0], out[0]) and not o2[2].any()


def test_decode_same_bits_every_time_and_wherever():
    """The same call gives the same bits, in a fresh workspace or one used by a
    call of other sizes before (counters are left zero), with permuted pages, on
    another stream and from a replayed graph."""
    c = make([5000, 64, 1200, 0, 2000], 8, 2, 256, seed=6)
    first = decode(c)
    ws = workspace(c)
    for _ in range(3):
        assert torch.equal(decode(c, ws=ws), first)
    assert not ws[:2048].any()                         # the counters
    perm = torch.randperm(c["pool"].num_blocks, generator=torch.Generator().manual_seed(0))
    inv = torch.argsort(perm)
    moved = binding.Kv4Pool(c["pool"].k[perm.to(DEV)].contiguous(),
                            c["pool"].v[perm.to(DEV)].contiguous(), KS, VS)
    t2 = np.where(c["table"] >= 0, inv.numpy()[np.maximum(c["table"], 0)], -1)
    assert torch.equal(decode(dict(c, pool=moved, table=t2)), first)
    side = torch.cuda.Stream()
    out, table, lens = torch.full_like(first, 3.0), i32(c["table"]), i32(c["lens"])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        decode(c, ws=ws, out=out, table=table)
    side.synchronize()
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    out.fill_(3.0)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        binding.paged_kv4_decode_attn_ws(c["q"], out, c["pool"], table, lens, 5000, ws,
                                         scale=c["scale"], softcap=c["softcap"],
                                         window=c["window"])
    for _ in range(2):
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


def test_one_workspace_for_calls_of_all_sizes():
    """Batches of other sizes and head dimensions in turn on one workspace: each
    gives the bits that it gives on a workspace of its own."""
    g = np.random.default_rng(4)
    cases = [make(g.integers(0, most, b).tolist(), 8, 2, d, seed=b, spare=2, pool_of=byte_pool)
             for b, d, most in ((2, 256, 5000), (70, 128, 400), (3, 128, 2500), (100, 256, 200),
                                (9, 256, 1500))]
    want = [decode(c) for c in cases]
    ws = torch.zeros(max(workspace(c).numel() for c in cases), dtype=torch.uint8, device=DEV)
    for i in (0, 1, 2, 3, 4, 3, 0, 1, 4, 2):
        assert torch.equal(decode(cases[i], ws=ws), want[i]), i
    for i in (1, 3):
        check(cases[i], want[i])


def test_rows_longer_than_max_seq_len():
    """max_seq_len only sizes the pieces: longer rows are right all the same."""
    for lens, promise in (([5000, 30], 64), ([12000, 30], 2000), ([900] * 90, 64),
                          ([9000] * 2 + [100] * 100, 1500)):
        c = make(lens, 8, 2, 128, seed=1, pool_of=byte_pool, poison=False)
        err = i32([0])
        out = decode(c, err=err, max_len=promise, ws=workspace(c, promise))
        torch.cuda.synchronize()
        assert err.item() == 0
        check(c, out)


def test_offsets_past_32_bits():
    """A pool of more than 4 GiB per tensor: its last blocks are written, read
    and expanded where they are."""
    D, hkv, nb = 256, 8, (1 << 32) // (8 * 2304) + 40
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB of free device memory")
    pool = binding.Kv4Pool(*(torch.zeros((nb, hkv, 2, 1152), dtype=torch.uint8, device=DEV)
                             for _ in range(2)), KS, VS)
    L = 40
    k, v = rows((L, hkv, D), 1), rows((L, hkv, D), 2)
    blocks = [nb - 1, nb - 30, nb - 2]
    slots = i32([blocks[t // 16] * 16 + t % 16 for t in range(L)])
    binding.paged_kv4_append(k, v, pool, slots)
    small = binding.Kv4Pool(*(torch.stack([p[b] for b in blocks]) for p in (pool.k, pool.v)), KS,
                            VS)
    assert small.k.any() and not pool.k[:nb - 40].view(torch.int64).any()
    c = dict(pool=small, table=np.array([[0, 1, 2]]), lens=[L], window=0, softcap=0.0,
             scale=1 / 16, q=rows((1, 16, D), 3))
    want = decode(c)
    check(c, want)
    assert torch.equal(decode(dict(c, pool=pool, table=np.array([blocks]))), want)
    k16 = torch.zeros((3, hkv, 16, D), dtype=torch.bfloat16, device=DEV)
    v16, k16b, v16b = (torch.zeros_like(k16) for _ in range(3))
    binding.paged_kv4_expand(pool, k16, v16, i32(blocks))
    binding.paged_kv4_expand(small, k16b, v16b, i32([0, 1, 2]))
    assert torch.equal(k16, k16b) and torch.equal(v16, v16b) and k16.any()


# ---------------------------------------------------------------- together
def test_a_stream_of_steps_sees_its_own_writes():
    """Decode steps in a row without a wait, each with lengths, slots, rows and
    queries that the kernels right before it wrote: the same bits as step by
    step with a wait between the kernels, eagerly and in a replayed graph."""
    D, hkv, Hq, B, steps = 128, 2, 8, 3, 24
    ks, vs = (torch.stack([rows((B, hkv, D), 100 * i + j) for i in range(steps)])
              for j in (1, 2))
    qs = torch.stack([rows((B, Hq, D), 100 * i + 3) for i in range(steps)])
    table = i32(np.arange(B * 4).reshape(B, 4))
    pool = binding.Kv4Pool.zeros(B * 4, hkv, D, KS, VS, device=DEV)
    start, first = i32([5, 0, 14]), table[:, 0] * 16
    lens, slots, at = start.clone(), start + first, torch.zeros(1, dtype=torch.int64, device=DEV)
    k, v, q = torch.zeros_like(ks[0]), torch.zeros_like(ks[0]), torch.zeros_like(qs[0])
    out = torch.zeros((steps, B, Hq, D), dtype=torch.bfloat16, device=DEV)
    nbytes = binding.paged_kv4_decode_attn_ws_bytes(B, Hq, hkv, D, 64)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device=DEV)

    def reset():
        pool.k.zero_()
        pool.v.zero_()
        lens.copy_(start)
        slots.copy_(start + first)
        at.zero_()
        out.zero_()
        torch.cuda.synchronize()

    def run(wait):
        for i in range(steps):
            for src, dst in ((ks, k), (vs, v), (qs, q)):
                torch.index_select(src, 0, at, out=dst.unsqueeze(0))
                wait()
            binding.paged_kv4_append(k, v, pool, slots)
            wait()
            lens.add_(1)
            wait()
            binding.paged_kv4_decode_attn_ws(q, out[i], pool, table, lens, 64, ws, scale=0.1)
            wait()
            slots.add_(1)
            at.add_(1)
            wait()

    reset()
    run(torch.cuda.synchronize)
    want = out.clone()
    assert torch.isfinite(want).all() and want[-1].any()
    reset()
    run(lambda: None)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(lambda: None)
    for _ in range(2):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_prompt_decode_fork_and_compact_together():
    """A prompt written to a 4-bit cache and attended by the prefill kernel over
    its expanded blocks, decoded, forked with its last block copied, the parent
    freed and the pool closed up: the child's decode keeps its bits."""
    D, hkv, hq, L = 128, 2, 8, 150
    nb = 64
    pool = binding.Kv4Pool.zeros(nb, hkv, D, KS, VS)
    used = -(-L // 16)
    parent = [50 - 3 * i for i in range(used)]
    table = i32([parent])
    pos = torch.arange(L, device=DEV)
    slots = (table[0].long()[pos // 16] * 16 + pos % 16).to(torch.int32)
    k, v = rows((L, hkv, D), 4), rows((L, hkv, D), 5)
    binding.paged_kv4_append(k, v, pool, slots)
    # prefill of the last 20 tokens over the expanded blocks
    k16 = torch.zeros((used, hkv, 16, D), dtype=torch.bfloat16, device=DEV)
    v16 = torch.zeros_like(k16)
    binding.paged_kv4_expand(pool, k16, v16, table)
    q = rows((20, hq, D), 6, 0.0)
    out = torch.empty_like(q)
    order = torch.arange(used, dtype=torch.int32, device=DEV)[None]
    binding.paged_prefill_attn(q, out, k16, v16, order, i32([0, 20]), i32([L]), 20, L, scale=0.1)
    ref, _ = oracle.paged_attention(f64(q), f64(k16), f64(v16), np.arange(used)[None], [L], [0, 20],
                                    0.1)
    assert np.abs(f64(out) - ref).max() <= 2e-2
    # the last of them again as a decode row, over the 4-bit cache itself
    c = dict(pool=pool, table=np.array([parent]), lens=[L], q=q[-1:].contiguous(), scale=0.1,
             window=0, softcap=0.0)
    want = decode(c)
    check(c, want)
    # fork: the child shares the full blocks and owns a copy of the last one
    refs = torch.zeros(nb, dtype=torch.int32, device=DEV)
    lens = i32([L])
    binding.paged_kv_ref_blocks(table, lens, refs, 1)
    child = table.clone()
    child[0, -1] = 63
    binding.paged_kv_ref_blocks(child, lens, refs, 1)
    binding.paged_kv_copy_blocks([pool.k, pool.v], table[0, -1:], child[0, -1:])
    assert torch.equal(decode(dict(c, table=child.cpu().numpy())), want)
    # the parent ends, the pool is closed up
    binding.paged_kv_ref_blocks(table, lens, refs, -1)
    remap, moves = torch.empty_like(refs), torch.empty(nb + 2, dtype=torch.int32, device=DEV)
    binding.paged_kv_compact([pool.k, pool.v], refs, child, lens, refs, child, remap, moves)
    torch.cuda.synchronize()
    assert int(child.max()) == used - 1 and refs[:used].eq(1).all() and not refs[used:].any()
    pool.k[used:] = 255
    pool.v[used:] = 255
    assert torch.equal(decode(dict(c, table=child.cpu().numpy())), want)


def test_binding_refusals_on_device_tensors():
    c = make([64], 8, 2, 128)
    x = rows((4, 2, 128), 1)
    with pytest.raises(ValueError):
        binding.paged_kv4_append(x, x[:3], c["pool"], i32([0, 1, 2, 3]))
    with pytest.raises(ValueError):
        binding.paged_kv4_append(x, x.float(), c["pool"], i32([0, 1, 2, 3]))
    with pytest.raises(ValueError):                    # rows of a token not contiguous
        binding.paged_kv4_append(x.transpose(0, 1).contiguous().transpose(0, 1), x, c["pool"],
                                 i32([0, 1, 2, 3]))
    with pytest.raises(ValueError):
        binding.paged_kv4_append(x, x, c["pool"], i32([0, 1, 2, 3]).long())
    with pytest.raises(ValueError):
        decode(c, out=torch.empty((1, 4, 128), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(binding.PagedAttnError):
        decode(c, ws=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(binding.PagedAttnError):        # the scale of the pool
        decode(dict(c, pool=binding.Kv4Pool(c["pool"].k, c["pool"].v, 0.0, 1.0)))
