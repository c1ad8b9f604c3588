"""GPU checks of 4-bit decode at the ends of its parameters' ranges, and of the ids
and lengths that it and the expansion correct."""
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


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def make(lens, D, *, seed=0, ks=0.004, vs=0.002, qmag=1.0, scale=None, softcap=0.0, spare=3):
    """A call of 8 query and 2 KV heads over random codes with e4m3 scales from
    0.25 to 4."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    nbs = [-(-n // 16) for n in lens]
    shape = (sum(nbs) + spare, 2, D // 128, 1152)
    pools = []
    for _ in range(2):
        p = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
        p[..., 1024:] = p[..., 1024:] % 33 + 0x28
        pools.append(p)
    perm = np.random.default_rng(seed).permutation(shape[0])
    table, at = np.full((len(lens), max(nbs) + 1), -1), 0
    for b, n in enumerate(nbs):
        table[b, :n] = perm[at:at + n]
        at += n
    q = torch.randn((len(lens), 8, D), generator=torch.Generator().manual_seed(seed)) * qmag
    return dict(pool=binding.Kv4Pool(*pools, ks, vs), table=table, lens=list(lens),
                q=q.to(torch.bfloat16).to(DEV), scale=scale or 1 / math.sqrt(D), softcap=softcap)


def run(c, lens=None, err=None):
    B, hq, D = c["q"].shape
    most = max(c["lens"])
    n = binding.paged_kv4_decode_attn_ws_bytes(B, hq, 2, D, most)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    out = torch.full_like(c["q"], float("nan"))
    binding.paged_kv4_decode_attn_ws(c["q"], out, c["pool"], i32(c["table"]),
                                     i32(c["lens"] if lens is None else lens), most, ws,
                                     scale=c["scale"], softcap=c["softcap"], err=err)
    torch.cuda.synchronize()
    return out


def check(c, out):
    """Against fp64 attention over the values the pool holds.  The capped logit
    moves by less than the logit does (tanh's slope is at most 1), and its own
    rounding is relative to it, whatever the cap: at most 2^-18 of the largest
    one (the exp2 form is taken from tanh = 0.24 on, with an absolute error of
    tanh below 5e-7).  The logits' fp32 sums: (D + 8) 2^-23 of the sum of
    |scale q_c k_c|; the exponential 2^-20.  Weights are rounded to f16 (2^-11,
    below 2^-14 of the largest 2^-33 of it), outputs to bf16 (half a step: 2^-8,
    below 2^-126 2^-134)."""
    p = c["pool"]
    kp = oracle.kv4_decode(p.k.cpu().numpy(), p.k_scale, False)
    vp = oracle.kv4_decode(p.v.cpu().numpy(), p.v_scale, True)
    q, D = f64(c["q"]), c["q"].shape[2]
    args = (c["table"], c["lens"], c["scale"], c["softcap"], 0)
    ref, _ = oracle.paged_decode(q, kp, vp, *args)
    mag, _ = oracle.paged_decode(q, kp, np.abs(vp), *args)
    s, top, small = 0.0, 0.0, np.zeros(mag.shape)
    for b, n in enumerate(c["lens"]):
        if n:
            key = oracle.gather_request_kv(kp, c["table"][b], n, 16)
            one = np.einsum("hgd,thd->hgt", q[b].reshape(2, 4, D), key) * c["scale"]
            a = np.einsum("hgd,thd->hgt", np.abs(q[b]).reshape(2, 4, D), np.abs(key))
            s, top = max(s, abs(c["scale"]) * a.max()), max(top, np.abs(one).max())
            v = oracle.gather_request_kv(vp, c["table"][b], n, 16)
            small[b] = 2.0 ** -33 * np.abs(v).sum(0).repeat(4, 0)
    if c["softcap"] > 0:
        top = c["softcap"] * np.tanh(top / c["softcap"])
    delta = (D + 8) * 2.0 ** -23 * s + 2.0 ** -20 + 2.0 ** -18 * top
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -134 + (2.0 ** -11 + 2 * delta) * mag + small
    worst = float(((np.abs(f64(out) - ref) - tol) / np.abs(mag).max()).max())
    assert worst <= 0, (worst, delta, top)             # NaN fails too


@pytest.mark.parametrize("softcap", [1e-40, 1e-3, 5.0, 50.0, 300.0, 1e4, 1e6, 1e20, 3e38])
@pytest.mark.parametrize("D,lens", [(128, [70, 1, 0, 300]), (256, [9000, 40])])
def test_caps_of_every_size(D, lens, softcap):
    """A cap far above the logits leaves them as they are, one far below makes
    them all alike; a query of zeros averages its values."""
    c = make(lens, D, seed=len(lens), qmag=4.0, ks=0.05, softcap=softcap)
    c["q"][0, 3] = 0.0
    check(c, run(c))


@pytest.mark.parametrize("ks,vs,qmag", [(0.004, 1.2e-38, 1.0), (0.004, 3e-34, 1.0),
                                        (0.004, 1e36, 1.0), (1e-36, 0.002, 1e34),
                                        (1e35, 0.002, 1e-36)])
@pytest.mark.parametrize("D,lens", [(128, [1100, 50]), (256, [9000])])
def test_pool_scales_of_every_size(D, lens, ks, vs, qmag):
    """Pool scales near both ends of fp32: the output is as accurate as ever."""
    c = make(lens, D, seed=3, ks=ks, vs=vs, qmag=qmag, scale=0.05)
    c["pool"].v[..., :1024] &= 0x77                    # no value below 0: means are large
    c["q"][0, 6] = 0.0                                 # every weight the same
    check(c, run(c))


@pytest.mark.parametrize("lens", [[40, 0, 7], [9000, 0, 7]])
def test_query_of_minus_infinity(lens):
    """Keys are visible but every logit is -infinity: the softmax is 0 / 0.  A
    row without keys stays 0."""
    c = make(lens, 128)
    c["pool"].k[..., :1024] = 0x22                     # every code 1
    c["q"].fill_(1.0)
    c["q"][:, 5, 0] = -math.inf
    out = run(c)
    assert torch.isnan(out[0, 5]).all() and torch.isnan(out[2, 5]).all() and not out[1].any()
    out[:, 5] = 0
    assert torch.isfinite(out).all()


def test_bad_ids_read_as_zeros_and_long_rows_end_with_their_table():
    c = make([64, 61, 64], 128, seed=4)
    t = c["table"].copy()
    nb = c["pool"].num_blocks
    t[1, 2], t[1, 3], t[2, 1] = nb, 2 ** 31 - 1, -1
    err = i32([0])
    out = run(dict(c, table=t), err=err)
    assert err.item() == binding.DEVERR_BAD_TABLE
    # the same call with a block of zeros where the bad ids were
    more = binding.Kv4Pool(*(torch.cat([p, torch.zeros_like(p[:1])]) for p in
                             (c["pool"].k, c["pool"].v)), c["pool"].k_scale, c["pool"].v_scale)
    z = c["table"].copy()
    z[1, 2] = z[1, 3] = z[2, 1] = nb
    same = dict(c, pool=more, table=z)
    err.zero_()
    assert torch.equal(run(same, err=err), out) and err.item() == 0
    check(same, out)
    # lengths behind the table's last entry, and negative ones
    full = np.maximum(c["table"], 0)
    width = 16 * full.shape[1]
    got = run(dict(c, table=full), lens=[10 ** 6, width, -3], err=err)
    assert err.item() == binding.DEVERR_SEQ_LEN
    ends = dict(c, table=full, lens=[width, width, 0])
    assert torch.equal(run(ends), got) and not got[2].any()
    check(ends, got)


def test_expand_leaves_what_bad_ids_name():
    c = make([48], 128, spare=0)
    k16 = torch.full((2, 2, 16, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    v16, err = k16.clone(), i32([0])
    binding.paged_kv4_expand(c["pool"], k16, v16, i32([3, 0, -1, 1]), i32([0, 2, 1, -5]), err)
    torch.cuda.synchronize()
    assert err.item() == binding.DEVERR_BAD_TABLE
    assert k16.eq(3.0).all() and v16.eq(3.0).all()


def test_wide_tables_of_many_heads():
    """512 segments over table rows of 2 million entries: the requests' blocks are
    counted, not each KV head's again."""
    lens = [5000] + [40 + i for i in range(63)]
    c = make(lens, 128, seed=1)
    p = c["pool"]
    pool = binding.Kv4Pool(*(t.repeat(1, 4, 1, 1) for t in (p.k, p.v)), p.k_scale, p.v_scale)
    q = c["q"].repeat(1, 4, 1)
    ws = torch.zeros(binding.paged_kv4_decode_attn_ws_bytes(64, 32, 8, 128, 5000),
                     dtype=torch.uint8, device=DEV)
    table = torch.full((64, (1 << 21) - 15), -1, dtype=torch.int32, device=DEV)
    narrow = i32(c["table"])
    table[:, :narrow.shape[1]] = narrow
    out = [torch.full_like(q, float("nan")) for _ in range(2)]
    for t, o in zip((table, narrow), out):
        binding.paged_kv4_decode_attn_ws(q, o, pool, t, i32(lens), 5000, ws, scale=c["scale"])
    torch.cuda.synchronize()
    assert torch.equal(*out) and torch.isfinite(out[0]).all()
