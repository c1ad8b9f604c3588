"""GPU checks of NaN in keys and queries: it reaches every query head that sees
it and no other row, with a logit cap and without, over 4-bit and bf16 pools."""
import math

import pytest
import torch

import oracle
from paged_kv_attention_12_gb300 import _build, binding, workload
from tests.parity import assert_close, to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    binding.lib()


def kv4_case(D, lens, softcap, seed=0):
    """A call over random codes with scales from 0.25 to 4, pages in random order."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    nbs = [-(-n // 16) for n in lens]
    shape = (sum(nbs) + 3, 2, D // 128, 1152)
    k, v = (torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
            for _ in range(2))
    for p in (k, v):
        p[..., 1024:] = p[..., 1024:] % 33 + 0x28
    perm = torch.randperm(shape[0], generator=torch.Generator().manual_seed(seed))
    table = torch.full((len(lens), max(nbs) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(nbs):
        table[b, :n] = perm[at:at + n]
        at += n
    q = torch.randn((len(lens), 8, D), generator=g, device=DEV).to(torch.bfloat16)
    return dict(pool=binding.Kv4Pool(k, v, 0.2, 0.1), table=table.to(DEV), q=q, softcap=softcap,
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV), most=max(lens))


def kv4_run(c):
    B, hq, D = c["q"].shape
    n = binding.paged_kv4_decode_attn_ws_bytes(B, hq, 2, D, c["most"])
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    out = torch.full_like(c["q"], 7.0)
    binding.paged_kv4_decode_attn_ws(c["q"], out, c["pool"], c["table"], c["lens"], c["most"], ws,
                                     scale=1 / math.sqrt(D), softcap=c["softcap"])
    return out


@pytest.mark.parametrize("softcap", [0.0, 2.0, 50.0])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("lens,t", [([90, 70], 53), ([9000, 70], 4805), ([9000, 70], 8999)])
def test_kv4_decode(D, lens, t, softcap):
    """A visible key whose group holds a NaN scale, in whole and cut segments;
    then a query with a NaN element."""
    c = kv4_case(D, lens, softcap)
    clean = kv4_run(c)
    assert torch.isfinite(clean).all()
    unit = c["pool"].k[int(c["table"][0, t // 16]), 1, D // 128 - 1]
    at = oracle.kv4_place(t % 16, 32, False)[2]
    held = int(unit[at])
    unit[at] = 127
    out = kv4_run(c)
    assert torch.isnan(out[0, 4:]).all()
    assert torch.equal(out[0, :4], clean[0, :4]) and torch.equal(out[1], clean[1])
    unit[at] = held
    c["q"][0, 2, D - 3] = NAN
    out = kv4_run(c)
    assert torch.isnan(out[0, 2]).all()
    out[0, 2] = clean[0, 2]
    assert torch.equal(out, clean)


# ------------------------------------------------ over bf16 pools
def bf16_batch(D, L, n, softcap, seed=5):
    return workload.make_batch(seq_lens=L, q_lens=n, num_q_heads=8, num_kv_heads=2, head_dim=D,
                               num_blocks=sum(-(-x // 16) for x in L) + 8, device=DEV, poison=True,
                               cfg_id=41, seed=seed, softcap=softcap)


def follow_nan(b, t, paths):
    """Every path of the batch with key t of its first request's KV head 1 NaN,
    then with its last query's head 2: exactly what sees them is NaN, the rest
    is what it was."""
    L, n = b.seq_lens_host[0], b.q_lens_host[0]
    clean = dict(paths(b))
    for name, x in clean.items():
        assert torch.isfinite(x).all(), name

    def compare(mask, what):
        for name, out in paths(b):
            assert torch.equal(torch.isnan(out), mask[..., None].expand_as(out)), (what, name)
            assert_close(to_f64(out[~mask]), to_f64(clean[name][~mask]), f"{what} {name}")
    row = b.k_pool[int(b.block_tables[0, t // 16]), 1, t % 16]
    held = row[-7].clone()
    row[-7] = NAN
    mask = torch.zeros(b.q.shape[:2], dtype=torch.bool, device=DEV)
    mask[:n, 4:] = (torch.arange(L - n, L, device=DEV) >= t)[:, None]
    compare(mask, "key")
    row[-7] = held
    b.q[n - 1, 2, 5] = NAN
    mask.zero_()
    mask[n - 1, 2] = True
    compare(mask, "query")


def one_piece_paths(b):
    out = torch.full_like(b.q, 7.0)
    if max(b.q_lens_host) == 1:
        binding.paged_decode_attn(b.q, out, b.k_pool, b.v_pool, b.block_tables, b.seq_lens,
                                  b.max_seq_len, scale=b.scale, softcap=b.softcap)
        yield "decode", out.clone()
    else:
        yield "mixed", binding.MixedBatch(b).run().clone()
    yield "prefill", binding.run_batch(b, out).clone()


@pytest.mark.parametrize("softcap", [0.0, 2.0, 8.0, 50.0])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("L,n,t", [
    ([90, 70], [1, 1], 53), ([5000, 70], [1, 1], 2601),     # decode
    ([200, 333], [120, 50], 150),      # chunks, some of whose rows see the key
    ([9000, 40], [64, 1], 4000)])      # a long prefix, cut along its keys
def test_bf16_pools(D, L, n, t, softcap):
    follow_nan(bf16_batch(D, L, n, softcap), t, one_piece_paths)


def cut_paths(b):
    """Decode in pieces whose partial results are merged."""
    out = torch.full_like(b.q, 7.0)
    binding.paged_decode_attn_noalloc(b.q, out, b.k_pool, b.v_pool, b.block_tables, b.seq_lens,
                                      b.max_seq_len, scale=b.scale, softcap=b.softcap)
    yield "noalloc", out
    split = binding.DecodeSplitK(b)
    lse = torch.zeros(b.q.shape[:2], dtype=torch.float32, device=DEV)
    yield "split-K", split.run(lse_out=lse)
    yield "split-K LSE", lse[..., None]
    yield "fused", binding.DecodeFused(b).run()
    yield "mixed", binding.MixedBatch(b).run()


@pytest.mark.parametrize("softcap", [0.0, 50.0])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("L,t", [([90, 70], 53), ([5000, 70], 2601), ([5000, 70], 4999)])
def test_bf16_pools_in_pieces(D, L, t, softcap):
    """The merge drops no piece that is NaN, nor a row all of whose pieces are."""
    follow_nan(bf16_batch(D, L, [1, 1], softcap), t, cut_paths)


@pytest.mark.parametrize("softcap", [0.0, 50.0])
def test_expanded_blocks(softcap):
    """A 4-bit group that held an infinity, read by a chunk over its expanded
    blocks and by decode over the 4-bit blocks themselves."""
    D, L = 128, 100
    c = kv4_case(D, [L], softcap)
    table = c["table"][0, :7].contiguous()
    k = torch.randn((1, 2, D), device=DEV).to(torch.bfloat16)
    k[0, 0, 40] = math.inf
    slot = (table[3:4] * 16 + 2).to(torch.int32)       # key 50
    binding.paged_kv4_append(k, k[:, [1, 1]].contiguous(), c["pool"], slot)
    dec = kv4_run(c)
    assert torch.isnan(dec[0, :4]).all() and torch.isfinite(dec[0, 4:]).all()
    k16 = torch.zeros((7, 2, 16, D), dtype=torch.bfloat16, device=DEV)
    v16 = torch.zeros_like(k16)
    binding.paged_kv4_expand(c["pool"], k16, v16, table)
    q = torch.randn((80, 8, D), device=DEV).to(torch.bfloat16)
    out = torch.full_like(q, 7.0)
    i32 = dict(dtype=torch.int32, device=DEV)
    binding.paged_prefill_attn(q, out, k16, v16, torch.arange(7, **i32)[None],
                               torch.tensor([0, 80], **i32), c["lens"], 80, L,
                               scale=1 / math.sqrt(D), softcap=softcap)
    want = torch.zeros((80, 8), dtype=torch.bool, device=DEV)
    want[30:, :4] = True                               # queries at positions 20 .. 99
    assert torch.equal(torch.isnan(out), want[..., None].expand_as(out))
