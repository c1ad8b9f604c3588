"""Host-side refusals of the draft trees and of the eviction: found before any
CUDA call, so these run without a GPU."""
import ctypes
import math

import pytest
import torch

from paged_kv_attention_12_gb300 import _build, binding


@pytest.fixture(scope="module")
def L():
    _build.build()
    return binding.lib()


def name(st):
    return binding.STATUS[st]


def plan(L, **kw):
    a = dict(parents=64, first=64, lens=64, total=None, tables=64, max_blocks=4, num_blocks=8, B=2,
             rows=10, most=8, masks=64, positions=64, slots=64, err=None, stream=None)
    a.update(kw)
    return name(L.paged_tree_plan(*a.values()))


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), "PKA_OK"), (dict(most=65), "PKA_ERR_UNSUPPORTED"), (dict(most=-1), "PKA_ERR_SHAPE"),
    (dict(B=-1), "PKA_ERR_SHAPE"), (dict(B=2 ** 31 - 1), "PKA_ERR_SHAPE"),
    (dict(rows=-1), "PKA_ERR_SHAPE"), (dict(max_blocks=0), "PKA_ERR_SHAPE"),
    (dict(max_blocks=2 ** 27), "PKA_ERR_SHAPE"), (dict(num_blocks=0), "PKA_ERR_SHAPE"),
    (dict(num_blocks=2 ** 27), "PKA_ERR_SHAPE"), (dict(parents=None), "PKA_ERR_NULL"),
    (dict(first=None), "PKA_ERR_NULL"), (dict(lens=None), "PKA_ERR_NULL"),
    (dict(tables=None), "PKA_ERR_NULL"), (dict(masks=68), "PKA_ERR_ALIGN")])
def test_plan_refusals(L, kw, want):
    assert plan(L, **kw) == want


def attn(L, pool=None, scale=0.1, softcap=0.0, window=0, **kw):
    p = dict(k=64, v=64, num_blocks=8, hkv=2, bs=16, d=128)
    p.update(pool or {})
    kv = binding.PkaKvPool(*p.values())
    par = binding.PkaAttnParams(scale, softcap, window, None)
    a = dict(q=64, out=64, kv=ctypes.byref(kv), tables=64, max_blocks=4, first=64, masks=64,
             lens=64, B=2, hq=8, rows=10, most=8, max_len=64, par=ctypes.byref(par), ws=64,
             ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return name(L.paged_tree_attn_ws(*a.values()))


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), "PKA_OK"), (dict(B=0), "PKA_OK"), (dict(most=0), "PKA_OK"),
    (dict(most=65), "PKA_ERR_UNSUPPORTED"), (dict(hq=7), "PKA_ERR_SHAPE"),
    (dict(hq=6), "PKA_ERR_UNSUPPORTED"), (dict(hq=32), "PKA_ERR_UNSUPPORTED"),
    (dict(hq=0), "PKA_ERR_SHAPE"), (dict(B=-1), "PKA_ERR_SHAPE"), (dict(rows=-1), "PKA_ERR_SHAPE"),
    (dict(max_len=65), "PKA_ERR_SHAPE"), (dict(max_len=-1), "PKA_ERR_SHAPE"),
    (dict(max_blocks=0), "PKA_ERR_SHAPE"), (dict(scale=math.nan), "PKA_ERR_SHAPE"),
    (dict(scale=math.inf), "PKA_ERR_SHAPE"), (dict(softcap=math.nan), "PKA_ERR_SHAPE"),
    (dict(pool=dict(d=64)), "PKA_ERR_UNSUPPORTED"), (dict(pool=dict(bs=32)), "PKA_ERR_UNSUPPORTED"),
    (dict(pool=dict(num_blocks=0)), "PKA_ERR_SHAPE"), (dict(pool=dict(num_blocks=2 ** 26)), "PKA_ERR_SHAPE"),
    (dict(pool=dict(k=None)), "PKA_ERR_NULL"), (dict(pool=dict(v=72)), "PKA_ERR_ALIGN"),
    (dict(q=None), "PKA_ERR_NULL"), (dict(q=72), "PKA_ERR_ALIGN"), (dict(out=None), "PKA_ERR_NULL"),
    (dict(out=72), "PKA_ERR_ALIGN"), (dict(masks=None), "PKA_ERR_NULL"), (dict(masks=68), "PKA_ERR_ALIGN"),
    (dict(first=None), "PKA_ERR_NULL"), (dict(lens=None), "PKA_ERR_NULL"),
    (dict(tables=None), "PKA_ERR_NULL"), (dict(ws=None), "PKA_ERR_NULL"), (dict(ws=72), "PKA_ERR_ALIGN"),
    (dict(ws_bytes=1000), "PKA_ERR_WORKSPACE"), (dict(kv=None), "PKA_ERR_NULL"),
    (dict(par=None), "PKA_ERR_NULL"), (dict(B=2 ** 20, max_blocks=2 ** 12), "PKA_ERR_SHAPE"),
    # 2^30 requests x 2^26 heads x 4 tiles x (44 + 20): 2^64
    (dict(pool=dict(num_blocks=1, hkv=2 ** 26), hq=2 ** 29, B=2 ** 30, most=64, max_blocks=44),
     "PKA_ERR_SHAPE"),
    (dict(B=1, pool=dict(hkv=1), hq=1, max_blocks=2 ** 26 + 1), "PKA_ERR_SHAPE"),
    (dict(B=1, window=5, max_blocks=2 ** 26 + 1), "PKA_ERR_SHAPE")])
def test_attention_refusals(L, kw, want):
    assert attn(L, **kw) == want


def test_attention_workspace(L):
    n = binding.paged_tree_attn_ws_bytes(8, 2, 256, 64)
    assert 0 < n <= 320 * 128 * 257 * 4 + 65536
    assert binding.paged_tree_attn_ws_bytes(8, 2, 256, 16) < n
    assert binding.paged_tree_attn_ws_bytes(8, 3, 256, 16) == 0
    assert binding.paged_tree_attn_ws_bytes(8, 2, 256, 65) == 0


def accept(L, num_pools=2, pool=64, **kw):
    ptrs = (ctypes.c_void_p * max(1, num_pools))(*[pool] * max(0, num_pools))
    a = dict(pools=ptrs, num_pools=num_pools, num_blocks=8, hkv=2, bs=16, d=128, parents=64,
             tokens=64, targets=64, slots=64, first=64, lens=64, B=2, rows=10, most=8, path=64,
             accepted=64, next_tokens=64, new_lens=64, err=None, stream=None)
    a.update(kw)
    return name(L.paged_tree_accept(*a.values()))


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), "PKA_OK"), (dict(most=65), "PKA_ERR_UNSUPPORTED"), (dict(num_pools=-1), "PKA_ERR_SHAPE"),
    (dict(pools=None), "PKA_ERR_NULL"), (dict(pool=None), "PKA_ERR_NULL"), (dict(pool=72), "PKA_ERR_ALIGN"),
    (dict(hkv=1025), "PKA_ERR_SHAPE"), (dict(d=64), "PKA_ERR_UNSUPPORTED"), (dict(bs=8), "PKA_ERR_UNSUPPORTED"),
    (dict(num_blocks=0), "PKA_ERR_SHAPE"), (dict(rows=-1), "PKA_ERR_SHAPE")] + [
    ({key: None}, "PKA_ERR_NULL") for key in ("parents", "tokens", "targets", "slots", "first", "lens",
                                              "path", "accepted", "next_tokens", "new_lens")])
def test_accept_refusals(L, kw, want):
    assert accept(L, **kw) == want


@pytest.mark.parametrize("n", [2, 40, 256, 257, 600])
def test_pools_that_share_memory_are_refused(L, n):
    """Rows of a pool named twice would move twice; the last of 8 x 2 x 16 x 256
    bytes may touch the next pool's first byte only."""
    size = 8 * 2 * 16 * 256
    order = [(7 * i) % n if math.gcd(7, n) == 1 else i for i in range(n)]
    for at, by in ((0, size), (n // 2, 16), (n - 1, size)):
        ptrs = [64 + i * size for i in order]
        ptrs[at] = ptrs[at - 1] + (size - by)        # the same pool, or its last row
        again = (ctypes.c_void_p * n)(*ptrs)
        assert accept(L, n, pools=again) == "PKA_ERR_SHAPE"
        if n % 2 == 0:
            assert evict(L, n // 2, pools=again) == "PKA_ERR_SHAPE"
    apart = (ctypes.c_void_p * n)(*[64 + i * size for i in order])
    assert accept(L, n, pools=apart, B=0) == "PKA_OK"


def evict(L, num_layers=1, pool=64, **kw):
    ptrs = (ctypes.c_void_p * 2)(pool, pool)
    a = dict(pools=ptrs, layers=num_layers, num_blocks=8, hkv=2, bs=16, d=128, tables=64,
             max_blocks=4, lens=64, total=None, B=2, budget=10, sinks=2, recent=3, mass=64,
             new_mass=64, pos=64, new_pos=64, new_lens=64, refs=None, ws=64, ws_bytes=1 << 40,
             err=None, stream=None)
    a.update(kw)
    return name(L.paged_kv_evict(*a.values()))


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), "PKA_OK"), (dict(budget=0), "PKA_ERR_SHAPE"), (dict(sinks=-1), "PKA_ERR_SHAPE"),
    (dict(recent=-1), "PKA_ERR_SHAPE"), (dict(sinks=5, recent=6), "PKA_ERR_SHAPE"),
    (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), "PKA_ERR_SHAPE"), (dict(layers=0), "PKA_ERR_SHAPE"),
    (dict(B=-1), "PKA_ERR_SHAPE"), (dict(B=2 ** 27), "PKA_ERR_SHAPE"), (dict(max_blocks=0), "PKA_ERR_SHAPE"),
    (dict(max_blocks=2 ** 27), "PKA_ERR_SHAPE"), (dict(max_blocks=2 ** 26 + 1), "PKA_ERR_SHAPE"),
    (dict(bs=8), "PKA_ERR_UNSUPPORTED"), (dict(d=512), "PKA_ERR_UNSUPPORTED"), (dict(num_blocks=0), "PKA_ERR_SHAPE"),
    (dict(pools=None), "PKA_ERR_NULL"), (dict(pool=None), "PKA_ERR_NULL"), (dict(pool=72), "PKA_ERR_ALIGN"),
    (dict(ws=66), "PKA_ERR_ALIGN"), (dict(ws_bytes=100), "PKA_ERR_WORKSPACE")] + [
    ({key: None}, "PKA_ERR_NULL") for key in ("tables", "lens", "mass", "new_mass", "pos", "new_pos",
                                              "new_lens", "ws")])
def test_evict_refusals(L, kw, want):
    assert evict(L, **kw) == want


def test_evict_workspace(L):
    assert binding.paged_kv_evict_ws_bytes(1, 2, 2, 4, 10) == 4 * (4 * (1 + 4 * 10) + 2)
    assert binding.paged_kv_evict_ws_bytes(1, 2, 2, 4, 60) == 4 * (4 * (1 + 4 * 4) + 2)
    assert binding.paged_kv_evict_ws_bytes(1, 2, 2, 4, 100) == 4 * (4 + 2)
    assert binding.paged_kv_evict_ws_bytes(1, 2, 2, 4, 0) == 0


def test_tensors_on_the_host_are_refused():
    x = torch.zeros(4, dtype=torch.int32)
    table = torch.zeros((1, 1), dtype=torch.int32)
    pool = torch.zeros((1, 1, 16, 128), dtype=torch.bfloat16)
    q = torch.zeros((4, 1, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="parents"):
        binding.paged_tree_plan(x, x[:2], x[:1], table, 1, 4, None, None, None)
    with pytest.raises(ValueError, match="q"):
        binding.paged_tree_attn_ws(q, q, pool, pool, table, x[:2], x.long(), x[:1], 4, 16, x,
                                   scale=1.0)
    with pytest.raises(ValueError, match="pools"):
        binding.paged_tree_accept([pool, pool], x, x, x, x, x[:2], x[:1], table, x[:1], x[:1], x[:1])
    with pytest.raises(ValueError, match="pools"):
        binding.paged_kv_evict([pool, pool], q, q, table, x[:1], None, 1, 0, 0, q, q, x[:1], x)
