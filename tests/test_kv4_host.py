"""Host-side refusals of the 4-bit cache and page entry points: argument errors
are found before any CUDA call, so these run without a GPU."""
import ctypes

import pytest
import torch

from paged_kv_attention_12_gb300 import _build, binding


@pytest.fixture(scope="module")
def L():
    _build.build()
    return binding.lib()


def _kv4(**kw):
    d = dict(k=256, v=512, num_blocks=8, num_kv_heads=2, block_size=16, head_dim=128, k_scale=0.5,
             v_scale=0.25)
    d.update(kw)
    return binding.PkaKv4Pool(*d.values())


def _kv16(**kw):
    d = dict(k=256, v=512, num_blocks=8, num_kv_heads=2, block_size=16, head_dim=128)
    d.update(kw)
    return binding.PkaKvPool(*d.values())


BAD_POOLS = [(dict(num_blocks=0), -2), (dict(num_kv_heads=0), -2), (dict(block_size=32), -4),
             (dict(head_dim=64), -4), (dict(head_dim=192), -4), (dict(k_scale=0.0), -2),
             (dict(v_scale=-1.0), -2), (dict(k_scale=float("nan")), -2),
             (dict(v_scale=float("inf")), -2), (dict(k_scale=3e38), -2)]


def test_pool_bytes(L):
    assert L.paged_kv4_pool_bytes(8, 2, 128) == 8 * 2 * 1152
    assert L.paged_kv4_pool_bytes(1 << 20, 8, 256) == (1 << 20) * 8 * 2304
    for bad in ((0, 2, 128), (8, -1, 128), (8, 2, 96)):
        assert L.paged_kv4_pool_bytes(*bad) == 0


def _append(L, pool=None, k=32, v=64, ks=256, vs=256, slots=128, T=4):
    return L.paged_kv4_append(k, v, ks, vs, ctypes.byref(pool or _kv4()), slots, T, None, None)


def test_append_refusals(L):
    assert _append(L, T=0, k=0, v=0, slots=0) == 0
    assert L.paged_kv4_append(32, 64, 256, 256, None, 128, 4, None, None) == -1
    for kw, st in BAD_POOLS:
        assert _append(L, pool=_kv4(**kw)) == st, kw
        assert _append(L, pool=_kv4(**kw), T=0) == st, kw
    assert _append(L, T=-1) == -2
    assert _append(L, ks=255) == -2 and _append(L, vs=248) == -2     # rows would overlap
    assert _append(L, ks=260) == -3                                  # not a multiple of 8
    assert _append(L, pool=_kv4(num_blocks=1 << 28)) == -2           # slots past 31 bits
    for kw in (dict(k=0), dict(v=0), dict(slots=0), dict(pool=_kv4(k=0)), dict(pool=_kv4(v=0))):
        assert _append(L, **kw) == -1, kw
    for kw in (dict(k=40), dict(v=72), dict(pool=_kv4(k=264)), dict(pool=_kv4(v=8))):
        assert _append(L, **kw) == -3, kw


def _expand(L, pool=None, dst=None, src=64, to=128, n=4):
    return L.paged_kv4_expand(ctypes.byref(pool or _kv4()), ctypes.byref(dst or _kv16()), src, to,
                              n, None, None)


def test_expand_refusals(L):
    assert _expand(L, n=0, src=0, to=0) == 0
    assert L.paged_kv4_expand(None, ctypes.byref(_kv16()), 64, 64, 1, None, None) == -1
    assert L.paged_kv4_expand(ctypes.byref(_kv4()), None, 64, 64, 1, None, None) == -1
    for kw, st in BAD_POOLS:
        assert _expand(L, pool=_kv4(**kw)) == st, kw
    for kw in (dict(num_blocks=0), dict(num_kv_heads=1), dict(head_dim=256), dict(block_size=32)):
        assert _expand(L, dst=_kv16(**kw)) == -2, kw
    assert _expand(L, n=-1) == -2
    assert _expand(L, n=9, to=0) == -2                               # block i past dst
    for kw in (dict(src=0), dict(pool=_kv4(k=0)), dict(dst=_kv16(v=0))):
        assert _expand(L, **kw) == -1, kw
    for kw in (dict(pool=_kv4(v=8)), dict(dst=_kv16(k=8))):
        assert _expand(L, **kw) == -3, kw


def _decode(L, pool=None, q=32, out=64, tables=128, max_blocks=4, lens=256, B=2, Hq=8, max_len=64,
            scale=0.1, softcap=0.0, par=True, ws=512, nbytes=1 << 30):
    p = binding.PkaAttnParams(scale, softcap, 0, None)
    return L.paged_kv4_decode_attn_ws(q, out, ctypes.byref(pool or _kv4()), tables, max_blocks,
                                      lens, B, Hq, max_len, ctypes.byref(p) if par else None, ws,
                                      nbytes, None)


def test_decode_refusals(L):
    assert _decode(L, B=0) == 0
    for kw, st in BAD_POOLS:
        assert _decode(L, pool=_kv4(**kw)) == st, kw
    for kw in (dict(q=0), dict(out=0), dict(tables=0), dict(lens=0), dict(par=False), dict(ws=0),
               dict(pool=_kv4(k=0)), dict(pool=_kv4(v=0))):
        assert _decode(L, **kw) == -1, kw
    nan, inf = float("nan"), float("inf")
    for kw in (dict(B=-1), dict(Hq=0), dict(Hq=7), dict(max_blocks=0), dict(max_len=-1),
               dict(max_len=65), dict(scale=nan), dict(scale=inf), dict(softcap=nan),
               dict(max_blocks=1 << 28), dict(B=1 << 20, max_blocks=1 << 16, nbytes=1 << 50)):
        assert _decode(L, **kw) == -2, kw
    assert _decode(L, Hq=18) == -4                                   # 9 heads a group
    for kw in (dict(q=40), dict(out=72), dict(ws=520), dict(pool=_kv4(k=8))):
        assert _decode(L, **kw) == -3, kw
    need = L.paged_kv4_decode_attn_ws_bytes(2, 8, 2, 128, 64, 0)
    # 64 tokens: one piece of 4 tiles, 2 slots; counters, rows, LSEs
    assert need == 2048 + 2 * 8 * 2 * 128 * 4 + 2 * 8 * 2 * 4
    assert _decode(L, nbytes=need - 1) == -5
    assert L.paged_kv4_decode_attn_ws_bytes(0, 8, 2, 128, 64, 0) == 0
    for n, w in ((1, 0), (131072, 0), (1 << 30, 0), (131072, 512), (0, 0)):
        slots = (L.paged_kv4_decode_attn_ws_bytes(1, 4, 1, 256, n, w) - 2048) // (4 * 257 * 4)
        assert 1 <= slots <= 30, (n, w, slots)
    # an empty batch needs no tensors, its sizes are checked all the same
    assert _decode(L, B=0, q=0, out=0, tables=0, lens=0, ws=0) == 0
    assert _decode(L, B=0, q=0, Hq=7) == -2


def test_page_refusals(L):
    def ref(tables=64, width=4, lens=128, B=2, n=8, refs=256):
        return L.paged_kv_ref_blocks(tables, width, lens, B, n, 1, refs, None, None)
    assert ref(B=0, tables=0, lens=0, refs=0) == 0
    for kw in (dict(B=-1), dict(width=0), dict(n=0), dict(width=1 << 28)):
        assert ref(**kw) == -2, kw
    for kw in (dict(tables=0), dict(lens=0), dict(refs=0)):
        assert ref(**kw) == -1, kw

    two = (ctypes.c_void_p * 2)(256, 512)

    def copy(pools=two, k=2, n=8, nbytes=64, src=64, dst=128, pairs=3):
        return L.paged_kv_copy_blocks(pools, k, n, nbytes, src, dst, pairs, None, None)
    assert copy(pairs=0, src=0, dst=0) == 0 and copy(k=0) == 0
    for kw in (dict(k=-1), dict(n=0), dict(nbytes=0), dict(nbytes=72), dict(nbytes=-16),
               dict(pairs=-1)):
        assert copy(**kw) == -2, kw
    for kw in (dict(pools=None), dict(src=0), dict(dst=0),
               dict(pools=(ctypes.c_void_p * 2)(256, None))):
        assert copy(**kw) == -1, kw
    assert copy(pools=(ctypes.c_void_p * 2)(256, 520)) == -3

    def compact(pools=two, k=2, n=8, nbytes=64, refs=64, new=64, tables=128, out=128, width=4,
                lens=192, B=2, remap=256, moves=320):
        return L.paged_kv_compact(pools, k, n, nbytes, refs, new, tables, out, width, lens, B,
                                  remap, moves, None, None)
    for kw in (dict(k=-1), dict(n=0), dict(nbytes=8), dict(B=-1), dict(width=0),
               dict(n=(1 << 30) + 1), dict(width=1 << 28)):
        assert compact(**kw) == -2, kw
    for kw in (dict(pools=None), dict(refs=0), dict(new=0), dict(tables=0), dict(out=0),
               dict(lens=0), dict(remap=0), dict(moves=0)):
        assert compact(**kw) == -1, kw
    assert compact(pools=(ctypes.c_void_p * 2)(264, 512)) == -3


def test_binding_refuses_host_tensors():
    k = torch.zeros((4, 2, 1, 1152), dtype=torch.uint8)
    with pytest.raises(ValueError):
        binding.Kv4Pool(k, k, 1.0, 1.0)
    t = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.paged_kv_ref_blocks(t, t[:, 0], t[0], 1)
    with pytest.raises(ValueError):
        binding.paged_kv_copy_blocks([k], t[0], t[1])
    with pytest.raises(ValueError):
        binding.Kv4Pool.zeros(4, 2, 64, 1.0, 1.0)
