"""Oracle of the 4-bit cache (TEST INFRASTRUCTURE; see the package doc).

A value is held as e2m1 (levels 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign) with
one e4m3 scale per 16 channels of a token and one fp32 scale per pool.  The
levels of both small formats are tabulated from their definitions here and
every rounding is a search for the nearest level (ties to the even code), in
fp64 on operands rounded to fp32 where the definition rounds.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# e4m3: codes 0 .. 126 are the non-negative finite values, 127 is NaN
E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])
UNIT = 1152


def nearest(levels: np.ndarray, x: np.ndarray) -> np.ndarray:
    """Index of the level nearest to x >= 0 (saturating; ties to the even index)."""
    x = np.minimum(np.asarray(x, dtype=np.float64), levels[-1])
    hi = np.clip(np.searchsorted(levels, x, side="left"), 1, len(levels) - 1)
    lo = hi - 1
    up, down = levels[hi] - x, x - levels[lo]
    return np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))


def kv4_quantise(x: np.ndarray, pool_scale: float):
    """x [..., D] -> (codes uint8 [..., D], scale bytes uint8 [..., D / 16])."""
    f32 = np.float32
    g = np.asarray(x, dtype=f32).reshape(*x.shape[:-1], -1, 16)
    with np.errstate(all="ignore"):
        top = np.abs(g).max(-1)
        bad = ~np.isfinite(g).all(-1)
        r = np.where(bad, f32(0), top) / (f32(6) * f32(pool_scale))
        sb = nearest(E4M3, np.minimum(r, f32(448)))
        step = (E4M3[sb].astype(f32) * f32(pool_scale))[..., None]
        y = np.where(step > 0, np.where(bad[..., None], f32(0), g) / np.where(step > 0, step, f32(1)),
                     f32(0))
    code = nearest(E2M1, np.abs(y)) + 8 * np.signbit(g)
    code = np.where(bad[..., None], 0, code)
    sb = np.where(bad, 127, sb)
    return code.reshape(x.shape).astype(np.uint8), sb.astype(np.uint8)


def kv4_place(tok: int, ch: int, is_v: bool):
    """(byte of the code, shift of its nibble, byte of its scale) inside a unit."""
    grp, c = ch // 16, ch % 16
    if is_v:
        first = (tok + 8) % 16 if grp % 2 else tok
        return grp * 128 + first * 8 + c // 2, 4 * (c % 2), 1024 + grp * 16 + tok
    return tok * 64 + ch // 2, 4 * (ch % 2), 1024 + tok * 8 + grp


def _maps(is_v):
    byte = np.zeros((16, 128), dtype=np.int64)
    shift, scale = byte.copy(), byte.copy()
    for t in range(16):
        for c in range(128):
            byte[t, c], shift[t, c], scale[t, c] = kv4_place(t, c, is_v)
    return byte, shift, scale


_MAPS = {v: _maps(v) for v in (False, True)}


def kv4_append(pool: np.ndarray, rows: np.ndarray, slot_mapping, pool_scale: float, is_v: bool):
    """A copy of ``pool`` uint8 [num_blocks][Hkv][U][1152] with token t's rows
    [T][Hkv][D] at slot_mapping[t] (< 0 or past the pool: skipped)."""
    out = pool.copy()
    codes, scales = kv4_quantise(rows, pool_scale)
    byte, shift, scale = _MAPS[is_v]
    U = pool.shape[2]
    for t, s in enumerate(np.asarray(slot_mapping).tolist()):
        blk, tok = divmod(int(s), 16)
        if s < 0 or blk >= pool.shape[0]:
            continue
        for u in range(U):
            unit = out[blk, :, u]
            c = codes[t][:, u * 128:(u + 1) * 128]
            for sh in (0, 4):
                at = shift[tok] == sh
                b = byte[tok][at]
                unit[:, b] = (unit[:, b] & (0xf0 if sh == 0 else 0x0f)) | (c[:, at] << sh)
            unit[:, scale[tok][::16]] = scales[t][:, u * 8:(u + 1) * 8]
    return out


def kv4_decode(pool: np.ndarray, pool_scale: float, is_v: bool, exact: bool = True):
    """Values [num_blocks][Hkv][16][D] of a pool: fp64 (``exact``), or fp32
    with the product by the pool scale rounded to fp32."""
    byte, shift, scale = _MAPS[is_v]
    code = (pool[..., byte] >> shift.astype(np.uint8)) & 15      # [n][h][U][16][128]
    sb = pool[..., scale]
    fac = np.where((sb & 127) == 127, np.nan, np.append(E4M3, 0.0)[sb & 127])
    val = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7] * fac
    val = val * np.float64(np.float32(pool_scale)) if exact else \
        val.astype(np.float32) * np.float32(pool_scale)
    n, h, U = pool.shape[:3]
    return np.moveaxis(val, 2, 3).reshape(n, h, 16, U * 128)
