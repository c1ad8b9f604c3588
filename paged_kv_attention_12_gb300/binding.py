"""ctypes binding of the C ABI in ``include/paged_attn.h``.

Argument marshalling only: every function here forwards device pointers,
sizes and the current CUDA stream to the library, where all of the work runs
in CUDA kernels.  There is no CPU fallback: if the library is missing or was
built for another machine, loading it raises.

The raw C functions are available under their C names on :func:`lib`; the
helpers below take torch tensors for convenience (the tensors are only used
for their device pointers, shapes and the current stream).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "lib", "libpaged_attn.so")

PKA_OK = 0
STATUS = {
    0: "PKA_OK", -1: "PKA_ERR_NULL", -2: "PKA_ERR_SHAPE", -3: "PKA_ERR_ALIGN",
    -4: "PKA_ERR_UNSUPPORTED", -5: "PKA_ERR_WORKSPACE", -6: "PKA_ERR_BAD_TABLE",
    -7: "PKA_ERR_TIMEOUT", -8: "PKA_ERR_CUDA",
}
DEVERR_BAD_TABLE = 1
DEVERR_TIMEOUT = 2
DEVERR_SEQ_LEN = 4
DEVERR_QUERY_LOC = 8
DEVERR_REFCOUNT = 16
DEVERR_TREE = 32

EXPORTS = [
    "pka_version", "pka_status_string", "paged_decode_attn", "paged_decode_splitk_plan",
    "paged_decode_splitk_workspace_bytes", "paged_decode_splitk",
    "paged_decode_splitk_combine", "paged_prefill_attn", "paged_attn_check_tables",
    "paged_decode_attn_noalloc", "paged_decode_attn_ws_bytes", "paged_decode_attn_ws",
    "paged_kv_append", "paged_decode_splitk_logits", "paged_decode_key_mass",
    "paged_kv_append_rope", "paged_prefill_attn_ws_bytes", "paged_prefill_attn_ws",
    "pka_selftest_bounded_wait", "paged_kv4_pool_bytes", "paged_kv4_append", "paged_kv4_expand",
    "paged_kv4_decode_attn_ws_bytes", "paged_kv4_decode_attn_ws", "paged_kv_ref_blocks",
    "paged_kv_copy_blocks", "paged_kv_compact", "paged_tree_plan", "paged_tree_attn_ws_bytes",
    "paged_tree_attn_ws", "paged_tree_accept", "paged_kv_evict_ws_bytes", "paged_kv_evict",
]

KV4_UNIT_BYTES = 1152  # 16 tokens x 128 channels of a 4-bit pool


class PkaKvPool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("num_blocks", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class PkaAttnParams(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float),
                ("window", ctypes.c_int32), ("err", ctypes.c_void_p)]


class PkaKv4Pool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("num_blocks", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class PagedAttnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")
        self.status = status


_lib = None


def use_library(path: str) -> None:
    """Load ``path`` (an instrumented build of the same library) instead of
    the default one; only before the first call into the library."""
    global LIB_PATH
    if _lib is not None and os.path.abspath(path) != os.path.abspath(LIB_PATH):
        raise RuntimeError("the library is already loaded")
    LIB_PATH = path


def lib() -> ctypes.CDLL:
    """Load the CUDA library (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, VP = ctypes.POINTER, ctypes.c_int32, ctypes.c_void_p
    L.pka_version.restype = ctypes.c_int
    L.pka_version.argtypes = []
    L.pka_status_string.restype = ctypes.c_char_p
    L.pka_status_string.argtypes = [ctypes.c_int]
    L.paged_decode_attn.restype = ctypes.c_int
    L.paged_decode_attn.argtypes = [VP, VP, P(PkaKvPool), VP, I32, VP, I32, I32, I32,
                                    P(PkaAttnParams), VP]
    L.paged_decode_splitk_plan.restype = ctypes.c_int
    L.paged_decode_splitk_plan.argtypes = [I32, I32, I32, I32, I32, I32, P(I32), P(I32)]
    L.paged_decode_splitk_workspace_bytes.restype = ctypes.c_size_t
    L.paged_decode_splitk_workspace_bytes.argtypes = [I32, I32, I32, I32]
    L.paged_decode_splitk.restype = ctypes.c_int
    L.paged_decode_splitk.argtypes = [VP, VP, VP, P(PkaKvPool), VP, I32, VP, I32, I32, I32,
                                      I32, I32, P(PkaAttnParams), VP]
    L.paged_decode_splitk_combine.restype = ctypes.c_int
    L.paged_decode_splitk_combine.argtypes = [VP, VP, I32, I32, I32, I32, VP, VP, VP]
    L.paged_prefill_attn.restype = ctypes.c_int
    L.paged_prefill_attn.argtypes = [VP, VP, P(PkaKvPool), VP, I32, VP, VP, I32, I32, I32,
                                     I32, I32, P(PkaAttnParams), VP]
    L.paged_attn_check_tables.restype = ctypes.c_int
    L.paged_attn_check_tables.argtypes = [VP, I32, VP, I32, I32, I32, VP, VP]
    L.paged_decode_attn_ws_bytes.restype = ctypes.c_size_t
    L.paged_decode_attn_ws_bytes.argtypes = [I32, I32, I32, I32, I32, I32]
    L.paged_decode_attn_ws.restype = ctypes.c_int
    L.paged_decode_attn_ws.argtypes = [VP, VP, P(PkaKvPool), VP, I32, VP, I32, I32, I32,
                                       P(PkaAttnParams), VP, ctypes.c_size_t, VP]
    L.paged_decode_attn_noalloc.restype = ctypes.c_int
    L.paged_decode_attn_noalloc.argtypes = [VP, VP, P(PkaKvPool), VP, I32, VP, I32, I32, I32,
                                            P(PkaAttnParams), VP]
    L.paged_decode_splitk_logits.restype = ctypes.c_int
    L.paged_decode_splitk_logits.argtypes = [VP, VP, VP, VP, P(PkaKvPool), VP, I32, VP, I32, I32,
                                             I32, I32, I32, P(PkaAttnParams), VP]
    L.paged_decode_key_mass.restype = ctypes.c_int
    L.paged_decode_key_mass.argtypes = [VP, VP, VP, I32, I32, I32, I32, I32, I32, VP, VP]
    L.paged_kv_append_rope.restype = ctypes.c_int
    L.paged_kv_append_rope.argtypes = [VP, VP, VP, VP, VP, I32, I32, I32, I32, I32, VP, VP, I32,
                                       VP, VP, I32, ctypes.c_float, ctypes.c_float, I32, VP, VP]
    L.paged_prefill_attn_ws_bytes.restype = ctypes.c_size_t
    L.paged_prefill_attn_ws_bytes.argtypes = [I32, I32, I32, I32, I32, I32]
    L.paged_prefill_attn_ws.restype = ctypes.c_int
    L.paged_prefill_attn_ws.argtypes = [VP, VP, P(PkaKvPool), VP, I32, VP, VP, I32, I32, I32, I32,
                                        I32, P(PkaAttnParams), VP, ctypes.c_size_t, VP]
    L.pka_selftest_bounded_wait.restype = ctypes.c_int
    L.pka_selftest_bounded_wait.argtypes = [VP, ctypes.c_int64, VP]
    L.paged_kv_append.restype = ctypes.c_int
    L.paged_kv_append.argtypes = [VP, VP, VP, VP, I32, I32, I32, I32, VP, I32, VP, VP]
    I64 = ctypes.c_int64
    L.paged_kv4_pool_bytes.restype = ctypes.c_size_t
    L.paged_kv4_pool_bytes.argtypes = [I32, I32, I32]
    L.paged_kv4_append.restype = ctypes.c_int
    L.paged_kv4_append.argtypes = [VP, VP, I64, I64, P(PkaKv4Pool), VP, I32, VP, VP]
    L.paged_kv4_expand.restype = ctypes.c_int
    L.paged_kv4_expand.argtypes = [P(PkaKv4Pool), P(PkaKvPool), VP, VP, I32, VP, VP]
    L.paged_kv4_decode_attn_ws_bytes.restype = ctypes.c_size_t
    L.paged_kv4_decode_attn_ws_bytes.argtypes = [I32, I32, I32, I32, I32, I32]
    L.paged_kv4_decode_attn_ws.restype = ctypes.c_int
    L.paged_kv4_decode_attn_ws.argtypes = [VP, VP, P(PkaKv4Pool), VP, I32, VP, I32, I32, I32,
                                           P(PkaAttnParams), VP, ctypes.c_size_t, VP]
    L.paged_kv_ref_blocks.restype = ctypes.c_int
    L.paged_kv_ref_blocks.argtypes = [VP, I32, VP, I32, I32, I32, VP, VP, VP]
    L.paged_kv_copy_blocks.restype = ctypes.c_int
    L.paged_kv_copy_blocks.argtypes = [VP, I32, I32, I64, VP, VP, I32, VP, VP]
    L.paged_kv_compact.restype = ctypes.c_int
    L.paged_kv_compact.argtypes = [VP, I32, I32, I64, VP, VP, VP, VP, I32, VP, I32, VP, VP, VP, VP]
    L.paged_tree_plan.restype = ctypes.c_int
    L.paged_tree_plan.argtypes = [VP, VP, VP, VP, VP, I32, I32, I32, I32, I32, VP, VP, VP, VP, VP]
    L.paged_tree_attn_ws_bytes.restype = ctypes.c_size_t
    L.paged_tree_attn_ws_bytes.argtypes = [I32, I32, I32, I32]
    L.paged_tree_attn_ws.restype = ctypes.c_int
    L.paged_tree_attn_ws.argtypes = [VP, VP, P(PkaKvPool), VP, I32, VP, VP, VP, I32, I32, I32, I32,
                                     I32, P(PkaAttnParams), VP, ctypes.c_size_t, VP]
    L.paged_tree_accept.restype = ctypes.c_int
    L.paged_tree_accept.argtypes = [VP, I32, I32, I32, I32, I32, VP, VP, VP, VP, VP, VP, I32, I32,
                                    I32, VP, VP, VP, VP, VP, VP]
    L.paged_kv_evict_ws_bytes.restype = ctypes.c_size_t
    L.paged_kv_evict_ws_bytes.argtypes = [I32, I32, I32, I32, I32]
    L.paged_kv_evict.restype = ctypes.c_int
    L.paged_kv_evict.argtypes = [VP, I32, I32, I32, I32, I32, VP, I32, VP, VP, I32, I32, I32, I32,
                                 VP, VP, VP, VP, VP, VP, VP, ctypes.c_size_t, VP, VP]
    _lib = L
    return L


def _check(fn: str, status: int) -> None:
    if status != PKA_OK:
        raise PagedAttnError(fn, status)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def kv_pool(k_pool, v_pool) -> PkaKvPool:
    nb, hkv, bs, d = k_pool.shape
    return PkaKvPool(k_pool.data_ptr(), v_pool.data_ptr(), nb, hkv, bs, d)


def attn_params(scale: float, softcap: float = 0.0, window: int = 0, err=None) -> PkaAttnParams:
    return PkaAttnParams(float(scale), float(softcap), int(window), _ptr(err))


# ------------------------------------------------------------------ helpers
def paged_decode_attn(q, out, k_pool, v_pool, block_tables, seq_lens, max_seq_len, *,
                      scale, softcap=0.0, window=0, err=None, stream=None):
    pool = kv_pool(k_pool, v_pool)
    par = attn_params(scale, softcap, window, err)
    st = lib().paged_decode_attn(q.data_ptr(), out.data_ptr(), ctypes.byref(pool),
                                 block_tables.data_ptr(), block_tables.shape[1],
                                 seq_lens.data_ptr(), q.shape[0], q.shape[1], int(max_seq_len),
                                 ctypes.byref(par), _stream(stream))
    _check("paged_decode_attn", st)


def paged_decode_attn_noalloc(q, out, k_pool, v_pool, block_tables, seq_lens, max_seq_len, *,
                              scale, softcap=0.0, window=0, err=None, stream=None):
    """Split-K decode with the partials in the library's own fixed array (no
    device allocation by anyone); raises PagedAttnError(PKA_ERR_WORKSPACE)
    when the partials would not fit its 16 MiB."""
    pool = kv_pool(k_pool, v_pool)
    par = attn_params(scale, softcap, window, err)
    st = lib().paged_decode_attn_noalloc(q.data_ptr(), out.data_ptr(), ctypes.byref(pool),
                                         block_tables.data_ptr(), block_tables.shape[1],
                                         seq_lens.data_ptr(), q.shape[0], q.shape[1],
                                         int(max_seq_len), ctypes.byref(par), _stream(stream))
    _check("paged_decode_attn_noalloc", st)


def paged_decode_attn_ws_bytes(B, Hq, Hkv, D, max_seq_len, window=0) -> int:
    return int(lib().paged_decode_attn_ws_bytes(B, Hq, Hkv, D, int(max_seq_len), int(window)))


def paged_decode_attn_ws(q, out, k_pool, v_pool, block_tables, seq_lens, max_seq_len, workspace,
                         *, scale, softcap=0.0, window=0, err=None, stream=None):
    pool = kv_pool(k_pool, v_pool)
    par = attn_params(scale, softcap, window, err)
    st = lib().paged_decode_attn_ws(q.data_ptr(), out.data_ptr(), ctypes.byref(pool),
                                    block_tables.data_ptr(), block_tables.shape[1],
                                    seq_lens.data_ptr(), q.shape[0], q.shape[1], int(max_seq_len),
                                    ctypes.byref(par), workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    _check("paged_decode_attn_ws", st)


def paged_decode_splitk_plan(B, Hkv, max_seq_len, block_size=16, window=0, sm_count=0):
    s, c = ctypes.c_int32(), ctypes.c_int32()
    st = lib().paged_decode_splitk_plan(B, Hkv, int(max_seq_len), block_size, int(window),
                                        int(sm_count), ctypes.byref(s), ctypes.byref(c))
    _check("paged_decode_splitk_plan", st)
    return s.value, c.value


def paged_decode_splitk_workspace_bytes(B, Hq, D, num_splits) -> int:
    return int(lib().paged_decode_splitk_workspace_bytes(B, Hq, D, num_splits))


def paged_decode_splitk(q, partial_o, partial_lse, k_pool, v_pool, block_tables, seq_lens,
                        max_seq_len, num_splits, split_blocks, *, scale, softcap=0.0, window=0,
                        err=None, stream=None):
    pool = kv_pool(k_pool, v_pool)
    par = attn_params(scale, softcap, window, err)
    st = lib().paged_decode_splitk(q.data_ptr(), partial_o.data_ptr(), partial_lse.data_ptr(),
                                   ctypes.byref(pool), block_tables.data_ptr(),
                                   block_tables.shape[1], seq_lens.data_ptr(), q.shape[0],
                                   q.shape[1], int(max_seq_len), int(num_splits),
                                   int(split_blocks), ctypes.byref(par), _stream(stream))
    _check("paged_decode_splitk", st)


def paged_decode_splitk_logits(q, partial_o, partial_lse, logits, k_pool, v_pool, block_tables,
                               seq_lens, max_seq_len, num_splits, split_blocks, *, scale,
                               softcap=0.0, window=0, err=None, stream=None):
    """paged_decode_splitk that also stores the visible keys' log2-domain
    logits in ``logits`` fp32 [B][Hq][max_blocks * 16]."""
    pool = kv_pool(k_pool, v_pool)
    par = attn_params(scale, softcap, window, err)
    st = lib().paged_decode_splitk_logits(q.data_ptr(), partial_o.data_ptr(),
                                          partial_lse.data_ptr(), logits.data_ptr(),
                                          ctypes.byref(pool), block_tables.data_ptr(),
                                          block_tables.shape[1], seq_lens.data_ptr(), q.shape[0],
                                          q.shape[1], int(max_seq_len), int(num_splits),
                                          int(split_blocks), ctypes.byref(par), _stream(stream))
    _check("paged_decode_splitk_logits", st)


def paged_decode_key_mass(logits, lse, seq_lens, num_kv_heads, key_mass, *, window=0,
                          block_size=16, stream=None):
    """key_mass fp32 [B][Hkv][max_blocks * 16] += each visible key's attention
    probability summed over its KV head's query heads (``lse``: [B][Hq]
    natural-log LSE from the combine)."""
    B, Hq, nk = logits.shape
    st = lib().paged_decode_key_mass(logits.data_ptr(), lse.data_ptr(), seq_lens.data_ptr(), B,
                                     Hq, int(num_kv_heads), nk // block_size, block_size,
                                     int(window), key_mass.data_ptr(), _stream(stream))
    _check("paged_decode_key_mass", st)


def paged_decode_splitk_combine(partial_o, partial_lse, out, lse_out=None, stream=None):
    B, Hq, S, D = partial_o.shape
    st = lib().paged_decode_splitk_combine(partial_o.data_ptr(), partial_lse.data_ptr(), B, Hq,
                                           D, S, out.data_ptr(), _ptr(lse_out), _stream(stream))
    _check("paged_decode_splitk_combine", st)


def paged_prefill_attn(q, out, k_pool, v_pool, block_tables, query_start_loc, seq_lens,
                       max_query_len, max_seq_len, *, scale, softcap=0.0, window=0, err=None,
                       stream=None):
    pool = kv_pool(k_pool, v_pool)
    par = attn_params(scale, softcap, window, err)
    st = lib().paged_prefill_attn(q.data_ptr(), out.data_ptr(), ctypes.byref(pool),
                                  block_tables.data_ptr(), block_tables.shape[1],
                                  query_start_loc.data_ptr(), seq_lens.data_ptr(),
                                  seq_lens.shape[0], q.shape[1], q.shape[0], int(max_query_len),
                                  int(max_seq_len), ctypes.byref(par), _stream(stream))
    _check("paged_prefill_attn", st)


def paged_prefill_attn_ws_bytes(B, Hq, Hkv, D, max_seq_len, window=0) -> int:
    return int(lib().paged_prefill_attn_ws_bytes(B, Hq, Hkv, D, int(max_seq_len), int(window)))


def paged_prefill_attn_ws(q, out, k_pool, v_pool, block_tables, query_start_loc, seq_lens,
                          max_query_len, max_seq_len, workspace, *, scale, softcap=0.0, window=0,
                          err=None, stream=None):
    """Mixed batch in one launch: decode rows on decode pipelines, chunks on
    the tensor-core prefill pipeline.  ``workspace``: zero-initialised device
    bytes, at least ``paged_prefill_attn_ws_bytes``; left zeroed."""
    pool = kv_pool(k_pool, v_pool)
    par = attn_params(scale, softcap, window, err)
    st = lib().paged_prefill_attn_ws(q.data_ptr(), out.data_ptr(), ctypes.byref(pool),
                                     block_tables.data_ptr(), block_tables.shape[1],
                                     query_start_loc.data_ptr(), seq_lens.data_ptr(),
                                     seq_lens.shape[0], q.shape[1], q.shape[0],
                                     int(max_query_len), int(max_seq_len), ctypes.byref(par),
                                     workspace.data_ptr(), workspace.numel(), _stream(stream))
    _check("paged_prefill_attn_ws", st)


def selftest_bounded_wait(err, budget_cycles, stream=None):
    """A wait that can never complete, with the library's wait routine and a
    budget of ``budget_cycles``: it must end with PKA_DEVERR_TIMEOUT in
    ``err`` (device int32)."""
    st = lib().pka_selftest_bounded_wait(err.data_ptr(), int(budget_cycles), _stream(stream))
    _check("pka_selftest_bounded_wait", st)


def paged_attn_check_tables(block_tables, seq_lens, num_blocks, err, block_size=16, stream=None):
    st = lib().paged_attn_check_tables(block_tables.data_ptr(), block_tables.shape[1],
                                       seq_lens.data_ptr(), seq_lens.shape[0], int(num_blocks),
                                       block_size, err.data_ptr(), _stream(stream))
    _check("paged_attn_check_tables", st)


def paged_kv_append(k_new, v_new, k_pool, v_pool, slot_mapping, err=None, stream=None):
    """Write token t's K/V rows (``k_new``/``v_new`` bf16 [T][Hkv][D]) into
    the pools at slot ``slot_mapping[t]`` (int32, block * bs + offset; < 0
    skips the token)."""
    nb, hkv, bs, d = k_pool.shape
    st = lib().paged_kv_append(k_new.data_ptr(), v_new.data_ptr(), k_pool.data_ptr(),
                               v_pool.data_ptr(), nb, hkv, bs, d, slot_mapping.data_ptr(),
                               slot_mapping.shape[0], err.data_ptr() if err is not None else None,
                               _stream(stream))
    _check("paged_kv_append", st)


def paged_kv_append_rope(q, k_new, v_new, k_pool, v_pool, slot_mapping, positions, *,
                         q_norm_weight=None, k_norm_weight=None, v_norm=False, eps=1e-6,
                         rope_theta=10000.0, rotary_dim=None, err=None, stream=None):
    """RMS-norm q / k / v, rotate q and k (rotate-half RoPE over the first
    ``rotary_dim`` channels, default all), append k / v at their slots and
    overwrite q (or skip it when ``q`` is None)."""
    nb, hkv, bs, d = k_pool.shape
    rd = d if rotary_dim is None else int(rotary_dim)
    st = lib().paged_kv_append_rope(
        _ptr(q), k_new.data_ptr(), v_new.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), nb,
        q.shape[1] if q is not None else 0, hkv, bs, d, slot_mapping.data_ptr(),
        _ptr(positions), slot_mapping.shape[0], _ptr(q_norm_weight), _ptr(k_norm_weight),
        1 if v_norm else 0, float(eps), float(rope_theta), rd, _ptr(err), _stream(stream))
    _check("paged_kv_append_rope", st)


# ------------------------------------------------- 4-bit cache and its pages
# These check their tensors (device, type, layout, shape) before the call and
# raise ValueError; they run on the tensors' device, on its current stream
# unless one is given.  A decode step makes these calls for every layer, so the
# checks are plain comparisons, and build no text unless one fails.
def _refuse(t, name: str, want: str):
    raise ValueError(f"{name}: {want} is wanted, got {t.dtype} {list(t.shape)} with strides "
                     f"{t.stride()} on {t.device}")


def _dims(*shape) -> str:
    return "".join(f"[{x}]" for x in shape)


def _tensor(t, name: str, dtype, device, shape) -> None:
    """Refuses what is no contiguous tensor of ``dtype`` and ``shape`` on ``device``."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    _refuse(t, name, f"contiguous {dtype} {_dims(*shape)} on {device}")


def _cuda_device(t, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name}: a tensor on a CUDA device is wanted, got one on {t.device}")
    return t.device


def _err(err, device) -> int:
    import torch
    _tensor(err, "err", torch.int32, device, (max(1, err.numel()),))
    return err.data_ptr()


def _elsewhere(device) -> bool:
    """Whether ``device`` is not the current one (the library launches there)."""
    import torch
    return device.index != torch._C._cuda_getDevice()


def _raw_stream(device, stream):
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None \
        else stream.cuda_stream


class Kv4Pool:
    """A layer's 4-bit cache: uint8 ``k`` and ``v`` of shape
    ``[num_blocks][Hkv][D / 128][1152]`` and their fp32 scales (the format is
    described at ``pka_kv4_pool`` in ``include/paged_attn.h``)."""

    def __init__(self, k, v, k_scale: float, v_scale: float):
        import torch
        dev = _cuda_device(k, "k")
        for t, name in ((k, "k"), (v, "v")):
            _tensor(t, name, torch.uint8, dev, k.shape)
            if t.dim() != 4 or t.shape[3] != KV4_UNIT_BYTES or t.shape[2] not in (1, 2):
                _refuse(t, name, f"uint8 [num_blocks][Hkv][D / 128][{KV4_UNIT_BYTES}]")
        self.k, self.v = k, v
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.num_blocks, self.num_kv_heads, units, _ = k.shape
        self.head_dim = 128 * units
        self.device = dev
        self._c = PkaKv4Pool(k.data_ptr(), v.data_ptr(), self.num_blocks, self.num_kv_heads, 16,
                             self.head_dim, self.k_scale, self.v_scale)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def zeros(cls, num_blocks: int, num_kv_heads: int, head_dim: int, k_scale: float,
              v_scale: float, device="cuda") -> "Kv4Pool":
        """An empty pool (every value 0)."""
        import torch
        if head_dim not in (128, 256):
            raise ValueError(f"head_dim 128 or 256 is wanted, got {head_dim}")
        shape = (num_blocks, num_kv_heads, head_dim // 128, KV4_UNIT_BYTES)
        return cls(torch.zeros(shape, dtype=torch.uint8, device=device),
                   torch.zeros(shape, dtype=torch.uint8, device=device), k_scale, v_scale)


def _token_rows(t, name: str, T: int, pool: Kv4Pool) -> int:
    """Checks bf16 rows [T][Hkv][D], contiguous within a token; their token stride."""
    import torch
    h, d = pool.num_kv_heads, pool.head_dim
    if t.dtype is not torch.bfloat16 or t.device != pool.device or t.shape != (T, h, d):
        _refuse(t, name, f"bfloat16 {_dims(T, h, d)} on {pool.device}")
    if T == 0:
        return h * d
    s0, s1, s2 = t.stride()
    if s2 != 1 or (h > 1 and s1 != d):
        _refuse(t, name, f"rows of a token side by side (strides [...][{d}][1])")
    # a single token has no next one: its stride says nothing
    return h * d if T == 1 else s0


def paged_kv4_append(k_new, v_new, pool: Kv4Pool, slot_mapping, err=None, stream=None):
    """Quantise token t's K/V rows (``k_new``/``v_new`` bf16 [T][Hkv][D]; the
    tokens may be strided, as slices of a wider projection are) and write them
    to ``pool`` at slot ``slot_mapping[t]`` (int32; < 0 skips the token)."""
    import torch
    dev, T = pool.device, slot_mapping.shape[0]
    ks, vs = _token_rows(k_new, "k_new", T, pool), _token_rows(v_new, "v_new", T, pool)
    _tensor(slot_mapping, "slot_mapping", torch.int32, dev, (T,))
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return paged_kv4_append(k_new, v_new, pool, slot_mapping, err, stream)
    st = lib().paged_kv4_append(
        k_new.data_ptr(), v_new.data_ptr(), ks, vs, pool._ref, slot_mapping.data_ptr(), T, None if
        err is None else _err(err, dev), _raw_stream(dev, stream))
    if st != PKA_OK:
        raise PagedAttnError("paged_kv4_append", st)


def paged_kv4_expand(pool: Kv4Pool, k_pool, v_pool, src_blocks, dst_blocks=None, err=None,
                     stream=None):
    """Write blocks ``src_blocks`` (int32, any shape; < 0 skips) of a 4-bit
    pool to blocks ``dst_blocks`` (default 0, 1, ...) of bf16 pools
    [num_blocks][Hkv][16][D], as the prefill entry points read them."""
    import torch
    dev = pool.device
    shape = (k_pool.shape[0], pool.num_kv_heads, 16, pool.head_dim)
    _tensor(k_pool, "k_pool", torch.bfloat16, dev, shape)
    _tensor(v_pool, "v_pool", torch.bfloat16, dev, shape)
    _tensor(src_blocks, "src_blocks", torch.int32, dev, src_blocks.shape)
    if dst_blocks is not None:
        _tensor(dst_blocks, "dst_blocks", torch.int32, dev, src_blocks.shape)
    dst = PkaKvPool(k_pool.data_ptr(), v_pool.data_ptr(), *shape)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return paged_kv4_expand(pool, k_pool, v_pool, src_blocks, dst_blocks, err, stream)
    st = lib().paged_kv4_expand(
        pool._ref, ctypes.byref(dst), src_blocks.data_ptr(), _ptr(dst_blocks), src_blocks.numel(),
        None if err is None else _err(err, dev), _raw_stream(dev, stream))
    if st != PKA_OK:
        raise PagedAttnError("paged_kv4_expand", st)


def paged_kv4_decode_attn_ws_bytes(B, Hq, Hkv, D, max_seq_len, window=0) -> int:
    return int(lib().paged_kv4_decode_attn_ws_bytes(B, Hq, Hkv, D, int(max_seq_len), int(window)))


def paged_kv4_decode_attn_ws(q, out, pool: Kv4Pool, block_tables, seq_lens, max_seq_len, workspace,
                             *, scale, softcap=0.0, window=0, err=None, stream=None):
    """Decode over a 4-bit cache in one launch: ``q``, ``out`` bf16
    [B][Hq][D].  ``workspace``: device bytes, zero before their first use, at
    least ``paged_kv4_decode_attn_ws_bytes``; not to be shared by calls that
    can overlap."""
    import torch
    dev = pool.device
    shape = B, Hq, _ = (seq_lens.shape[0], q.shape[1], pool.head_dim)
    width = block_tables.shape[-1]
    if not (q.dtype is torch.bfloat16 and out.dtype is torch.bfloat16 and
            block_tables.dtype is torch.int32 and seq_lens.dtype is torch.int32 and
            q.shape == shape and out.shape == shape and block_tables.shape == (B, width) and
            seq_lens.dim() == 1 and
            dev == q.device == out.device == block_tables.device == seq_lens.device ==
            workspace.device and
            q.is_contiguous() and out.is_contiguous() and block_tables.is_contiguous() and
            seq_lens.is_contiguous() and workspace.is_contiguous()):
        _tensor(q, "q", torch.bfloat16, dev, shape)
        _tensor(out, "out", torch.bfloat16, dev, shape)
        _tensor(block_tables, "block_tables", torch.int32, dev, (B, width))
        _tensor(seq_lens, "seq_lens", torch.int32, dev, (B,))
        _tensor(workspace, "workspace", workspace.dtype, dev, workspace.shape)
    par = PkaAttnParams(scale, softcap, window, None if err is None else _err(err, dev))
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return paged_kv4_decode_attn_ws(
                q, out, pool, block_tables, seq_lens, max_seq_len, workspace, scale=scale,
                softcap=softcap, window=window, err=err, stream=stream)
    st = lib().paged_kv4_decode_attn_ws(
        q.data_ptr(), out.data_ptr(), pool._ref, block_tables.data_ptr(), width,
        seq_lens.data_ptr(), B, Hq, int(max_seq_len), ctypes.byref(par), workspace.data_ptr(),
        workspace.nbytes, _raw_stream(dev, stream))
    if st != PKA_OK:
        raise PagedAttnError("paged_kv4_decode_attn_ws", st)


def paged_kv_ref_blocks(block_tables, seq_lens, refcounts, delta: int, err=None, stream=None):
    """Add ``delta`` to ``refcounts`` (int32 [num_blocks]) for every block the
    rows of ``block_tables`` use: +1 forks the requests, -1 frees them."""
    import torch
    dev = _cuda_device(block_tables, "block_tables")
    B, width = seq_lens.shape[0], block_tables.shape[-1]
    _tensor(block_tables, "block_tables", torch.int32, dev, (B, width))
    _tensor(seq_lens, "seq_lens", torch.int32, dev, (B,))
    n = refcounts.shape[0]
    _tensor(refcounts, "refcounts", torch.int32, dev, (n,))
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return paged_kv_ref_blocks(block_tables, seq_lens, refcounts, delta, err, stream)
    st = lib().paged_kv_ref_blocks(
        block_tables.data_ptr(), width, seq_lens.data_ptr(), B, n, int(delta), refcounts.data_ptr(),
        None if err is None else _err(err, dev), _raw_stream(dev, stream))
    if st != PKA_OK:
        raise PagedAttnError("paged_kv_ref_blocks", st)


def _pool_list(pools):
    """The pools' device pointers as a C array, their blocks, bytes per block and device."""
    first = pools[0]
    dev, shape, dtype = _cuda_device(first, "pools"), first.shape, first.dtype
    for p in pools:
        if p.shape != shape or p.dtype is not dtype or p.device != dev or not p.is_contiguous():
            _refuse(p, "pools", f"contiguous {dtype} {_dims(*shape)} on {dev}")
    n = shape[0]
    return ((ctypes.c_void_p * len(pools))(*[p.data_ptr() for p in pools]), n,
            first.nbytes // max(n, 1), dev)


def paged_kv_copy_blocks(pools, src, dst, err=None, stream=None):
    """Copy block ``src[i]`` to block ``dst[i]`` (int32) in each of ``pools``
    (tensors [num_blocks][...] of one shape and type: K and V of every layer).
    The destinations must be distinct and none of them a source."""
    import torch
    if not pools:
        return
    ptrs, n, nbytes, dev = _pool_list(pools)
    pairs = src.shape[0]
    _tensor(src, "src", torch.int32, dev, (pairs,))
    _tensor(dst, "dst", torch.int32, dev, (pairs,))
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return paged_kv_copy_blocks(pools, src, dst, err, stream)
    st = lib().paged_kv_copy_blocks(
        ptrs, len(ptrs), n, nbytes, src.data_ptr(), dst.data_ptr(), pairs, None if err is None else
        _err(err, dev), _raw_stream(dev, stream))
    if st != PKA_OK:
        raise PagedAttnError("paged_kv_copy_blocks", st)


def paged_kv_compact(pools, refcounts, block_tables, seq_lens, new_refcounts, new_tables, remap,
                     moves, err=None, stream=None):
    """Move the live blocks (``refcounts`` > 0) of every pool to ids 0, 1, ...
    and give the new counts, tables, the map old id -> new id and the moves
    (int32 [2 + num_blocks]: their number, the live blocks, then pairs).
    ``new_refcounts`` and ``new_tables`` may be the old ones.  Without pools
    only the plan and the tables are worked out."""
    import torch
    ptrs, n, nbytes, dev = _pool_list(pools) if pools else \
        (None, refcounts.shape[0], 0, _cuda_device(refcounts, "refcounts"))
    i32, B, width = torch.int32, seq_lens.shape[0], block_tables.shape[-1]
    _tensor(refcounts, "refcounts", i32, dev, (n,))
    _tensor(new_refcounts, "new_refcounts", i32, dev, (n,))
    _tensor(remap, "remap", i32, dev, (n,))
    _tensor(moves, "moves", i32, dev, (n + 2,))
    _tensor(block_tables, "block_tables", i32, dev, (B, width))
    _tensor(new_tables, "new_tables", i32, dev, (B, width))
    _tensor(seq_lens, "seq_lens", i32, dev, (B,))
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return paged_kv_compact(pools, refcounts, block_tables, seq_lens, new_refcounts,
                                    new_tables, remap, moves, err, stream)
    st = lib().paged_kv_compact(
        ptrs, len(pools), n, nbytes, refcounts.data_ptr(), new_refcounts.data_ptr(),
        block_tables.data_ptr(), new_tables.data_ptr(), width, seq_lens.data_ptr(), B,
        remap.data_ptr(), moves.data_ptr(), None if err is None else _err(err, dev),
        _raw_stream(dev, stream))
    if st != PKA_OK:
        raise PagedAttnError("paged_kv_compact", st)


# ------------------------------------- draft trees and eviction by mass
# These calls check their tensors as the ones above do (ValueError), in the
# module lib/_native.so: between small kernels the checks would cost more than
# the launch.
_native_module = None


def _native():
    global _native_module
    if _native_module is None:
        import importlib.machinery
        import importlib.util

        import torch  # noqa: F401  (its libraries come first)
        L = lib()
        path = os.path.join(HERE, "lib", "_native.so")
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
        from . import _build
        if not _build.native_fits():
            raise RuntimeError(
                f"{path} was built for another Python or torch: build it again (python -c 'import "
                "__graft_entry__ as g; g.build()')")
        loader = importlib.machinery.ExtensionFileLoader("_native", path)
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_native", loader))
        loader.exec_module(m)
        m.attach(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.paged_tree_plan, L.paged_tree_attn_ws, L.paged_tree_accept, L.paged_kv_evict)))
        _native_module = m
    return _native_module


def paged_tree_plan(parents, query_start_loc, seq_lens, block_tables, num_blocks: int,
                    max_query_len: int, tree_masks, positions, slots, *, total_lens=None, err=None,
                    stream=None):
    """Ancestor masks (int64 [total_q]), positions and cache slots (int32) of
    drafted tokens from their ``parents`` (int32 [total_q], indexes within a
    tree, -1: none).  An output may be None."""
    st = (_native_module or _native()).tree_plan(
        parents, query_start_loc, seq_lens, block_tables, num_blocks, max_query_len, tree_masks,
        positions, slots, total_lens, err, stream)
    if st != PKA_OK:
        raise PagedAttnError("paged_tree_plan", st)


def paged_tree_attn_ws_bytes(Hq, Hkv, D, max_query_len) -> int:
    return int(lib().paged_tree_attn_ws_bytes(Hq, Hkv, D, int(max_query_len)))


def paged_tree_attn_ws(q, out, k_pool, v_pool, block_tables, query_start_loc, tree_masks, seq_lens,
                       max_query_len, max_seq_len, workspace, *, scale, softcap=0.0, window=0,
                       err=None, stream=None):
    """Attention of drafted tokens over their requests' cached prefixes and, by
    ``tree_masks`` (int64 [total_q], bit j: token j), each other: ``q``, ``out``
    bf16 [total_q][Hq][D].  ``workspace``: device bytes, at least
    ``paged_tree_attn_ws_bytes``; not to be shared by calls that can overlap."""
    st = (_native_module or _native()).tree_attn_ws(
        q, out, k_pool, v_pool, block_tables, query_start_loc, tree_masks, seq_lens, max_query_len,
        max_seq_len, workspace, scale, softcap, window, err, stream)
    if st != PKA_OK:
        raise PagedAttnError("paged_tree_attn_ws", st)


def paged_tree_accept(pools, parents, tokens, targets, slots, query_start_loc, seq_lens, path,
                      accepted, next_tokens, new_seq_lens, err=None, stream=None):
    """Walk each tree along the target model's tokens (``targets``, one after
    each drafted token) and move the accepted tokens' rows in ``pools`` (bf16, K
    and V of every layer) to the tree's first ``slots``.  Writes ``path`` (int32
    [B][max_query_len]), ``accepted``, ``next_tokens`` and ``new_seq_lens``
    (may be ``seq_lens``).  Without pools the walk alone (``slots`` may be None)."""
    st = (_native_module or _native()).tree_accept(
        pools, parents, tokens, targets, slots, query_start_loc, seq_lens, path, accepted,
        next_tokens, new_seq_lens, err, stream)
    if st != PKA_OK:
        raise PagedAttnError("paged_tree_accept", st)


def paged_kv_evict_ws_bytes(num_layers, B, Hkv, max_blocks, budget) -> int:
    return int(lib().paged_kv_evict_ws_bytes(num_layers, B, Hkv, max_blocks, int(budget)))


def paged_kv_evict(pools, key_mass, key_pos, block_tables, seq_lens, total_lens, budget: int,
                   sinks: int, recent: int, new_mass, new_pos, new_seq_lens, workspace, *,
                   refcounts=None, err=None, stream=None):
    """Hold every (layer, request, KV head) of a cache to ``budget`` keys: those
    at positions below ``sinks``, the ``recent`` last ones and the heaviest by
    ``key_mass`` (fp32 [layers][B][Hkv][max_blocks * 16]; ``key_pos`` int32, -1:
    appended since the last eviction).  Rows move in ``pools`` (bf16, K and V of
    layer 0, 1, ...); the outputs may be the inputs.  ``total_lens`` None: the
    sequences' lengths are their caches'.  With ``refcounts`` requests that share
    a block to be written are left whole.  ``workspace``: device bytes, at least
    ``paged_kv_evict_ws_bytes``; not to be shared by calls that can overlap."""
    st = (_native_module or _native()).kv_evict(
        pools, key_mass, key_pos, block_tables, seq_lens, total_lens, budget, sinks, recent,
        new_mass, new_pos, new_seq_lens, workspace, refcounts, err, stream)
    if st != PKA_OK:
        raise PagedAttnError("paged_kv_evict", st)


# ------------------------------------------------------------ batch runners
class DecodeSplitK:
    """Split-K decode of one batch: plan once, own the fp32 partials, run.

    ``run`` issues two launches (split-K partials, then the combine) on the
    current stream.
    """

    def __init__(self, batch, sm_count: int = 0):
        import torch
        self.batch = batch
        B, Hkv, D, Hq = batch.num_requests, batch.num_kv_heads, batch.head_dim, batch.num_q_heads
        self.num_splits, self.split_blocks = paged_decode_splitk_plan(
            B, Hkv, batch.max_seq_len, batch.block_size, batch.window, sm_count)
        dev = batch.q.device
        self.partial_o = torch.empty((B, Hq, self.num_splits, D), dtype=torch.float32, device=dev)
        self.partial_lse = torch.empty((B, Hq, self.num_splits), dtype=torch.float32, device=dev)
        self.out = torch.empty_like(batch.q)

    def run(self, err=None, lse_out=None):
        b = self.batch
        paged_decode_splitk(b.q, self.partial_o, self.partial_lse, b.k_pool, b.v_pool,
                            b.block_tables, b.seq_lens, b.max_seq_len, self.num_splits,
                            self.split_blocks, scale=b.scale, softcap=b.softcap,
                            window=b.window, err=err)
        paged_decode_splitk_combine(self.partial_o, self.partial_lse, self.out, lse_out)
        return self.out


class DecodeFused:
    """Split-K decode with the combine fused in: one launch per call.  Owns a
    zero-initialised workspace (its counters are left zero by each call)."""

    def __init__(self, batch):
        import torch
        self.batch = batch
        nbytes = paged_decode_attn_ws_bytes(batch.num_requests, batch.num_q_heads,
                                            batch.num_kv_heads, batch.head_dim, batch.max_seq_len,
                                            batch.window)
        self.workspace = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device=batch.q.device)
        self.out = torch.empty_like(batch.q)

    def run(self, err=None):
        b = self.batch
        paged_decode_attn_ws(b.q, self.out, b.k_pool, b.v_pool, b.block_tables, b.seq_lens,
                             b.max_seq_len, self.workspace, scale=b.scale, softcap=b.softcap,
                             window=b.window, err=err)
        return self.out


class MixedBatch:
    """A varlen batch (decode rows and prefill chunks) in one launch through
    ``paged_prefill_attn_ws``.  Owns a zero-initialised workspace."""

    def __init__(self, batch):
        import torch
        self.batch = batch
        nbytes = paged_prefill_attn_ws_bytes(batch.num_requests, batch.num_q_heads,
                                             batch.num_kv_heads, batch.head_dim,
                                             batch.max_seq_len, batch.window)
        self.workspace = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device=batch.q.device)
        self.out = torch.empty_like(batch.q)

    def run(self, err=None):
        b = self.batch
        paged_prefill_attn_ws(b.q, self.out, b.k_pool, b.v_pool, b.block_tables,
                              b.query_start_loc, b.seq_lens, b.max_query_len, b.max_seq_len,
                              self.workspace, scale=b.scale, softcap=b.softcap, window=b.window,
                              err=err)
        return self.out


def run_batch(batch, out=None, err=None):
    """Attention of one batch through the library (decode or varlen prefill)."""
    import torch
    if out is None:
        out = torch.empty_like(batch.q)
    paged_prefill_attn(batch.q, out, batch.k_pool, batch.v_pool, batch.block_tables,
                       batch.query_start_loc, batch.seq_lens, batch.max_query_len,
                       batch.max_seq_len, scale=batch.scale, softcap=batch.softcap,
                       window=batch.window, err=err)
    return out
