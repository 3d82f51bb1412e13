"""Paged KV-cache attention for GB300 (sm_103a): Python binding of libpkv.

Argument marshalling only.  Every step of the computation runs in the CUDA
kernels of ``libpkv.so`` (built from ``csrc/`` by ``build()``); this module
checks shapes and dtypes, takes raw device pointers from torch tensors and
the current torch stream, and calls the C ABI declared in ``include/pkv.h``.
There is no CPU or PyTorch fallback: if the library is missing or a call
fails, an exception is raised.

Operations (same names as the C ABI):
  * ``reshape_and_cache`` -- write new K/V rows into the paged pools at
    ``slot_mapping`` (vLLM attention.py, PagedAttention.forward);
  * ``rope_reshape_and_cache`` -- the rotary embedding of q and k by position
    (neox or GPT-J pairing, partial rotary_dim, scaled tables from
    ``rope_cos_sin_table``) fused with that write (vLLM attention.py,
    PagedAttentionWithRoPE);
  * ``paged_decode`` (and ``paged_decode_noalloc``, which needs no workspace)
    -- one query per sequence over its pages through ``block_table`` /
    ``cache_seqlens`` (transformers docs "paged_attention", decode path),
    split-KV with 512-token partitions;
  * ``varlen_prefill`` -- varlen / chunk prefill addressed by
    ``cu_seq_lens_q`` / ``cu_seq_lens_k`` (transformers docs
    "paged_attention", varlen path), keys read from the pages, causal or not;
    ``varlen_prefill_contiguous`` reads them from [total_k, Hkv, D] arrays;
  * ``reshape_and_cache_fp8``, ``gather_cache_fp8`` and ``paged_decode_fp8`` --
    the write, the read back (as bf16) and the decode of an 8-bit cache: e4m3
    codes with one power-of-two scale per token and kv head;
  * ``qk_norm_rope_reshape_and_cache`` -- the RMS norm of the q and k heads, the
    rotary embedding and the cache write (bf16, float32 or 8-bit pools) fused;
  * ``paged_tree_attention`` -- attention of a tree of up to 256 drafted tokens
    per request over its pages (bf16 or 8-bit), for speculative decoding;
  * ``update_block_tables`` -- pages taken and given back, slots, positions and
    offsets of a step's tokens from the requests' lengths, on the GPU;
  * ``update_page_bounds``, ``select_pages`` and ``paged_sparse_attention`` -- a
    sparse step: 8-bit bounds of every page's keys, for each query the pages on
    which a key could score highest, and the attention over these pages alone;
  * ``minference_prefill`` -- MInference's vertical + slash sparse prefill of
    one sequence (nano-vllm minference.py): pattern estimate, top-k, then
    attention over the kept keys.
The attention calls support GQA, ``window_left``, the per-head attention sink
of FlashInfer's sink_attention_reference.py, ALiBi slopes, head sizes 64, 80,
96, 112, 128 and 256, and NHD or HND page layouts.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional

from ._build import LIB_PATH, build as _build_lib

__all__ = [
    "build", "load_library", "PkvError", "reshape_and_cache", "paged_decode",
    "varlen_prefill", "varlen_prefill_contiguous", "paged_decode_noalloc",
    "paged_decode_workspace_size", "varlen_prefill_workspace_size",
    "rope_cos_sin_table", "rope_reshape_and_cache", "get_device_error",
    "selftest_bounded_wait",
    "minference_sizes", "minference_prefill",
    "reshape_and_cache_fp8", "gather_cache_fp8", "paged_decode_fp8",
    "qk_norm_rope_reshape_and_cache", "paged_tree_attention",
    "paged_tree_attention_workspace_size",
    "update_block_tables", "update_page_bounds", "select_pages", "paged_sparse_attention",
    "DEVERR_BLOCK_ID", "DEVERR_SLOT", "DEVERR_SEQLEN", "DEVERR_TIMEOUT", "DEVERR_POSITION",
    "DEVERR_NO_BLOCKS", "EXPORTED_SYMBOLS",
]

PKV_F32 = 0
PKV_BF16 = 1
PKV_E4M3 = 2
DEVERR_BLOCK_ID = 1
DEVERR_SLOT = 2
DEVERR_SEQLEN = 4
DEVERR_TIMEOUT = 8
DEVERR_POSITION = 16
DEVERR_NO_BLOCKS = 32

EXPORTED_SYMBOLS = (
    "pkv_status_string", "pkv_version", "pkv_reshape_and_cache",
    "pkv_paged_decode_workspace_size", "pkv_paged_decode",
    "pkv_varlen_prefill_workspace_size", "pkv_varlen_prefill",
    "pkv_varlen_prefill_contiguous", "pkv_rope_cos_sin_table", "pkv_rope_reshape_and_cache",
    "pkv_minference_sizes", "pkv_minference_workspace_size", "pkv_minference_prefill",
    "pkv_paged_decode_noalloc", "pkv_get_device_error", "pkv_selftest_bounded_wait",
    "pkv_reshape_and_cache_fp8", "pkv_gather_cache_fp8", "pkv_paged_decode_fp8",
    "pkv_qk_norm_rope_reshape_and_cache", "pkv_paged_tree_attention_workspace_size",
    "pkv_paged_tree_attention",
    "pkv_update_block_tables", "pkv_update_page_bounds", "pkv_select_pages",
    "pkv_paged_sparse_attention",
)


class PkvError(RuntimeError):
    """A libpkv call returned a non-OK status."""

    def __init__(self, fn: str, status: int, name: str):
        super().__init__(f"{fn} failed: {name} ({status})")
        self.status = status
        self.status_name = name


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int64), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("layout", ctypes.c_int32)]


LAYOUTS = {"NHD": 0, "HND": 1}


_lib = None
_lock = threading.Lock()


def build(force: bool = False) -> str:
    """Compile libpkv.so for sm_103a (in-tree)."""
    return _build_lib(force=force)


def load_library(path: Optional[str] = None):
    """Load libpkv.so (building it first if it is absent) and declare the ABI."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            p = _build_lib()
        lib = ctypes.CDLL(p)
        P, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                                ctypes.c_size_t)
        lib.pkv_status_string.argtypes = [i32]
        lib.pkv_status_string.restype = ctypes.c_char_p
        lib.pkv_version.argtypes = []
        lib.pkv_version.restype = i32
        lib.pkv_reshape_and_cache.argtypes = [P, P, P, P, P, i64, CacheDesc, P, P]
        lib.pkv_reshape_and_cache.restype = i32
        lib.pkv_paged_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.pkv_paged_decode_workspace_size.restype = sz
        lib.pkv_paged_decode.argtypes = [P, P, P, P, CacheDesc, P, i32, P, i32, P, P, i32, i32,
                                         i32, f32, i32, P, P, sz, P, P]
        lib.pkv_paged_decode.restype = i32
        lib.pkv_varlen_prefill_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        lib.pkv_varlen_prefill_workspace_size.restype = sz
        lib.pkv_varlen_prefill.argtypes = [P, P, P, P, CacheDesc, P, i32, P, P, i32, i32, i32, P,
                                           P, i32, i32, i32, i32, f32, P, P, sz, i32, P, P]
        lib.pkv_varlen_prefill.restype = i32
        lib.pkv_varlen_prefill_contiguous.argtypes = [P, P, P, P, i32, i32, i32, i32, P, P, i32,
                                                      i32, i32, P, P, i32, i32, i32, i32, f32, P,
                                                      P, sz, P, P]
        lib.pkv_varlen_prefill_contiguous.restype = i32
        f64 = ctypes.c_double
        lib.pkv_rope_cos_sin_table.argtypes = [P, i32, i32, f64, f64, f64, P]
        lib.pkv_rope_cos_sin_table.restype = i32
        lib.pkv_rope_reshape_and_cache.argtypes = [P, P, P, P, P, P, P, i64, i32, CacheDesc, P,
                                                   i32, i32, i32, P, P]
        lib.pkv_rope_reshape_and_cache.restype = i32
        lib.pkv_minference_sizes.argtypes = [i32, i32, i32, f64, i32, i32, P, P]
        lib.pkv_minference_sizes.restype = i32
        lib.pkv_minference_workspace_size.argtypes = [i32, i32, i32, i32, i32, f64, i32, i32]
        lib.pkv_minference_workspace_size.restype = sz
        lib.pkv_minference_prefill.argtypes = [P, P, P, P, i32, i32, i32, i32, i32, i32, i32, f64,
                                               i32, i32, f32, P, P, P, sz, P, P]
        lib.pkv_minference_prefill.restype = i32
        lib.pkv_paged_decode_noalloc.argtypes = [P, P, P, P, CacheDesc, P, i32, P, i32, P, i32,
                                                 i32, i32, f32, i32, P, P, P]
        lib.pkv_paged_decode_noalloc.restype = i32
        lib.pkv_get_device_error.argtypes = [P, P, i32, P]
        lib.pkv_get_device_error.restype = i32
        lib.pkv_selftest_bounded_wait.argtypes = [P, P]
        lib.pkv_selftest_bounded_wait.restype = i32
        lib.pkv_reshape_and_cache_fp8.argtypes = [P, P, i64, i64, i32, P, P, P, P, P, i64,
                                                  CacheDesc, P, P]
        lib.pkv_reshape_and_cache_fp8.restype = i32
        lib.pkv_gather_cache_fp8.argtypes = [P, P, P, P, P, P, CacheDesc, P, i32, P, i32, i64, P,
                                             P]
        lib.pkv_gather_cache_fp8.restype = i32
        lib.pkv_paged_decode_fp8.argtypes = [P, P, P, P, P, P, CacheDesc, P, i32, P, i32, P, P,
                                             i32, i32, i32, f32, i32, P, P, sz, P, P]
        lib.pkv_paged_decode_fp8.restype = i32
        lib.pkv_qk_norm_rope_reshape_and_cache.argtypes = [
            P, P, P, i64, i64, i64, i32, P, P, i64, i64, P, P, P, P, P, P, i64, i32, CacheDesc, P,
            P, i32, f32, P, i32, i32, i32, P, P]
        lib.pkv_qk_norm_rope_reshape_and_cache.restype = i32
        lib.pkv_paged_tree_attention_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        lib.pkv_paged_tree_attention_workspace_size.restype = sz
        lib.pkv_paged_tree_attention.argtypes = [
            P, P, P, P, P, P, CacheDesc, P, i32, P, P, i32, i32, i32, P, i32, P, P, P, i32, i32,
            i32, f32, i32, P, P, sz, P, P]
        lib.pkv_paged_tree_attention.restype = i32
        lib.pkv_update_block_tables.argtypes = [P, i32, P, P, i32, P, i64, P, i32, P, P, i32, P, P,
                                                P, P]
        lib.pkv_update_block_tables.restype = i32
        lib.pkv_update_page_bounds.argtypes = [P, P, CacheDesc, P, P, P, i64, P, P]
        lib.pkv_update_page_bounds.restype = i32
        lib.pkv_select_pages.argtypes = [P, i32, P, P, P, i64, i32, i32, i32, P, i32, P, i32, P, i32,
                                         i32, i32, i32, i32, P, P]
        lib.pkv_select_pages.restype = i32
        lib.pkv_paged_sparse_attention.argtypes = [
            P, P, P, P, P, P, CacheDesc, P, i32, P, P, i32, i32, P, i32, P, i32, f32, P, P, P]
        lib.pkv_paged_sparse_attention.restype = i32
        _lib = lib
        return lib


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _check(fn: str, status: int):
    if status != 0:
        name = load_library().pkv_status_string(status).decode()
        raise PkvError(fn, status, name)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_handle(stream) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _dtype_code(dtype) -> int:
    torch = _torch()
    if dtype == torch.float32:
        return PKV_F32
    if dtype == torch.bfloat16:
        return PKV_BF16
    raise TypeError(f"unsupported dtype {dtype}: use torch.bfloat16 or torch.float32")


def _require(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def _cuda_contig(name, t, dtype=None, ndim=None):
    _require(t.is_cuda, f"{name} must be a CUDA tensor")
    _require(t.is_contiguous(), f"{name} must be contiguous")
    if dtype is not None:
        _require(t.dtype == dtype, f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None:
        _require(t.dim() == ndim, f"{name} must have {ndim} dims, got {t.dim()}")


def _pool_dims(k_cache, layout: str):
    """(num_blocks, block_size, num_kv_heads, head_dim) of a pool: NHD pools
    are [num_blocks, block_size, Hkv, D], HND pools [num_blocks, Hkv,
    block_size, D]."""
    _require(layout in LAYOUTS, f"layout must be one of {sorted(LAYOUTS)}")
    nb, a, b, d = k_cache.shape
    return (nb, a, b, d) if layout == "NHD" else (nb, b, a, d)


def _cache_desc(k_cache, v_cache, layout: str = "NHD") -> CacheDesc:
    _cuda_contig("k_cache", k_cache, ndim=4)
    _cuda_contig("v_cache", v_cache, ndim=4)
    _require(k_cache.shape == v_cache.shape and k_cache.dtype == v_cache.dtype,
             "k_cache and v_cache must have the same shape and dtype")
    nb, bs, hkv, d = _pool_dims(k_cache, layout)
    return CacheDesc(nb, bs, hkv, d, _dtype_code(k_cache.dtype), LAYOUTS[layout])


def _head_vector(name, t, Hq):
    if t is not None:
        _cuda_contig(name, t, _torch().float32, 1)
        _require(t.shape[0] == Hq, f"{name} must have num_qo_heads entries")


def paged_decode_workspace_size(batch: int, num_qo_heads: int, head_dim: int, max_seqlen: int,
                                partition_size: int = 512, window_left: int = -1) -> int:
    return int(load_library().pkv_paged_decode_workspace_size(
        batch, num_qo_heads, head_dim, max_seqlen, partition_size, window_left))


def varlen_prefill_workspace_size(batch: int, num_qo_heads: int, num_kv_heads: int,
                                  total_q: int, max_seqlen_q: int) -> int:
    return int(load_library().pkv_varlen_prefill_workspace_size(
        batch, num_qo_heads, num_kv_heads, total_q, max_seqlen_q))


def _workspace(nbytes: int, device, workspace):
    torch = _torch()
    if workspace is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    _cuda_contig("workspace", workspace)
    _require(workspace.numel() * workspace.element_size() >= nbytes,
             f"workspace too small: need {nbytes} bytes")
    return workspace


# ---------------------------------------------------------------------------
# public operations
# ---------------------------------------------------------------------------

def reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, dev_error=None,
                      stream=None, layout: str = "NHD") -> None:
    """k_cache/v_cache flat slot slot_mapping[t] <- key/value[t] (in place).

    key, value: [T, Hkv, D] contiguous, dtype of the cache; slot_mapping: [T]
    int64, negative = skip.  dev_error: optional int32 device tensor that
    receives PKV_DEVERR_SLOT for slots outside the pool.
    """
    torch = _torch()
    desc = _cache_desc(k_cache, v_cache, layout)
    _cuda_contig("key", key, k_cache.dtype, 3)
    _cuda_contig("value", value, k_cache.dtype, 3)
    _cuda_contig("slot_mapping", slot_mapping, torch.int64, 1)
    _require(key.shape == value.shape and key.shape[1:] == (desc.num_kv_heads, desc.head_dim),
             "key/value must be [T, num_kv_heads, head_dim] matching the cache")
    _require(slot_mapping.shape[0] == key.shape[0], "slot_mapping must have T entries")
    st = load_library().pkv_reshape_and_cache(
        _ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping),
        key.shape[0], desc, _ptr(dev_error), _stream_handle(stream))
    _check("pkv_reshape_and_cache", st)


def get_device_error(dev_error, clear: bool = False, stream=None, raise_on_error: bool = False):
    """The PKV_DEVERR_* bits the calls so far ORed into ``dev_error`` (an int32
    device tensor of one element).  Waits for ``stream`` (the current one by
    default); with ``clear`` the word is then zeroed on that stream.  With
    ``raise_on_error`` a set bit raises PkvError (PKV_ERR_OUT_OF_RANGE, or
    PKV_ERR_TIMEOUT for a pipeline wait that gave up)."""
    torch = _torch()
    _cuda_contig("dev_error", dev_error, torch.int32, 1)
    bits = ctypes.c_int32(0)
    st = load_library().pkv_get_device_error(_ptr(dev_error), ctypes.addressof(bits),
                                             int(bool(clear)), _stream_handle(stream))
    if st != 0 and (raise_on_error or st not in (5, 6)):
        _check("pkv_get_device_error", st)
    return int(bits.value)


def selftest_bounded_wait(dev_error, stream=None):
    """Run one bounded pipeline wait that nothing completes on ``stream``: it
    gives up by itself and ORs DEVERR_TIMEOUT into ``dev_error`` (an int32
    device tensor of one element); see get_device_error."""
    _cuda_contig("dev_error", dev_error, _torch().int32, 1)
    _check("pkv_selftest_bounded_wait",
           load_library().pkv_selftest_bounded_wait(_ptr(dev_error), _stream_handle(stream)))


def rope_cos_sin_table(max_position: int, rotary_dim: int, base: float = 10000.0,
                       position_scale: float = 1.0, ntk_alpha: float = 1.0, device=None,
                       stream=None):
    """The rotary table [max_position, rotary_dim // 2, 2] float32 of
    (cos, sin) of (pos / position_scale) * b^(-2i / rotary_dim), computed in
    fp64 on the GPU, b = base * ntk_alpha^(rotary_dim / (rotary_dim - 2)).
    position_scale is the linear scaling factor, ntk_alpha the NTK-aware
    context stretch (1: none)."""
    torch = _torch()
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    tab = torch.empty(max(max_position, 0), rotary_dim // 2, 2, dtype=torch.float32, device=dev)
    st = load_library().pkv_rope_cos_sin_table(_ptr(tab) if tab.numel() else None,
                                               int(max_position), int(rotary_dim), float(base),
                                               float(position_scale), float(ntk_alpha),
                                               _stream_handle(stream))
    _check("pkv_rope_cos_sin_table", st)
    return tab


def rope_reshape_and_cache(query, key, value, k_cache, v_cache, positions, slot_mapping,
                           cos_sin, rotary_dim: Optional[int] = None, is_neox_style: bool = True,
                           dev_error=None, stream=None, layout: str = "NHD") -> None:
    """Rotate query [T, Hq, D] and key [T, Hkv, D] in place by positions [T]
    (int64) using the table cos_sin ([max_position, rotary_dim // 2, 2]), then
    write the rotated key and the value to the pools at slot_mapping [T]
    (int64; negative = not cached).  query may be None."""
    torch = _torch()
    desc = _cache_desc(k_cache, v_cache, layout)
    _cuda_contig("key", key, k_cache.dtype, 3)
    _cuda_contig("value", value, k_cache.dtype, 3)
    _cuda_contig("positions", positions, torch.int64, 1)
    _cuda_contig("slot_mapping", slot_mapping, torch.int64, 1)
    _cuda_contig("cos_sin", cos_sin, torch.float32, 3)
    T = key.shape[0]
    _require(key.shape == value.shape and key.shape[1:] == (desc.num_kv_heads, desc.head_dim),
             "key/value must be [T, num_kv_heads, head_dim] matching the cache")
    _require(positions.shape[0] == T and slot_mapping.shape[0] == T,
             "positions and slot_mapping must have T entries")
    rd = int(rotary_dim) if rotary_dim is not None else 2 * cos_sin.shape[1]
    _require(cos_sin.shape[1] * 2 == rd and cos_sin.shape[2] == 2,
             "cos_sin must be [max_position, rotary_dim // 2, 2]")
    Hq = 0
    if query is not None:
        _cuda_contig("query", query, k_cache.dtype, 3)
        _require(query.shape[0] == T and query.shape[2] == key.shape[2],
                 "query must be [T, num_qo_heads, head_dim]")
        Hq = query.shape[1]
    st = load_library().pkv_rope_reshape_and_cache(
        _ptr(query), _ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache), _ptr(positions),
        _ptr(slot_mapping), T, Hq, desc, _ptr(cos_sin), cos_sin.shape[0], rd,
        int(bool(is_neox_style)), _ptr(dev_error), _stream_handle(stream))
    _check("pkv_rope_reshape_and_cache", st)


def _decode_args(q, k_cache, v_cache, block_table, cache_seqlens, sink, out, lse, layout):
    """Checks shared by the two decode entry points; returns (cache desc, out)."""
    torch = _torch()
    desc = _cache_desc(k_cache, v_cache, layout)
    _cuda_contig("q", q, k_cache.dtype, 3)
    _cuda_contig("block_table", block_table, torch.int32, 2)
    _cuda_contig("cache_seqlens", cache_seqlens, torch.int32, 1)
    B, Hq, D = q.shape
    _require(D == desc.head_dim, "head_dim of q and cache differ")
    _require(block_table.shape[0] == B and cache_seqlens.shape[0] == B,
             "block_table / cache_seqlens batch mismatch")
    if sink is not None:
        _cuda_contig("sink", sink, torch.float32, 1)
        _require(sink.shape[0] == Hq, "sink must have num_qo_heads entries")
    if out is None:
        out = torch.empty_like(q)
    else:
        _cuda_contig("out", out, q.dtype, 3)
        _require(out.shape == q.shape, "out must be shaped like q")
    if lse is not None:
        _cuda_contig("lse", lse, torch.float32, 2)
        _require(tuple(lse.shape) == (B, Hq), "lse must be [B, Hq]")
    return desc, out


def paged_decode(q, k_cache, v_cache, block_table, cache_seqlens, max_seqlen: int,
                 sink=None, window_left: int = -1, sm_scale: Optional[float] = None,
                 partition_size: int = 512, out=None, lse=None, workspace=None,
                 dev_error=None, stream=None, alibi_slopes=None, layout: str = "NHD"):
    """Single-token decode over the paged pools; returns out [B, Hq, D].

    q: [B, Hq, D] (dtype of the cache); block_table: [B, max_blocks] int32;
    cache_seqlens: [B] int32, the attended length (query at position L-1);
    max_seqlen: host int >= max(cache_seqlens); sink: [Hq] float32 or None;
    lse: optional [B, Hq] float32 output (natural log, sink included);
    alibi_slopes: [Hq] float32 or None (bias slope * (j - (L - 1)));
    layout: "NHD" pools [num_blocks, block_size, Hkv, D] or "HND" pools
    [num_blocks, Hkv, block_size, D].
    """
    torch = _torch()
    desc, out = _decode_args(q, k_cache, v_cache, block_table, cache_seqlens, sink, out, lse,
                             layout)
    B, Hq, D = q.shape
    _head_vector("alibi_slopes", alibi_slopes, Hq)
    scale = float(sm_scale) if sm_scale is not None else D ** -0.5
    need = paged_decode_workspace_size(B, Hq, D, max_seqlen, partition_size, window_left)
    ws = _workspace(need, q.device, workspace)
    st = load_library().pkv_paged_decode(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), desc, _ptr(block_table),
        block_table.shape[1], _ptr(cache_seqlens), int(max_seqlen), _ptr(sink),
        _ptr(alibi_slopes), B, Hq, int(window_left), scale, int(partition_size), _ptr(lse),
        _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_error), _stream_handle(stream))
    _check("pkv_paged_decode", st)
    return out


def varlen_prefill(q, k_cache, v_cache, block_table, cu_seq_lens_q, cu_seq_lens_k,
                   max_seqlen_q: int, max_seqlen_k: int, sink=None, causal: bool = True,
                   window_left: int = -1, sm_scale: Optional[float] = None, out=None, lse=None,
                   workspace=None, dev_error=None, stream=None, alibi_slopes=None,
                   layout: str = "NHD", max_ctas: int = 0):
    """Varlen / chunk prefill over the paged pools; returns out [total_q, Hq, D].

    q: [total_q, Hq, D] bf16; cu_seq_lens_q / cu_seq_lens_k: [B+1] int32;
    max_seqlen_q / max_seqlen_k: host ints; request r's queries sit at the end
    of its kv_len keys.  causal=False drops the j <= position bound (a window
    still bounds keys from below).  max_ctas: at most this many attention
    CTAs (one SM each) at once, 0 = one per SM; fewer leave SMs free for
    work on another stream.
    """
    torch = _torch()
    desc = _cache_desc(k_cache, v_cache, layout)
    _cuda_contig("q", q, k_cache.dtype, 3)
    _cuda_contig("block_table", block_table, torch.int32, 2)
    _cuda_contig("cu_seq_lens_q", cu_seq_lens_q, torch.int32, 1)
    _cuda_contig("cu_seq_lens_k", cu_seq_lens_k, torch.int32, 1)
    total_q, Hq, D = q.shape
    B = cu_seq_lens_q.shape[0] - 1
    _require(cu_seq_lens_k.shape[0] == B + 1, "cu_seq_lens_q/k lengths differ")
    _require(block_table.shape[0] == B, "block_table must have one row per request")
    if sink is not None:
        _cuda_contig("sink", sink, torch.float32, 1)
        _require(sink.shape[0] == Hq, "sink must have num_qo_heads entries")
    _head_vector("alibi_slopes", alibi_slopes, Hq)
    if out is None:
        out = torch.empty_like(q)
    else:
        _cuda_contig("out", out, q.dtype, 3)
        _require(out.shape == q.shape, "out must be shaped like q")
    if lse is not None:
        _cuda_contig("lse", lse, torch.float32, 2)
        _require(tuple(lse.shape) == (total_q, Hq), "lse must be [total_q, Hq]")
    scale = float(sm_scale) if sm_scale is not None else D ** -0.5
    need = varlen_prefill_workspace_size(B, Hq, desc.num_kv_heads, total_q, max_seqlen_q)
    ws = _workspace(need, q.device, workspace)
    st = load_library().pkv_varlen_prefill(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), desc, _ptr(block_table),
        block_table.shape[1], _ptr(cu_seq_lens_q), _ptr(cu_seq_lens_k), int(max_seqlen_q),
        int(max_seqlen_k), int(total_q), _ptr(sink), _ptr(alibi_slopes), B, Hq,
        int(bool(causal)), int(window_left), scale, _ptr(lse), _ptr(ws),
        ws.numel() * ws.element_size(), int(max_ctas), _ptr(dev_error), _stream_handle(stream))
    _check("pkv_varlen_prefill", st)
    return out


def varlen_prefill_contiguous(q, k, v, cu_seq_lens_q, cu_seq_lens_k, max_seqlen_q: int,
                              max_seqlen_k: int, sink=None, causal: bool = True,
                              window_left: int = -1, sm_scale: Optional[float] = None, out=None,
                              lse=None, workspace=None, dev_error=None, stream=None,
                              alibi_slopes=None):
    """Varlen prefill with contiguous keys: request r's keys and values are
    rows cu_seq_lens_k[r] .. cu_seq_lens_k[r+1]-1 of k and v ([total_k, Hkv, D]
    bf16).  Otherwise as varlen_prefill; returns out [total_q, Hq, D]."""
    torch = _torch()
    _cuda_contig("q", q, ndim=3)
    _cuda_contig("k", k, q.dtype, 3)
    _cuda_contig("v", v, q.dtype, 3)
    _cuda_contig("cu_seq_lens_q", cu_seq_lens_q, torch.int32, 1)
    _cuda_contig("cu_seq_lens_k", cu_seq_lens_k, torch.int32, 1)
    _require(k.shape == v.shape, "k and v must have the same shape")
    total_q, Hq, D = q.shape
    total_k, Hkv, Dk = k.shape
    _require(Dk == D, "head_dim of q and k differ")
    B = cu_seq_lens_q.shape[0] - 1
    _require(cu_seq_lens_k.shape[0] == B + 1, "cu_seq_lens_q/k lengths differ")
    if sink is not None:
        _cuda_contig("sink", sink, torch.float32, 1)
        _require(sink.shape[0] == Hq, "sink must have num_qo_heads entries")
    _head_vector("alibi_slopes", alibi_slopes, Hq)
    if out is None:
        out = torch.empty_like(q)
    else:
        _cuda_contig("out", out, q.dtype, 3)
        _require(out.shape == q.shape, "out must be shaped like q")
    if lse is not None:
        _cuda_contig("lse", lse, torch.float32, 2)
        _require(tuple(lse.shape) == (total_q, Hq), "lse must be [total_q, Hq]")
    scale = float(sm_scale) if sm_scale is not None else D ** -0.5
    need = varlen_prefill_workspace_size(B, Hq, Hkv, total_q, max_seqlen_q)
    ws = _workspace(need, q.device, workspace)
    st = load_library().pkv_varlen_prefill_contiguous(
        _ptr(out), _ptr(q), _ptr(k) if total_k else None, _ptr(v) if total_k else None,
        int(total_k), Hkv, D, _dtype_code(q.dtype), _ptr(cu_seq_lens_q), _ptr(cu_seq_lens_k),
        int(max_seqlen_q), int(max_seqlen_k), int(total_q), _ptr(sink), _ptr(alibi_slopes), B,
        Hq, int(bool(causal)), int(window_left), scale, _ptr(lse), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(dev_error), _stream_handle(stream))
    _check("pkv_varlen_prefill_contiguous", st)
    return out


def minference_sizes(seq_len: int, vertical_size: int = 1000, slash_size: int = 6096,
                     adaptive_budget: Optional[float] = 0.3, num_sink_tokens: int = 30,
                     num_recent_diags: int = 100):
    """(nv, ns): how many vertical columns and slash diagonals are kept."""
    nv, ns = ctypes.c_int(), ctypes.c_int()
    st = load_library().pkv_minference_sizes(
        int(seq_len), int(vertical_size), int(slash_size),
        float(adaptive_budget) if adaptive_budget is not None else 0.0, int(num_sink_tokens),
        int(num_recent_diags), ctypes.byref(nv), ctypes.byref(ns))
    _check("pkv_minference_sizes", st)
    return nv.value, ns.value


def lib_minference_workspace(seq_len: int, num_qo_heads: int, num_kv_heads: int,
                             vertical_size: int = 1000, slash_size: int = 6096,
                             adaptive_budget: Optional[float] = 0.3, num_sink_tokens: int = 30,
                             num_recent_diags: int = 100) -> int:
    """Workspace bytes minference_prefill needs."""
    return int(load_library().pkv_minference_workspace_size(
        int(seq_len), int(num_qo_heads), int(num_kv_heads), int(vertical_size), int(slash_size),
        float(adaptive_budget) if adaptive_budget is not None else 0.0, int(num_sink_tokens),
        int(num_recent_diags)))


def minference_prefill(q, k, v, vertical_size: int = 1000, slash_size: int = 6096,
                       adaptive_budget: Optional[float] = 0.3, num_sink_tokens: int = 30,
                       num_recent_diags: int = 100, sm_scale: Optional[float] = None, out=None,
                       return_pattern: bool = False, workspace=None, dev_error=None,
                       stream=None):
    """MInference vertical + slash sparse prefill of one sequence: q [S, Hq, D],
    k, v [S, Hkv, D] bf16.  Returns out [S, Hq, D] (and, with
    return_pattern, the kept vertical [Hq, nv] and slash [Hq, ns] indices)."""
    torch = _torch()
    _cuda_contig("q", q, torch.bfloat16, 3)
    _cuda_contig("k", k, torch.bfloat16, 3)
    _cuda_contig("v", v, torch.bfloat16, 3)
    S, Hq, D = q.shape
    _require(k.shape == v.shape and k.shape[0] == S and k.shape[2] == D,
             "k and v must be [S, num_kv_heads, head_dim] like q")
    Hkv = k.shape[1]
    budget = float(adaptive_budget) if adaptive_budget is not None else 0.0
    nv, ns = minference_sizes(S, vertical_size, slash_size, adaptive_budget, num_sink_tokens,
                              num_recent_diags)
    if out is None:
        out = torch.empty_like(q)
    else:
        _cuda_contig("out", out, q.dtype, 3)
        _require(out.shape == q.shape, "out must be shaped like q")
    vi = torch.empty(Hq, nv, dtype=torch.int32, device=q.device) if return_pattern else None
    si = torch.empty(Hq, ns, dtype=torch.int32, device=q.device) if return_pattern else None
    need = int(load_library().pkv_minference_workspace_size(
        S, Hq, Hkv, int(vertical_size), int(slash_size), budget, int(num_sink_tokens),
        int(num_recent_diags)))
    ws = _workspace(need, q.device, workspace)
    scale = float(sm_scale) if sm_scale is not None else D ** -0.5
    st = load_library().pkv_minference_prefill(
        _ptr(out), _ptr(q), _ptr(k), _ptr(v), S, Hq, Hkv, D, PKV_BF16, int(vertical_size),
        int(slash_size), budget, int(num_sink_tokens), int(num_recent_diags), scale, _ptr(vi),
        _ptr(si), _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_error),
        _stream_handle(stream))
    _check("pkv_minference_prefill", st)
    return (out, vi, si) if return_pattern else out


def paged_decode_noalloc(q, k_cache, v_cache, block_table, cache_seqlens, max_seqlen: int,
                         sink=None, window_left: int = -1, sm_scale: Optional[float] = None,
                         partition_size: int = 512, out=None, lse=None, dev_error=None,
                         stream=None, layout: str = "NHD"):
    """paged_decode without a caller workspace, for callers that cannot
    allocate device memory at the call site.  The library's fixed device
    scratch array (PKV_NOALLOC_DECODE_SCRATCH_BYTES, 32 MiB) replaces the
    workspace; problems that need more are rejected (PkvError
    PKV_ERR_WORKSPACE).  Calls share the array: do not overlap them on the
    GPU.  The first call on a device should come before any stream capture.
    ``out`` (and ``lse``) should be preallocated when the caller must not
    allocate at all."""
    desc, out = _decode_args(q, k_cache, v_cache, block_table, cache_seqlens, sink, out, lse,
                             layout)
    B, Hq, D = q.shape
    scale = float(sm_scale) if sm_scale is not None else D ** -0.5
    st = load_library().pkv_paged_decode_noalloc(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), desc, _ptr(block_table),
        block_table.shape[1], _ptr(cache_seqlens), int(max_seqlen), _ptr(sink), B, Hq,
        int(window_left), scale, int(partition_size), _ptr(lse), _ptr(dev_error),
        _stream_handle(stream))
    _check("pkv_paged_decode_noalloc", st)
    return out


# ---------------------------------------------------------------------------
# the 8-bit cache, the q/k norm and the attention of drafted tokens.  These
# calls are short on the GPU in a decode step, so a call first asks whether
# its arguments are of the usual kind in one expression; only if not are they
# checked one by one, which finds the reason or lets them pass.
# ---------------------------------------------------------------------------

def _cuda_index(name, t) -> int:
    """The index of the CUDA device ``t`` lives on."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _arg(name, t, dtype, ndim: int, dev: int):
    """A contiguous tensor of ``dtype`` with ``ndim`` dims on device ``dev``."""
    if (t.dtype is dtype and t.dim() == ndim and t.get_device() == dev and t.is_contiguous()):
        return
    if t.get_device() < 0 <= dev:
        raise ValueError(f"{name} must be a CUDA tensor")
    _require(t.get_device() == dev, f"{name} must be on the same device as the other tensors")
    _require(t.dtype is dtype, f"{name} must be {dtype}, got {t.dtype}")
    _require(t.dim() == ndim, f"{name} must have {ndim} dims, got {t.dim()}")
    raise ValueError(f"{name} must be contiguous")


def _arg_shape(name, t, dtype, shape, dev: int):
    """A contiguous tensor of that shape."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return
    _arg(name, t, dtype, len(shape), dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _arg_vector(name, t, dtype, n: int, dev: int):
    """A contiguous vector of n entries."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == (n,) and t.is_contiguous():
        return
    _arg_shape(name, t, dtype, (n,), dev)


_WIDEST = 2 ** 31 - 1  # a window that holds every key (lengths are at most 2^30)


def _int32(name, value) -> int:
    """A host integer that the library takes in 32 bits (ctypes would cut it off)."""
    value = int(value)
    if -2 ** 31 <= value < 2 ** 31:
        return value
    raise ValueError(f"{name} must be within 32 bits, got {value}")


def _error_word(dev_error, dev: int):
    """The address of the caller's error word, or None."""
    if dev_error is None:
        return None
    _arg("dev_error", dev_error, _torch().int32, 1, dev)
    _require(dev_error.shape[0] >= 1, "dev_error must have one element")
    return dev_error.data_ptr()


_descs = {}         # what a pool's shape says (building a CacheDesc costs as much as a check)
_scale_shapes = {}  # and the shape of the scales that go with it


def _desc(*fields) -> CacheDesc:
    """The CacheDesc of a shape."""
    d = _descs.get(fields)
    if d is None:
        if len(_descs) > 4096:
            _descs.clear()
        d = _descs[fields] = CacheDesc(*fields)
    return d


def _fp8_pools(k_cache, v_cache, k_scale, v_scale, layout: str, dev: int) -> CacheDesc:
    """Checks the pools and scales of the 8-bit cache."""
    ty = _types()
    if (k_scale is not None and v_scale is not None
            and k_cache.dtype is ty.e4m3 and v_cache.dtype is ty.e4m3
            and k_scale.dtype is ty.u8 and v_scale.dtype is ty.u8
            and k_cache.get_device() == v_cache.get_device() == k_scale.get_device()
            == v_scale.get_device() == dev
            and k_cache.is_contiguous() and v_cache.is_contiguous()
            and k_scale.is_contiguous() and v_scale.is_contiguous()):
        shape = k_cache.shape
        key = (shape, layout)
        d = _descs.get(key)
        if d is not None and v_cache.shape == shape and \
                k_scale.shape == v_scale.shape == _scale_shapes.get(key):
            return d
    _require(k_scale is not None, "k_scale is needed for an 8-bit cache")
    _require(v_scale is not None, "v_scale is needed for an 8-bit cache")
    d = _pools(k_cache, v_cache, k_scale, v_scale, None, layout, dev)
    if len(_scale_shapes) > 4096:
        _descs.clear()
        _scale_shapes.clear()
    _scale_shapes[(k_cache.shape, layout)] = k_scale.shape
    _descs[(k_cache.shape, layout)] = d
    return d


def _pools(k_cache, v_cache, k_scale, v_scale, dtype, layout: str, dev: int) -> CacheDesc:
    """Checks two pools: of ``dtype`` without scales, else of the 8-bit cache."""
    fp8 = k_scale is not None or v_scale is not None
    shape = k_cache.shape
    key = (shape, layout, dtype)
    if (not fp8 and k_cache.dtype is dtype and v_cache.dtype is dtype and v_cache.shape == shape
            and k_cache.get_device() == v_cache.get_device() == dev
            and k_cache.is_contiguous() and v_cache.is_contiguous()):
        d = _descs.get(key)
        if d is not None:
            return d
    torch = _torch()
    dt = torch.float8_e4m3fn if fp8 else dtype
    _arg("k_cache", k_cache, dt, 4, dev)
    _arg("v_cache", v_cache, dt, 4, dev)
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(LAYOUTS)}")
    nb, bs, hkv, d = shape
    if layout == "HND":
        bs, hkv = hkv, bs
    if not fp8:
        desc = _descs[key] = _desc(nb, bs, hkv, d, _dtype_code(dt), LAYOUTS[layout])
        return desc
    want = (nb, hkv, bs)
    for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
        if s is None:
            raise ValueError(f"{name} is needed for an 8-bit cache")
        _arg(name, s, torch.uint8, 3, dev)
        if s.shape != want:
            raise ValueError(f"{name} must be [num_blocks, num_kv_heads, block_size]")
    return _desc(nb, bs, hkv, d, PKV_E4M3, LAYOUTS[layout])


def _token_rows(name, t, dtype, tokens: int, heads: int, head_dim: int, dev: int) -> int:
    """Checks [tokens, heads, head_dim] rows whose heads are contiguous; returns
    the elements between tokens (a slice of a fused projection keeps its own)."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == (tokens, heads, head_dim):
        if t.is_contiguous():
            return heads * head_dim
        token, head, one = t.stride()
        if one == 1 and (heads == 1 or head == head_dim):
            return token if tokens > 1 else heads * head_dim
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    _require(t.get_device() == dev, f"{name} must be on the same device as the other tensors")
    _require(t.dtype is dtype, f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be [{tokens}, {heads}, {head_dim}], got {list(t.shape)}")


def _rows_meet(tokens: int, a: int, step_a: int, len_a: int, b: int, step_b: int,
               len_b: int) -> bool:
    """Whether one of ``tokens`` rows of len_a bytes at a, a + step_a, .. shares a
    byte with one of len_b at b, b + step_b, .."""
    if a >= b + (tokens - 1) * step_b + len_b or b >= a + (tokens - 1) * step_a + len_a or \
            not (len_a and len_b):
        return False
    if tokens <= 1 or step_a < len_a or step_b < len_b:
        return tokens == 1  # (shorter steps: the library refuses them)
    if step_a == step_b:    # slices of one projection: the rows lie alike in each step
        d = (b - a) % step_a
        return d < len_a or step_a - d < len_b
    i = j = 0
    while i < tokens and j < tokens:
        at_a, at_b = a + i * step_a, b + j * step_b
        if at_a + len_a <= at_b:
            i += 1
        elif at_b + len_b <= at_a:
            j += 1
        else:
            return True
    return False


_SAME_ROWS = (("query_out", "query"), ("key_out", "key"), ("key_out", "value"))


def _refuse_overlap(tokens: int, outs, ins) -> None:
    """Outputs (name, address, bytes between tokens, bytes of a row) overlap neither one
    another nor an input, but that of their own name as that input itself, and key_out
    value's rows likewise (a head's k and v are read before either is written)."""
    if _rows_meet(tokens, *outs[0][1:], *outs[1][1:]):
        raise ValueError(f"{outs[1][0]} must not overlap {outs[0][0]}")
    for out in outs:
        for row in ins:
            if out[1:] == row[1:] and (out[0], row[0]) in _SAME_ROWS:
                continue  # in place
            if _rows_meet(tokens, *out[1:], *row[1:]):
                raise ValueError(f"{out[0]} must not overlap {row[0]}")


class _Types:
    """torch and the dtypes the checks compare with, looked up once."""
    torch = bf16 = f32 = i32 = i64 = u8 = i8 = e4m3 = None
    codes = {}                  # pkv_dtype of the rows' dtypes
    device = raw_stream = None  # the current device, and a device's current stream handle


def _types():
    if _Types.torch is None:
        import torch
        _Types.bf16, _Types.f32, _Types.i32 = torch.bfloat16, torch.float32, torch.int32
        _Types.i64, _Types.u8, _Types.e4m3 = torch.int64, torch.uint8, torch.float8_e4m3fn
        _Types.i8 = torch.int8
        _Types.codes = {torch.bfloat16: PKV_BF16, torch.float32: PKV_F32}
        _Types.device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _Types.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        _Types.torch = torch
    return _Types


def _on_stream(dev: int, stream, call):
    """call(stream handle), with the device of the tensors current, and with a
    ``stream`` that stream, so that what the call allocates belongs to the
    stream its kernels run on."""
    if dev < 0:
        return call(_stream_handle(stream))
    t = _types()
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError("stream must be of the tensors' device")
        with t.torch.cuda.stream(stream):
            return call(stream.cuda_stream)
    if t.device() != dev:
        with t.torch.cuda.device(dev):
            return call(t.raw_stream(dev))
    return call(t.raw_stream(dev))


def _scratch(nbytes: int, dev: int, device, workspace):
    """(address, bytes) of the workspace, and the tensor that holds it."""
    if workspace is None:
        if nbytes == 0:
            return None, 0, None
        ty = _types()
        ws = ty.torch.empty(nbytes, dtype=ty.u8, device=device)
        return ws.data_ptr(), nbytes, ws
    size = workspace.numel() * workspace.element_size()
    if workspace.get_device() != dev or not workspace.is_contiguous() or size < nbytes:
        raise ValueError(f"workspace must be {nbytes} contiguous bytes on the tensors' device")
    return workspace.data_ptr(), size, workspace


@functools.lru_cache(maxsize=1024)
def _decode_ws(batch, Hq, D, max_seqlen, partition, window) -> int:
    return paged_decode_workspace_size(batch, Hq, D, max_seqlen, partition, window)


@functools.lru_cache(maxsize=1024)
def _tree_ws(batch, Hq, Hkv, D, max_q) -> int:
    return paged_tree_attention_workspace_size(batch, Hq, Hkv, D, max_q)


def reshape_and_cache_fp8(key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping,
                          dev_error=None, stream=None, layout: str = "NHD") -> None:
    """reshape_and_cache into the 8-bit cache (in place): each head row of
    key/value [T, Hkv, D] (bf16 or float32; a token's heads contiguous, tokens
    any stride) becomes e4m3 codes in k_cache/v_cache (torch.float8_e4m3fn, the
    pool shapes of ``layout``) and one E8M0 byte in k_scale/v_scale ([num_blocks,
    Hkv, block_size] uint8): value = code * 2^(byte - 127), the exponent the
    smallest that keeps max|x| within 448.  A row with a NaN or an infinity is
    stored as byte 255 and reads as NaN.  slot_mapping: [T] int64, negative =
    skip, each slot at most once (tokens that share one leave a mixture there);
    dev_error receives PKV_DEVERR_SLOT for slots outside the pool."""
    dev = _cuda_index("key", key)
    desc = _fp8_pools(k_cache, v_cache, k_scale, v_scale, layout, dev)
    dtype, T = key.dtype, key.shape[0]
    dt = _types().codes.get(dtype)
    if dt is None:
        dt = _dtype_code(dtype)  # which says what it is
    ks = _token_rows("key", key, dtype, T, desc.num_kv_heads, desc.head_dim, dev)
    vs = _token_rows("value", value, dtype, T, desc.num_kv_heads, desc.head_dim, dev)
    _arg_vector("slot_mapping", slot_mapping, _types().i64, T, dev)
    err = _error_word(dev_error, dev)
    lib = load_library()

    def call(handle):
        return lib.pkv_reshape_and_cache_fp8(
            key.data_ptr(), value.data_ptr(), ks, vs, dt, k_cache.data_ptr(), v_cache.data_ptr(),
            k_scale.data_ptr(), v_scale.data_ptr(), slot_mapping.data_ptr(), T, desc, err, handle)
    st = _on_stream(dev, stream, call)
    if st:
        _check("pkv_reshape_and_cache_fp8", st)


def gather_cache_fp8(k_cache, v_cache, k_scale, v_scale, block_table, cu_seq_lens_k,
                     total_k: int, key=None, value=None, dev_error=None, stream=None,
                     layout: str = "NHD"):
    """The cached rows of every request as bf16: returns (key, value), each
    [total_k, Hkv, D], request r's positions 0.. at rows cu_seq_lens_k[r] ..
    (the arrays varlen_prefill_contiguous takes).  block_table: [B, max_blocks]
    int32; cu_seq_lens_k: [B+1] int32; total_k: host int, the rows of the
    outputs.  Rows of no request are left as they were (uninitialised in
    outputs allocated here)."""
    ty = _types()
    dev = _cuda_index("k_cache", k_cache)
    desc = _fp8_pools(k_cache, v_cache, k_scale, v_scale, layout, dev)
    _arg("cu_seq_lens_k", cu_seq_lens_k, ty.i32, 1, dev)
    _arg("block_table", block_table, ty.i32, 2, dev)
    B = cu_seq_lens_k.shape[0] - 1
    rows, max_blocks = block_table.shape
    _require(B >= 0 and rows == B, "block_table must have one row per request")
    total_k = int(total_k)
    _require(total_k >= 0, "total_k must not be negative")
    shape = (total_k, desc.num_kv_heads, desc.head_dim)
    if key is not None:
        _arg_shape("key", key, ty.bf16, shape, dev)
    if value is not None:
        _arg_shape("value", value, ty.bf16, shape, dev)
    err = _error_word(dev_error, dev)
    lib = load_library()

    def call(handle):
        k = ty.torch.empty(shape, dtype=ty.bf16, device=k_cache.device) if key is None else key
        v = ty.torch.empty(shape, dtype=ty.bf16, device=k_cache.device) if value is None else value
        return k, v, lib.pkv_gather_cache_fp8(
            k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
            k_scale.data_ptr(), v_scale.data_ptr(), desc, block_table.data_ptr(),
            max_blocks, cu_seq_lens_k.data_ptr(), B, total_k, err, handle)
    key, value, st = _on_stream(dev, stream, call)
    if st:
        _check("pkv_gather_cache_fp8", st)
    return key, value


def _attention_extras(sink, alibi_slopes, out, lse, q, rows: int, Hq: int, dev: int):
    """Checks what both attention calls take beside q and the pools."""
    ty = _types()
    if sink is not None:
        _arg_vector("sink", sink, ty.f32, Hq, dev)
    if alibi_slopes is not None:
        _arg_vector("alibi_slopes", alibi_slopes, ty.f32, Hq, dev)
    if out is not None:
        _arg_shape("out", out, ty.bf16, q.shape, dev)
    if lse is not None:
        _arg_shape("lse", lse, ty.f32, (rows, Hq), dev)


def paged_decode_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, cache_seqlens,
                     max_seqlen: int, sink=None, window_left: int = -1,
                     sm_scale: Optional[float] = None, partition_size: int = 0, out=None,
                     lse=None, workspace=None, dev_error=None, stream=None, alibi_slopes=None,
                     layout: str = "NHD"):
    """paged_decode over the 8-bit cache of reshape_and_cache_fp8: q and out are
    bf16 [B, Hq, D]; everything else as paged_decode (workspace of
    paged_decode_workspace_size bytes for the same arguments), but for
    partition_size 0, which lets the library choose (512 or more)."""
    ty = _types()
    dev = _cuda_index("q", q)
    desc = _fp8_pools(k_cache, v_cache, k_scale, v_scale, layout, dev)
    _arg("q", q, ty.bf16, 3, dev)
    B, Hq, D = q.shape
    _require(D == desc.head_dim, "head_dim of q and cache differ")
    _arg("block_table", block_table, ty.i32, 2, dev)
    _arg_vector("cache_seqlens", cache_seqlens, ty.i32, B, dev)
    rows, max_blocks = block_table.shape
    _require(rows == B, "block_table / cache_seqlens batch mismatch")
    _attention_extras(sink, alibi_slopes, out, lse, q, B, Hq, dev)
    err = _error_word(dev_error, dev)
    scale = float(sm_scale) if sm_scale is not None else D ** -0.5
    max_seqlen = _int32("max_seqlen", max_seqlen)
    window_left = _int32("window_left", min(window_left, _WIDEST))
    partition_size = _int32("partition_size", partition_size)
    # one partition needs no workspace
    need = 0 if max_seqlen <= (partition_size or 512) else \
        _decode_ws(B, Hq, D, max_seqlen, partition_size, window_left)
    lib = load_library()

    def call(handle):
        o = ty.torch.empty_like(q) if out is None else out
        ws, ws_bytes, held = _scratch(need, dev, q.device, workspace)
        return o, lib.pkv_paged_decode_fp8(
            o.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
            k_scale.data_ptr(), v_scale.data_ptr(), desc, block_table.data_ptr(),
            max_blocks, cache_seqlens.data_ptr(), max_seqlen, _ptr(sink),
            _ptr(alibi_slopes), B, Hq, window_left, scale, partition_size, _ptr(lse), ws,
            ws_bytes, err, handle)
    out, st = _on_stream(dev, stream, call)
    if st:
        _check("pkv_paged_decode_fp8", st)
    return out


def qk_norm_rope_reshape_and_cache(query, key, value, k_cache, v_cache, positions, slot_mapping,
                                   cos_sin, q_weight, k_weight, eps: float = 1e-6,
                                   rotary_dim: Optional[int] = None, is_neox_style: bool = True,
                                   query_out=None, key_out=None, k_scale=None, v_scale=None,
                                   dev_error=None, stream=None, layout: str = "NHD") -> None:
    """RMS norm of every head of query [T, Hq, D] and key [T, Hkv, D] (weights
    q_weight and k_weight [D], float32 or the rows' dtype), rotary embedding by
    positions [T] with the table cos_sin, and the cache write of the rotated key
    and the value at slot_mapping [T], in one pass.

    Rows are bf16 or float32; a token's heads are contiguous and tokens may
    have any stride (slices of a fused projection).  The rotated rows go to
    query_out / key_out, or back in place when these are None; they may not
    overlap one another or an input, but may be it: query_out query, key_out key or
    value.  With k_scale and v_scale the pools are the 8-bit cache of reshape_and_cache_fp8, else
    pools of the rows' dtype.  query (with query_out and q_weight) may be None."""
    ty = _types()
    dev = _cuda_index("key", key)
    dtype = key.dtype
    dt = ty.codes.get(dtype)
    if dt is None:
        dt = _dtype_code(dtype)
    if k_scale is None and v_scale is None:
        desc = _pools(k_cache, v_cache, None, None, dtype, layout, dev)
    else:
        desc = _fp8_pools(k_cache, v_cache, k_scale, v_scale, layout, dev)
    D, Hkv, T = desc.head_dim, desc.num_kv_heads, key.shape[0]
    ks = _token_rows("key", key, dtype, T, Hkv, D, dev)
    vs = _token_rows("value", value, dtype, T, Hkv, D, dev)
    kos = ks
    if key_out is None:
        key_out = key
    else:
        kos = _token_rows("key_out", key_out, dtype, T, Hkv, D, dev)
    Hq, qs, qos = 0, 0, 0
    if query is None:
        query_out = q_weight = None
    else:
        _require(query.dim() == 3, "query must be [T, num_qo_heads, head_dim]")
        Hq = query.size(1)
        qs = qos = _token_rows("query", query, dtype, T, Hq, D, dev)
        if query_out is None:
            query_out = query
        else:
            qos = _token_rows("query_out", query_out, dtype, T, Hq, D, dev)
    _arg_vector("positions", positions, ty.i64, T, dev)
    _arg_vector("slot_mapping", slot_mapping, ty.i64, T, dev)
    _arg("cos_sin", cos_sin, ty.f32, 3, dev)
    maxpos, half, two = cos_sin.shape
    rd = int(rotary_dim) if rotary_dim is not None else 2 * half
    _require(2 * half == rd and two == 2, "cos_sin must be [max_position, rotary_dim // 2, 2]")
    _require(k_weight is not None and (q_weight is not None or query is None),
             "q_weight and k_weight are needed")
    w32 = k_weight.dtype is ty.f32
    wd = ty.f32 if w32 else dtype
    _arg_vector("k_weight", k_weight, wd, D, dev)
    if q_weight is not None:
        _arg_vector("q_weight", q_weight, wd, D, dev)
    err = _error_word(dev_error, dev)
    # outputs are written while other heads and tokens are still read: apart from the
    # inputs and one another, or in place in rows that lie q, k, v, or looked at closely
    es = key.element_size()
    k0, v0, ko0 = key.data_ptr(), value.data_ptr(), key_out.data_ptr()
    q0, qo0 = (k0, ko0) if query is None else (query.data_ptr(), query_out.data_ptr())
    kn, qn, span = Hkv * D * es, Hq * D * es, (T - 1) * es
    k1, v1, ko1 = k0 + span * ks + kn, v0 + span * vs + kn, ko0 + span * kos + kn
    q1, qo1 = q0 + span * qs + qn, qo0 + span * qos + qn
    lo, hi = min(q0, k0, v0), max(q1, k1, v1)
    if not ((ko1 <= lo or ko0 >= hi) and (qo1 <= lo or qo0 >= hi)
            and (ko1 <= qo0 or qo1 <= ko0)) and \
            not (q0 == qo0 and k0 == ko0 and qs == qos == ks == kos == vs
                 and q0 + qn <= k0 and k0 + kn <= v0 and v0 + kn <= q0 + qs * es):
        _refuse_overlap(T, (("key_out", ko0, kos * es, kn), ("query_out", qo0, qos * es, qn)),
                        (("key", k0, ks * es, kn), ("query", q0, qs * es, qn),
                         ("value", v0, vs * es, kn)))
    lib = load_library()

    def call(handle):
        return lib.pkv_qk_norm_rope_reshape_and_cache(
            q0 if Hq else None, k0, v0, qs, ks, vs, dt, qo0 if Hq else None, ko0, qos, kos,
            k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_scale), _ptr(v_scale),
            positions.data_ptr(), slot_mapping.data_ptr(), T, Hq, desc, _ptr(q_weight),
            k_weight.data_ptr(), w32, float(eps), cos_sin.data_ptr(), maxpos, rd,
            bool(is_neox_style), err, handle)
    st = _on_stream(dev, stream, call)
    if st:
        _check("pkv_qk_norm_rope_reshape_and_cache", st)


def paged_tree_attention_workspace_size(batch: int, num_qo_heads: int, num_kv_heads: int,
                                        head_dim: int, max_seqlen_q: int) -> int:
    return int(load_library().pkv_paged_tree_attention_workspace_size(
        batch, num_qo_heads, num_kv_heads, head_dim, max_seqlen_q))


def paged_tree_attention(q, k_cache, v_cache, block_table, cu_seq_lens_q, cache_seqlens,
                         max_seqlen_q: int, max_seqlen: int, tree_mask, tree_depth=None,
                         k_scale=None, v_scale=None, sink=None, window_left: int = -1,
                         sm_scale: Optional[float] = None, partition_size: int = 0, out=None,
                         lse=None, workspace=None, dev_error=None, stream=None,
                         alibi_slopes=None, layout: str = "NHD"):
    """Attention of up to 256 drafted tokens per request over its pages; returns
    out [total_q, Hq, D].

    q: [total_q, Hq, D] bf16, the drafts of request r at rows cu_seq_lens_q[r] ..
    ([B+1] int32); their K/V are the last q_len of the cache_seqlens[r] ([B]
    int32) positions in the pages.  Every draft sees the context before them,
    and draft n of its request iff bit n % 64 of tree_mask[row, n // 64] is set
    (tree_mask [total_q, words] int64, words * 64 >= max_seqlen_q): set a
    draft's own bit and its ancestors'.  tree_depth: [total_q] int32, a draft's
    depth below the first draft position, needed with window_left or
    alibi_slopes (positions are context length + depth).  Pools are bf16, or the
    8-bit cache when k_scale and v_scale are given.  max_seqlen_q / max_seqlen:
    host ints; partition_size: least keys a CTA takes in one go (a multiple of 128;
    0: 128).
    sink, lse ([total_q, Hq] float32), window, layout as paged_decode."""
    ty = _types()
    dev = _cuda_index("q", q)
    if k_scale is None and v_scale is None:
        desc = _pools(k_cache, v_cache, None, None, ty.bf16, layout, dev)
    else:
        desc = _fp8_pools(k_cache, v_cache, k_scale, v_scale, layout, dev)
    _arg("q", q, ty.bf16, 3, dev)
    total_q, Hq, D = q.shape
    _require(D == desc.head_dim, "head_dim of q and cache differ")
    _arg("block_table", block_table, ty.i32, 2, dev)
    _arg("cache_seqlens", cache_seqlens, ty.i32, 1, dev)
    B = cache_seqlens.shape[0]
    _arg_vector("cu_seq_lens_q", cu_seq_lens_q, ty.i32, B + 1, dev)
    rows, max_blocks = block_table.shape
    _require(rows == B, "block_table must have one row per request")
    _arg("tree_mask", tree_mask, ty.i64, 2, dev)
    rows, words = tree_mask.shape
    max_seqlen_q = _int32("max_seqlen_q", max_seqlen_q)
    max_seqlen = _int32("max_seqlen", max_seqlen)
    window_left = _int32("window_left", min(window_left, _WIDEST))
    partition_size = _int32("partition_size", partition_size)
    _require(rows == total_q and 64 * words >= max_seqlen_q,
             "tree_mask must be [total_q, words] with words * 64 >= max_seqlen_q")
    if tree_depth is not None:
        _arg_vector("tree_depth", tree_depth, ty.i32, total_q, dev)
    elif window_left >= 0 or alibi_slopes is not None:
        raise ValueError("tree_depth is needed with a window or ALiBi slopes")
    _attention_extras(sink, alibi_slopes, out, lse, q, total_q, Hq, dev)
    err = _error_word(dev_error, dev)
    scale = float(sm_scale) if sm_scale is not None else D ** -0.5
    need = _tree_ws(B, Hq, desc.num_kv_heads, D, max_seqlen_q)
    lib = load_library()

    def call(handle):
        o = ty.torch.empty_like(q) if out is None else out
        ws, ws_bytes, held = _scratch(need, dev, q.device, workspace)
        return o, lib.pkv_paged_tree_attention(
            o.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_scale),
            _ptr(v_scale), desc, block_table.data_ptr(), max_blocks,
            cu_seq_lens_q.data_ptr(), cache_seqlens.data_ptr(), max_seqlen_q, max_seqlen,
            total_q, tree_mask.data_ptr(), words, _ptr(tree_depth), _ptr(sink),
            _ptr(alibi_slopes), B, Hq, window_left, scale, partition_size, _ptr(lse), ws,
            ws_bytes, err, handle)
    out, st = _on_stream(dev, stream, call)
    if st:
        _check("pkv_paged_tree_attention", st)
    return out


# ---------------------------------------------------------------------------
# a sparse decode step
# ---------------------------------------------------------------------------

def _disjoint(tensors) -> None:
    """Refuses (name, tensor) pairs of which two share memory (all contiguous)."""
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), name)
                   for name, t in tensors if t.numel())
    for (_, end, a), (start, _, b) in zip(spans, spans[1:]):
        if start < end:
            raise ValueError(f"{b} must not overlap {a}")


def update_block_tables(block_table, old_seqlens, new_seqlens, free_blocks, num_free,
                        block_size: int, num_rows: int, slot_mapping=None, positions=None,
                        cu_seq_lens_q=None, cu_seq_lens_k=None, dev_error=None, stream=None):
    """The bookkeeping of a step on the GPU: request r goes from old_seqlens[r] to
    new_seqlens[r] cached tokens ([B] int32).  Returns (slot_mapping [num_rows] int64,
    positions [num_rows] int64, cu_seq_lens_q [B+1] int32, cu_seq_lens_k [B+1] int32)
    of the new tokens, those of request r at rows cu_seq_lens_q[r] ..; rows behind the
    last one have slot -1 and position 0.

    block_table [B, max_blocks] int32, free_blocks [num_blocks] int32 (a stack of the
    pool's free pages) and num_free [1] int32 (its height) are changed in place:
    requests that grow take pages off the stack, requests that shrink (0: done) give
    theirs back, which are there to be taken in the same step.  All or nothing: with
    too few free pages (DEVERR_NO_BLOCKS) or metadata out of range nothing is moved,
    all slots are -1 and all offsets 0."""
    ty = _types()
    dev = _cuda_index("block_table", block_table)
    i32 = ty.i32
    shape = old_seqlens.shape
    if not (block_table.dtype is old_seqlens.dtype is new_seqlens.dtype is free_blocks.dtype
            is num_free.dtype is i32 and block_table.dim() == 2 and block_table.is_contiguous()
            and old_seqlens.is_contiguous() and new_seqlens.is_contiguous()
            and free_blocks.is_contiguous() and free_blocks.dim() == 1
            and shape == new_seqlens.shape == block_table.shape[:1] and num_free.numel() == 1
            and num_free.dim() == 1 and dev == old_seqlens.get_device() == new_seqlens.get_device()
            == free_blocks.get_device() == num_free.get_device()):
        _arg("block_table", block_table, i32, 2, dev)
        _arg_vector("old_seqlens", old_seqlens, i32, block_table.shape[0], dev)
        _arg_vector("new_seqlens", new_seqlens, i32, block_table.shape[0], dev)
        _arg("free_blocks", free_blocks, i32, 1, dev)
        _arg_vector("num_free", num_free, i32, 1, dev)
    B, max_blocks = block_table.shape
    nb = free_blocks.shape[0]
    num_rows, block_size = int(num_rows), int(block_size)
    if not (0 <= num_rows <= _WIDEST and 0 < block_size <= _WIDEST):
        _int32("num_rows", num_rows)
        _int32("block_size", block_size)
        _require(num_rows >= 0, "num_rows must not be negative")
    err = _error_word(dev_error, dev)
    # what is changed in place lies apart from the rest
    t0, f0, n0 = block_table.data_ptr(), free_blocks.data_ptr(), num_free.data_ptr()
    o0, w0 = old_seqlens.data_ptr(), new_seqlens.data_ptr()
    t1, f1, lb = t0 + 4 * B * max_blocks, f0 + 4 * nb, 4 * B
    fresh = (slot_mapping is None and positions is None and cu_seq_lens_q is None
             and cu_seq_lens_k is None)
    if not (fresh and (t1 <= f0 or f1 <= t0) and not (t0 <= n0 < t1 or f0 <= n0 < f1)
            and (o0 + lb <= t0 or t1 <= o0) and (w0 + lb <= t0 or t1 <= w0)
            and (o0 + lb <= f0 or f1 <= o0) and (w0 + lb <= f0 or f1 <= w0)
            and not (o0 <= n0 < o0 + lb or w0 <= n0 < w0 + lb)):
        if slot_mapping is not None:
            _arg_vector("slot_mapping", slot_mapping, ty.i64, num_rows, dev)
        if positions is not None:
            _arg_vector("positions", positions, ty.i64, num_rows, dev)
        if cu_seq_lens_q is not None:
            _arg_vector("cu_seq_lens_q", cu_seq_lens_q, i32, B + 1, dev)
        if cu_seq_lens_k is not None:
            _arg_vector("cu_seq_lens_k", cu_seq_lens_k, i32, B + 1, dev)
        given = [(n, t) for n, t in (
            ("block_table", block_table), ("free_blocks", free_blocks), ("num_free", num_free),
            ("slot_mapping", slot_mapping), ("positions", positions),
            ("cu_seq_lens_q", cu_seq_lens_q), ("cu_seq_lens_k", cu_seq_lens_k)) if t is not None]
        _disjoint(given + [("old_seqlens", old_seqlens)])
        _disjoint(given + [("new_seqlens", new_seqlens)])
    lib = load_library()

    def call(handle):
        empty, device = ty.torch.empty, block_table.device
        slots = empty(num_rows, dtype=ty.i64, device=device) if slot_mapping is None else slot_mapping
        pos = empty(num_rows, dtype=ty.i64, device=device) if positions is None else positions
        cuq = empty(B + 1, dtype=i32, device=device) if cu_seq_lens_q is None else cu_seq_lens_q
        cuk = empty(B + 1, dtype=i32, device=device) if cu_seq_lens_k is None else cu_seq_lens_k
        return (slots, pos, cuq, cuk), lib.pkv_update_block_tables(
            t0, max_blocks, o0, w0, B, f0, nb, n0, block_size, slots.data_ptr(), pos.data_ptr(),
            num_rows, cuq.data_ptr(), cuk.data_ptr(), err, handle)
    outs, st = _on_stream(dev, stream, call)
    if st:
        _check("pkv_update_block_tables", st)
    return outs


def _bounds(page_bounds, bounds_scale, dev: int):
    """Checks the bounds of a pool's pages; returns (num_blocks, num_kv_heads, head_dim)."""
    ty = _types()
    if not (page_bounds.dtype is ty.i8 and bounds_scale.dtype is ty.u8 and page_bounds.dim() == 4
            and page_bounds.is_contiguous() and bounds_scale.is_contiguous()
            and page_bounds.get_device() == bounds_scale.get_device() == dev
            and bounds_scale.shape == page_bounds.shape[:2]):
        _arg("page_bounds", page_bounds, ty.i8, 4, dev)
        _arg_shape("bounds_scale", bounds_scale, ty.u8, page_bounds.shape[:2], dev)
    nb, hkv, two, d = page_bounds.shape
    _require(two == 2, "page_bounds must be [num_blocks, num_kv_heads, 2, head_dim]")
    return nb, hkv, d


def update_page_bounds(k_cache, page_bounds, bounds_scale, slot_mapping, k_scale=None,
                       dev_error=None, stream=None, layout: str = "NHD") -> None:
    """The bounds of every page that a cache write at slot_mapping [T] (int64, negative =
    skipped) has written to, from the keys in k_cache (bf16, or the 8-bit cache with
    k_scale): page_bounds [num_blocks, Hkv, 2, D] int8 (the least and the largest key of
    each channel, rounded outward) and bounds_scale [num_blocks, Hkv] uint8 (E8M0 bytes;
    255: a key that is not finite) are changed in place.  The tokens of a page come in
    ascending order with fewer than 32 others between two of them, as update_block_tables
    orders them (a request's tokens side by side; else two of them race for the bounds, and
    nothing tells); rows of the page before its last token here count as written."""
    ty = _types()
    dev = _cuda_index("k_cache", k_cache)
    if k_scale is None:
        desc = _pools(k_cache, k_cache, None, None, ty.bf16, layout, dev)
    else:
        desc = _fp8_pools(k_cache, k_cache, k_scale, k_scale, layout, dev)
    nb, hkv, d = _bounds(page_bounds, bounds_scale, dev)
    _require((nb, hkv, d) == (desc.num_blocks, desc.num_kv_heads, desc.head_dim),
             "page_bounds must be [num_blocks, num_kv_heads, 2, head_dim] of the cache")
    if not (slot_mapping.dtype is ty.i64 and slot_mapping.dim() == 1
            and slot_mapping.get_device() == dev and slot_mapping.is_contiguous()):
        _arg("slot_mapping", slot_mapping, ty.i64, 1, dev)
    err = _error_word(dev_error, dev)
    lib = load_library()

    def call(handle):
        return lib.pkv_update_page_bounds(
            k_cache.data_ptr(), _ptr(k_scale), desc, page_bounds.data_ptr(),
            bounds_scale.data_ptr(), slot_mapping.data_ptr(), slot_mapping.shape[0], err, handle)
    st = _on_stream(dev, stream, call)
    if st:
        _check("pkv_update_page_bounds", st)


def _rows(q, head_dim: int, block_table, cache_seqlens, cu_seq_lens_q, dev: int):
    """Checks the queries and their requests; returns (total_q, Hq, batch, max_blocks)."""
    ty = _types()
    if not (q.dtype is ty.bf16 and block_table.dtype is cache_seqlens.dtype is ty.i32
            and q.dim() == 3 and block_table.dim() == 2 and q.is_contiguous()
            and block_table.is_contiguous() and cache_seqlens.is_contiguous()
            and dev == q.get_device() == block_table.get_device() == cache_seqlens.get_device()
            and cache_seqlens.shape == block_table.shape[:1]):
        _arg("q", q, ty.bf16, 3, dev)
        _arg("cache_seqlens", cache_seqlens, ty.i32, 1, dev)
        _arg("block_table", block_table, ty.i32, 2, dev)
        _require(block_table.shape[0] == cache_seqlens.shape[0],
                 "block_table must have one row per request")
    total_q, Hq, D = q.shape
    B, max_blocks = block_table.shape
    _require(D == head_dim, "head_dim of q and cache differ")
    if cu_seq_lens_q is not None:
        _arg_vector("cu_seq_lens_q", cu_seq_lens_q, ty.i32, B + 1, dev)
    else:
        _require(total_q == B, "without cu_seq_lens_q there is one query per request")
    return total_q, Hq, B, max_blocks


def select_pages(q, page_bounds, bounds_scale, block_table, cache_seqlens, max_seqlen: int,
                 top_k: int, block_size: int, num_first: int = 1, num_recent: int = 1,
                 cu_seq_lens_q=None, pages=None, dev_error=None, stream=None):
    """For every query and kv head the top_k pages of its request on which a key could
    score highest by the bounds of update_page_bounds (the highest over the group's
    heads); returns pages [total_q, Hkv, top_k] int32, ascending page numbers of the
    request, -1 behind them.

    q: [total_q, Hq, D] bf16, one query per request, or with cu_seq_lens_q ([B+1]
    int32) the last queries of each; block_table [B, max_blocks] and cache_seqlens [B]
    int32 (with the queries' own tokens); max_seqlen: host int >= every length.  The
    first num_first and the last num_recent (at least 1: a query's own) pages are always
    taken, equal scores from the lowest page."""
    ty = _types()
    dev = _cuda_index("q", q)
    nb, hkv, d = _bounds(page_bounds, bounds_scale, dev)
    total_q, Hq, B, max_blocks = _rows(q, d, block_table, cache_seqlens, cu_seq_lens_q, dev)
    max_seqlen, top_k, block_size = int(max_seqlen), int(top_k), int(block_size)
    num_first, num_recent = int(num_first), int(num_recent)
    if not (0 <= max_seqlen <= _WIDEST and 0 < top_k <= _WIDEST and 0 < block_size <= _WIDEST
            and 0 <= num_first <= _WIDEST and 0 < num_recent <= _WIDEST):
        for name, value in (("max_seqlen", max_seqlen), ("top_k", top_k),
                            ("block_size", block_size), ("num_first", num_first),
                            ("num_recent", num_recent)):
            _int32(name, value)
        _require(top_k > 0, "top_k must be positive")
    if pages is not None:
        _arg_shape("pages", pages, ty.i32, (total_q, hkv, top_k), dev)
    err = _error_word(dev_error, dev)
    lib = load_library()

    def call(handle):
        out = pages
        if out is None:
            out = ty.torch.empty(total_q, hkv, top_k, dtype=ty.i32, device=q.device)
        return out, lib.pkv_select_pages(
            out.data_ptr(), top_k, q.data_ptr(), page_bounds.data_ptr(), bounds_scale.data_ptr(),
            nb, block_size, hkv, d, block_table.data_ptr(), max_blocks, cache_seqlens.data_ptr(),
            max_seqlen, _ptr(cu_seq_lens_q), B, total_q, Hq, num_first, num_recent, err, handle)
    out, st = _on_stream(dev, stream, call)
    if st:
        _check("pkv_select_pages", st)
    return out


def paged_sparse_attention(q, k_cache, v_cache, block_table, cache_seqlens, pages,
                           cu_seq_lens_q=None, k_scale=None, v_scale=None, sink=None,
                           sm_scale: Optional[float] = None, out=None, lse=None, dev_error=None,
                           stream=None, layout: str = "NHD"):
    """Attention of every query over its list of pages; returns out [total_q, Hq, D].

    q [total_q, Hq, D] bf16, block_table, cache_seqlens and cu_seq_lens_q as in
    select_pages; pages [total_q, Hkv, top_k] int32, for each kv head strictly ascending
    page numbers of the request, -1 behind them (of select_pages, or any other choice).
    A query sees the keys of these pages up to its own position.  Pools are bf16, or the
    8-bit cache when k_scale and v_scale are given; sink, lse ([total_q, Hq] float32) and
    layout as paged_decode; out must not overlap q."""
    ty = _types()
    dev = _cuda_index("q", q)
    if k_scale is None and v_scale is None:
        desc = _pools(k_cache, v_cache, None, None, ty.bf16, layout, dev)
    else:
        desc = _fp8_pools(k_cache, v_cache, k_scale, v_scale, layout, dev)
    total_q, Hq, B, max_blocks = _rows(q, desc.head_dim, block_table, cache_seqlens,
                                       cu_seq_lens_q, dev)
    shape = pages.shape
    top_k = shape[-1] if shape else 0
    if not (pages.dtype is ty.i32 and shape == (total_q, desc.num_kv_heads, top_k)
            and pages.get_device() == dev and pages.is_contiguous()):
        _arg("pages", pages, ty.i32, 3, dev)
        _arg_shape("pages", pages, ty.i32, (total_q, desc.num_kv_heads, top_k), dev)
    _attention_extras(sink, None, out, lse, q, total_q, Hq, dev)
    if out is not None:
        _disjoint((("q", q), ("out", out)))
    err = _error_word(dev_error, dev)
    scale = float(sm_scale) if sm_scale is not None else desc.head_dim ** -0.5
    lib = load_library()

    def call(handle):
        o = ty.torch.empty_like(q) if out is None else out
        return o, lib.pkv_paged_sparse_attention(
            o.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_scale),
            _ptr(v_scale), desc, block_table.data_ptr(), max_blocks, cache_seqlens.data_ptr(),
            _ptr(cu_seq_lens_q), B, total_q, pages.data_ptr(), top_k, _ptr(sink), Hq, scale,
            _ptr(lse), err, handle)
    out, st = _on_stream(dev, stream, call)
    if st:
        _check("pkv_paged_sparse_attention", st)
    return out
