"""Python binding of libpa (argument marshalling only).

Every function here forwards to the C ABI declared in ``include/pa.h`` under
the same name; torch tensors are used only as device (or host) memory and
their current CUDA stream.  No computation of the method happens in Python:
if ``libpa.so`` is missing, importing the functions raises instead of
falling back to anything else.

Ordering of ``seq_lens``: every decode call (pa_decode*, pa_decode_cascade,
pa_decode_noalloc) launches as a programmatic dependent of the work before
it on the stream and reads ``seq_lens`` to split its work BEFORE it waits
for that work.  The calls of this library that write ``seq_lens``
(pa_append_slots_device, pa_trim_slots_device) do not let their dependents
start early, so a decode call may follow them.  If a kernel of yours writes ``seq_lens`` and calls ``griddepcontrol.launch_dependents``
(lets its dependents start early), do not launch a decode call directly
after it on the same stream: put a copy or any kernel
without that trigger in between.  Ordinary stream order (torch ops, copies)
needs nothing.
"""
from __future__ import annotations

import ctypes
import itertools
import os
import time

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpa.so")

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_OUT_OF_BLOCKS, PA_ERR_BAD_BLOCK_ID = 0, 1, 2, 3
PA_ERR_CUDA, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE = 4, 5, 6
PA_KV_BF16, PA_KV_FP8_E4M3, PA_KV_NVFP4 = 0, 1, 2

DEVERR_BAD_BLOCK_ID, DEVERR_BAD_SEQ_LEN, DEVERR_BAD_SLOT = 0x1, 0x2, 0x4
DEVERR_BAD_PAIR, DEVERR_TIMEOUT, DEVERR_LAUNCH = 0x8, 0x10, 0x20
DEVERR_OUT_OF_BLOCKS, DEVERR_BAD_QUERY = 0x40, 0x80

_lib = None

_c_int = ctypes.c_int32
_c_ptr = ctypes.c_void_p
_c_size = ctypes.c_size_t

# name -> (restype, argtypes); must match include/pa.h
SIGNATURES = {
    "pa_abi_version": (_c_int, []),
    "pa_testing_set_wait_limit": (_c_int, [ctypes.c_uint32, _c_int]),
    "pa_status_string": (ctypes.c_char_p, [_c_int]),
    "pa_get_device_error": (_c_int, [ctypes.POINTER(ctypes.c_uint32)]),
    "pa_cache_write": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_int, _c_ptr, _c_ptr, _c_int,
                                _c_int, _c_int, _c_int, _c_int, _c_ptr]),
    "pa_cache_write_fp8": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_int, _c_ptr, _c_ptr, _c_ptr,
                                    _c_ptr, _c_int, _c_int, _c_int, _c_int, _c_ptr]),
    "pa_swap_out": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int, _c_ptr, _c_ptr,
                             _c_ptr, _c_ptr, _c_int, _c_int, _c_int, _c_int, _c_int, _c_ptr]),
    "pa_swap_in": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int, _c_ptr, _c_ptr,
                            _c_ptr, _c_ptr, _c_int, _c_int, _c_int, _c_int, _c_int, _c_ptr]),
    "pa_copy_blocks": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int, _c_int,
                                _c_int, _c_int, _c_int, _c_int, _c_ptr]),
    "pa_quantize_fp8": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int, _c_ptr, _c_ptr,
                                 _c_ptr, _c_ptr, _c_int, _c_int, _c_int, _c_int, _c_ptr]),
    "pa_decode_workspace_size": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int,
                                          ctypes.POINTER(_c_size)]),
    "pa_decode": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int, _c_ptr, _c_int,
                           _c_ptr, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                           ctypes.c_float, _c_ptr, _c_ptr, _c_size, _c_int, _c_ptr]),
    "pa_decode_append": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr,
                                  _c_int, _c_ptr, _c_int, _c_int, _c_int, _c_int, _c_int,
                                  _c_int, ctypes.c_float, _c_ptr, _c_ptr, _c_size, _c_int,
                                  _c_ptr]),
    "pa_decode_cascade_workspace_size": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int,
                                                  _c_int, _c_int, ctypes.POINTER(_c_size)]),
    "pa_decode_cascade": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int, _c_ptr, _c_int,
                                   _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                   ctypes.c_float, _c_ptr, _c_ptr, _c_size, _c_int, _c_ptr]),
    "pa_decode_append_fp8": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr,
                                      _c_ptr, _c_ptr, _c_int, _c_ptr, _c_int, _c_int, _c_int,
                                      _c_int, _c_int, _c_int, ctypes.c_float, _c_ptr, _c_ptr,
                                      _c_size, _c_int, _c_ptr]),
    "pa_decode_noalloc": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int, _c_ptr,
                                   _c_int, _c_ptr, _c_int, _c_int, _c_int, _c_int, _c_int,
                                   _c_int, ctypes.c_float, _c_ptr, _c_int, _c_ptr]),
    "pa_cache_write_nvfp4": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_int, _c_ptr, _c_ptr, _c_ptr,
                                      _c_ptr, ctypes.c_float, ctypes.c_float, _c_int, _c_int,
                                      _c_int, _c_int, _c_ptr]),
    "pa_decode_nvfp4": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, ctypes.c_float,
                                 ctypes.c_float, _c_ptr, _c_int, _c_ptr, _c_int, _c_int, _c_int,
                                 _c_int, _c_int, _c_int, ctypes.c_float, _c_ptr, _c_ptr,
                                 _c_size, _c_int, _c_ptr]),
    "pa_decode_append_nvfp4": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr,
                                        _c_ptr, ctypes.c_float, ctypes.c_float, _c_ptr, _c_int,
                                        _c_ptr, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                        ctypes.c_float, _c_ptr, _c_ptr, _c_size, _c_int,
                                        _c_ptr]),
    "pa_append_slots_device": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_int, _c_ptr, _c_ptr, _c_int,
                                        _c_int, _c_int, _c_int, _c_ptr, _c_ptr, _c_ptr, _c_ptr,
                                        _c_ptr, _c_ptr]),
    "pa_trim_slots_device": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_int, _c_ptr, _c_ptr, _c_int,
                                      _c_int, _c_int, _c_ptr, _c_ptr, _c_ptr]),
    "pa_attention_workspace_size": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int,
                                             ctypes.POINTER(_c_size)]),
    "pa_prefill": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int, _c_ptr, _c_int,
                            _c_ptr, _c_ptr, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                            _c_int, ctypes.c_float, _c_ptr, _c_ptr, _c_size, _c_int, _c_ptr]),
    "pa_cross_attention": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int, _c_ptr,
                                    _c_int, _c_ptr, _c_ptr, _c_int, _c_int, _c_int, _c_int,
                                    _c_int, _c_int, _c_int, ctypes.c_float, _c_ptr, _c_ptr,
                                    _c_size, _c_int, _c_ptr]),
    "pa_allocator_create": (_c_int, [_c_int, ctypes.POINTER(_c_ptr)]),
    "pa_allocator_destroy": (None, [_c_ptr]),
    "pa_block_alloc": (_c_int, [_c_ptr, _c_int, _c_ptr]),
    "pa_block_free": (_c_int, [_c_ptr, _c_ptr, _c_int]),
    "pa_block_fork": (_c_int, [_c_ptr, _c_ptr, _c_int]),
    "pa_block_refcount": (_c_int, [_c_ptr, _c_int, ctypes.POINTER(_c_int)]),
    "pa_block_num_free": (_c_int, [_c_ptr]),
    "pa_seq_append_slots": (_c_int, [_c_ptr, _c_ptr, _c_int, _c_int, _c_int, _c_int,
                                     _c_ptr, _c_ptr, ctypes.POINTER(_c_int)]),
    "pa_allocator_usage": (_c_int, [_c_ptr, _c_ptr, _c_int, _c_ptr, _c_int, _c_int, _c_ptr]),
    "pa_batch_append_slots": (_c_int, [_c_ptr, _c_ptr, _c_int, _c_ptr, _c_ptr, _c_int, _c_int,
                                       _c_ptr, _c_ptr, _c_ptr, ctypes.POINTER(_c_int)]),
}


class PAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")


def lib() -> ctypes.CDLL:
    """The loaded libpa; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m paged_kv_cache_228_gb300.build` (there is no fallback)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().pa_status_string(status).decode()


def _check(fn: str, status: int):
    if status != PA_OK:
        raise PAError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _need(t, dtype, name, ndim=None):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got {t.dim()}")


def _kv_dtype(cache):
    if cache.dtype == torch.bfloat16:
        return PA_KV_BF16
    if cache.dtype in (torch.uint8, torch.float8_e4m3fn):
        return PA_KV_FP8_E4M3
    raise TypeError(f"unsupported cache dtype {cache.dtype}")


# ------------------------------------------------------------------ misc ---
def pa_abi_version() -> int:
    return int(lib().pa_abi_version())


def pa_get_device_error() -> int:
    v = ctypes.c_uint32(0)
    _check("pa_get_device_error", lib().pa_get_device_error(ctypes.byref(v)))
    return int(v.value)


# ----------------------------------------------------------------- cache ---
def pa_cache_write(k_new, v_new, slot_mapping, k_cache, v_cache, stream=None):
    """Scatter k_new/v_new [T, Hkv, d] into the pools at slot_mapping[T]."""
    _need(slot_mapping, torch.int64, "slot_mapping", 1)
    nb, hkv, bs, d = k_cache.shape
    _need(k_new, k_cache.dtype, "k_new", 3)
    _need(v_new, k_cache.dtype, "v_new", 3)
    _check("pa_cache_write", lib().pa_cache_write(
        _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), k_new.shape[0], _ptr(k_cache),
        _ptr(v_cache), nb, hkv, bs, d, _kv_dtype(k_cache), _stream(stream)))


def pa_cache_write_fp8(k_new, v_new, slot_mapping, k_cache, v_cache, k_scale, v_scale,
                       stream=None):
    """Append bf16 k_new/v_new [T, Hkv, d] to an E4M3 cache (uint8 pools,
    fp32 scales [num_blocks, Hkv]) at slot_mapping[T]; grow-only scales."""
    _need(slot_mapping, torch.int64, "slot_mapping", 1)
    _need(k_new, torch.bfloat16, "k_new", 3)
    _need(v_new, torch.bfloat16, "v_new", 3)
    _need(k_scale, torch.float32, "k_scale", 2)
    _need(v_scale, torch.float32, "v_scale", 2)
    if _kv_dtype(k_cache) != PA_KV_FP8_E4M3:
        raise TypeError("pa_cache_write_fp8: the cache must hold E4M3 bytes")
    nb, hkv, bs, d = k_cache.shape
    _check("pa_cache_write_fp8", lib().pa_cache_write_fp8(
        _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), k_new.shape[0], _ptr(k_cache),
        _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), nb, hkv, bs, d, _stream(stream)))


def pa_swap_out(k_cache, v_cache, block_ids, host_k, host_v, k_scale=None, v_scale=None,
                host_k_scale=None, host_v_scale=None, stream=None):
    """Copy the listed blocks (device int32 ids) of the pools into pinned
    host tensors [n, Hkv, bs, d] (and FP8 scales [n, Hkv])."""
    _need(block_ids, torch.int32, "block_ids", 1)
    nb, hkv, bs, d = k_cache.shape
    _check("pa_swap_out", lib().pa_swap_out(
        _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_ids),
        block_ids.shape[0], _ptr(host_k), _ptr(host_v), _ptr(host_k_scale),
        _ptr(host_v_scale), nb, hkv, bs, d, _kv_dtype(k_cache), _stream(stream)))


def pa_swap_in(host_k, host_v, block_ids, k_cache, v_cache, host_k_scale=None,
               host_v_scale=None, k_scale=None, v_scale=None, stream=None):
    """The reverse of pa_swap_out: pinned host slots i -> blocks block_ids[i]."""
    _need(block_ids, torch.int32, "block_ids", 1)
    nb, hkv, bs, d = k_cache.shape
    _check("pa_swap_in", lib().pa_swap_in(
        _ptr(host_k), _ptr(host_v), _ptr(host_k_scale), _ptr(host_v_scale), _ptr(block_ids),
        block_ids.shape[0], _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), nb,
        hkv, bs, d, _kv_dtype(k_cache), _stream(stream)))


def pa_copy_blocks(k_cache, v_cache, pairs, k_scale=None, v_scale=None, stream=None):
    """Copy-on-write: pairs int32 [P, 3] rows (src, dst, valid slots)."""
    _need(pairs, torch.int32, "pairs", 2)
    nb, hkv, bs, d = k_cache.shape
    _check("pa_copy_blocks", lib().pa_copy_blocks(
        _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(pairs),
        pairs.shape[0], nb, hkv, bs, d, _kv_dtype(k_cache), _stream(stream)))


def pa_quantize_fp8(k_src, v_src, block_ids, valid_lens, k_dst, v_dst, k_scale,
                    v_scale, stream=None):
    """Quantise listed bf16 blocks to E4M3 with per-(block, head) scales."""
    _need(block_ids, torch.int32, "block_ids", 1)
    _need(valid_lens, torch.int32, "valid_lens", 1)
    _need(k_scale, torch.float32, "k_scale", 2)
    _need(v_scale, torch.float32, "v_scale", 2)
    nb, hkv, bs, d = k_src.shape
    _check("pa_quantize_fp8", lib().pa_quantize_fp8(
        _ptr(k_src), _ptr(v_src), _ptr(block_ids), _ptr(valid_lens), block_ids.shape[0],
        _ptr(k_dst), _ptr(v_dst), _ptr(k_scale), _ptr(v_scale), nb, hkv, bs, d,
        _stream(stream)))


# ---------------------------------------------------------------- decode ---
def pa_testing_set_wait_limit(polls: int, stall: bool = False):
    """Test hook (include/pa_testing.h): polls before a decode pipeline wait
    gives up (0 restores the default and clears stall); stall=True makes
    every decode CTA first wait on a barrier nothing arrives at."""
    _check("pa_testing_set_wait_limit", lib().pa_testing_set_wait_limit(polls, int(stall)))


def pa_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                             num_splits=0) -> int:
    n = ctypes.c_size_t(0)
    _check("pa_decode_workspace_size", lib().pa_decode_workspace_size(
        num_seqs, num_q_heads, num_kv_heads, head_dim, num_splits, ctypes.byref(n)))
    return int(n.value)


def pa_decode(q, k_cache, v_cache, block_tables, seq_lens, scale, out, workspace=None,
              k_scale=None, v_scale=None, num_splits=0, stream=None):
    """Paged decode attention: out[B, Hq, d] (bf16) from q[B, Hq, d] (bf16).
    ``seq_lens`` is read before the wait for the preceding kernel (see the
    module docstring)."""
    _need(q, torch.bfloat16, "q", 3)
    _need(out, torch.bfloat16, "out", 3)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    B, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("pa_decode", lib().pa_decode(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
        _kv_dtype(k_cache), _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), B,
        hq, hkv, d, bs, nb, float(scale), _ptr(out), _ptr(workspace), ws_bytes, num_splits,
        _stream(stream)))


def pa_decode_append(q, k_new, v_new, slot_mapping, k_cache, v_cache, block_tables, seq_lens,
                     scale, out, workspace=None, num_splits=0, stream=None):
    """This step's cache write and decode in one launch (bf16 cache): the
    same cache and out as pa_cache_write(k_new, v_new, slot_mapping, ...)
    then pa_decode(...), where row b of k_new / v_new is sequence b's new
    token and slot_mapping[b] its slot (< 0: none)."""
    _need(q, torch.bfloat16, "q", 3)
    _need(k_new, torch.bfloat16, "k_new", 3)
    _need(v_new, torch.bfloat16, "v_new", 3)
    _need(slot_mapping, torch.int64, "slot_mapping", 1)
    _need(out, torch.bfloat16, "out", 3)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    if k_cache.dtype != torch.bfloat16 or v_cache.dtype != torch.bfloat16:
        raise ValueError("pa_decode_append: the cache must be bf16")
    B, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    if tuple(k_new.shape) != (B, hkv, d) or tuple(v_new.shape) != (B, hkv, d) or \
            slot_mapping.shape[0] != B:
        raise ValueError("pa_decode_append: k_new/v_new must be [B, Hkv, d], slot_mapping [B]")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("pa_decode_append", lib().pa_decode_append(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache),
        _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), B, hq, hkv, d, bs, nb,
        float(scale), _ptr(out), _ptr(workspace), ws_bytes, num_splits, _stream(stream)))


def pa_decode_append_fp8(q, k_new, v_new, slot_mapping, k_cache, v_cache, k_scale, v_scale,
                         block_tables, seq_lens, scale, out, workspace=None, num_splits=0,
                         stream=None):
    """The FP8 decode step in one launch: pa_cache_write_fp8 of row b of
    k_new / v_new at slot_mapping[b], then pa_decode, bit for bit (block
    size 8 or 16)."""
    _need(q, torch.bfloat16, "q", 3)
    _need(k_new, torch.bfloat16, "k_new", 3)
    _need(v_new, torch.bfloat16, "v_new", 3)
    _need(slot_mapping, torch.int64, "slot_mapping", 1)
    _need(k_scale, torch.float32, "k_scale", 2)
    _need(v_scale, torch.float32, "v_scale", 2)
    _need(out, torch.bfloat16, "out", 3)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    if _kv_dtype(k_cache) != PA_KV_FP8_E4M3:
        raise TypeError("pa_decode_append_fp8: the cache must hold E4M3 bytes")
    B, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("pa_decode_append_fp8", lib().pa_decode_append_fp8(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache),
        _ptr(k_scale), _ptr(v_scale), _ptr(block_tables), block_tables.shape[1],
        _ptr(seq_lens), B, hq, hkv, d, bs, nb, float(scale), _ptr(out), _ptr(workspace),
        ws_bytes, num_splits, _stream(stream)))


# ----------------------------------------------------------------- NVFP4 ---
def nvfp4_empty_cache(num_blocks, num_kv_heads, block_size, head_dim, device="cuda"):
    """Zeroed NVFP4 pools (k, k_sf, v, v_sf), uint8, in the layout of
    include/pa.h: k [nb, Hkv, bs, d/2], k_sf [nb, Hkv, bs, d/16],
    v [nb, Hkv, bs/2, d], v_sf [nb, Hkv, d/16, bs]."""
    nb, h, bs, d = num_blocks, num_kv_heads, block_size, head_dim
    z = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device=device)
    return z(nb, h, bs, d // 2), z(nb, h, bs, d // 16), z(nb, h, bs // 2, d), z(nb, h, d // 16, bs)


def _nvfp4_dims(cache):
    k, k_sf, v, v_sf = cache
    for t, n in zip(cache, ("k", "k_sf", "v", "v_sf")):
        _need(t, torch.uint8, n, 4)
    nb, hkv, bs, d2 = k.shape
    d = 2 * d2
    if tuple(k_sf.shape) != (nb, hkv, bs, d // 16) or tuple(v.shape) != (nb, hkv, bs // 2, d) \
            or tuple(v_sf.shape) != (nb, hkv, d // 16, bs):
        raise ValueError("NVFP4 cache: inconsistent pool shapes")
    return nb, hkv, bs, d


def pa_cache_write_nvfp4(k_new, v_new, slot_mapping, cache, k_gscale, v_gscale, stream=None):
    """Quantise k_new/v_new [T, Hkv, d] (bf16) into the NVFP4 pools
    cache = (k, k_sf, v, v_sf) at slot_mapping[T] with tensor scales
    k_gscale / v_gscale."""
    _need(k_new, torch.bfloat16, "k_new", 3)
    _need(v_new, torch.bfloat16, "v_new", 3)
    _need(slot_mapping, torch.int64, "slot_mapping", 1)
    nb, hkv, bs, d = _nvfp4_dims(cache)
    k, k_sf, v, v_sf = cache
    _check("pa_cache_write_nvfp4", lib().pa_cache_write_nvfp4(
        _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), k_new.shape[0], _ptr(k), _ptr(v),
        _ptr(k_sf), _ptr(v_sf), float(k_gscale), float(v_gscale), nb, hkv, bs, d,
        _stream(stream)))


def pa_decode_nvfp4(q, cache, k_gscale, v_gscale, block_tables, seq_lens, scale, out,
                    workspace=None, num_splits=0, stream=None):
    """Paged decode attention over NVFP4 pools cache = (k, k_sf, v, v_sf)."""
    _need(q, torch.bfloat16, "q", 3)
    _need(out, torch.bfloat16, "out", 3)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    nb, hkv, bs, d = _nvfp4_dims(cache)
    k, k_sf, v, v_sf = cache
    B, hq, dq = q.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("pa_decode_nvfp4", lib().pa_decode_nvfp4(
        _ptr(q), _ptr(k), _ptr(v), _ptr(k_sf), _ptr(v_sf), float(k_gscale), float(v_gscale),
        _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), B, hq, hkv, dq, bs, nb,
        float(scale), _ptr(out), _ptr(workspace), ws_bytes, num_splits, _stream(stream)))


def pa_decode_append_nvfp4(q, k_new, v_new, slot_mapping, cache, k_gscale, v_gscale,
                           block_tables, seq_lens, scale, out, workspace=None, num_splits=0,
                           stream=None):
    """The NVFP4 decode step in one launch: pa_cache_write_nvfp4 of row b of
    k_new / v_new at slot_mapping[b], then pa_decode_nvfp4, bit for bit."""
    _need(q, torch.bfloat16, "q", 3)
    _need(k_new, torch.bfloat16, "k_new", 3)
    _need(v_new, torch.bfloat16, "v_new", 3)
    _need(slot_mapping, torch.int64, "slot_mapping", 1)
    _need(out, torch.bfloat16, "out", 3)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    nb, hkv, bs, d = _nvfp4_dims(cache)
    k, k_sf, v, v_sf = cache
    B, hq, dq = q.shape
    if tuple(k_new.shape) != (B, hkv, dq) or tuple(v_new.shape) != (B, hkv, dq) or \
            slot_mapping.shape[0] != B:
        raise ValueError("pa_decode_append_nvfp4: k_new/v_new must be [B, Hkv, d], "
                         "slot_mapping [B]")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("pa_decode_append_nvfp4", lib().pa_decode_append_nvfp4(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k), _ptr(v), _ptr(k_sf),
        _ptr(v_sf), float(k_gscale), float(v_gscale), _ptr(block_tables), block_tables.shape[1],
        _ptr(seq_lens), B, hq, hkv, dq, bs, nb, float(scale), _ptr(out), _ptr(workspace),
        ws_bytes, num_splits, _stream(stream)))


def pa_decode_cascade_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                     block_size, prefix_len, num_splits=0):
    n = _c_size(0)
    _check("pa_decode_cascade_workspace_size", lib().pa_decode_cascade_workspace_size(
        num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, prefix_len, num_splits,
        ctypes.byref(n)))
    return n.value


def pa_decode_cascade(q, k_cache, v_cache, block_tables, seq_lens, prefix_len, scale, out,
                      workspace, num_splits=0, stream=None):
    """pa_decode for a batch whose sequences share their first prefix_len
    tokens (the same physical blocks): the prefix is read once."""
    _need(q, torch.bfloat16, "q", 3)
    _need(out, torch.bfloat16, "out", 3)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    if k_cache.dtype != torch.bfloat16 or v_cache.dtype != torch.bfloat16:
        raise ValueError("pa_decode_cascade: the cache must be bf16")
    B, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("pa_decode_cascade", lib().pa_decode_cascade(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
        _ptr(seq_lens), B, hq, hkv, d, bs, nb, int(prefix_len), float(scale), _ptr(out),
        _ptr(workspace), ws_bytes, num_splits, _stream(stream)))


NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024


def pa_decode_noalloc(q, k_cache, v_cache, block_tables, seq_lens, scale, out,
                      k_scale=None, v_scale=None, num_splits=0, stream=None):
    """pa_decode without a workspace argument, for callers that cannot
    allocate device memory: the library's own 16 MiB device array serves as
    scratch.  Calls on one device share it, so calls whose kernels overlap
    (unordered streams) race; requests needing more scratch raise
    PA_ERR_WORKSPACE."""
    _need(q, torch.bfloat16, "q", 3)
    _need(out, torch.bfloat16, "out", 3)
    _need(block_tables, torch.int32, "block_tables", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    B, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    _check("pa_decode_noalloc", lib().pa_decode_noalloc(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
        _kv_dtype(k_cache), _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), B,
        hq, hkv, d, bs, nb, float(scale), _ptr(out), num_splits, _stream(stream)))


# ----------------------------------------------------------- prompt side ---
# These calls are made between short kernels, so what a call checks is one
# expression of attribute reads; only where it fails are the tensors looked
# at one by one for the message.  (10 tensors: 7 us a call on a Grace core,
# 21 us with a helper call per check.)  Unlike the decode calls, they may be
# made while another device is current: they run on their tensors' device.
def _bad(t, name, dtype, shape):
    """Why `t` is not a contiguous `dtype` tensor of `shape`."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != len(shape) or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: must be contiguous")


def _refuse(named):
    """Raise for the first of (name, tensor or None, dtype, shape) that is not
    as it should be, or for tensors on the CPU or on different devices."""
    for name, t, dtype, shape in named:
        if t is not None and (t.dtype != dtype or tuple(t.shape) != tuple(shape) or
                              not t.is_contiguous()):
            _bad(t, name, dtype, shape)
    for name, t, _, _ in named:
        if t is not None and t.get_device() < 0:
            raise ValueError(f"{name}: must be a CUDA tensor, is on {t.device}")
    raise ValueError("tensors on different devices: " + ", ".join(
        f"{name} on {t.device}" for name, t, _, _ in named if t is not None))


_raw_stream, _current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _call(fn, dev, stream, args):
    if stream is None:
        stream = _raw_stream(dev)
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    if _current() == dev:
        status = getattr(_lib or lib(), fn)(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = getattr(_lib or lib(), fn)(*args, stream)
    if status != PA_OK:
        raise PAError(fn, status)


def pa_append_slots_device(lens, n_new, block_tables, free_ids, num_free, block_size,
                           slot_mapping, q_start, seq_lens, num_free_out, num_done, stream=None):
    """Grow sequence b from lens[b] by n_new[b] tokens on the GPU: new table
    entries from the stack free_ids[0 .. num_free), the new tokens' slots,
    the query offsets q_start [B + 1] and seq_lens.  seq_lens may be lens,
    num_free_out may be num_free.  len(slot_mapping) is the token capacity
    (rows past the last sequence get -1)."""
    i32 = torch.int32
    of_b, of_n, of_t = lens.shape, free_ids.shape, slot_mapping.shape
    (B,), (N,), (T,) = of_b, of_n, of_t
    width = block_tables.shape[-1]
    dev = lens.get_device()
    if not (dev >= 0 and lens.dtype is i32 and lens.is_contiguous() and
            n_new.dtype is i32 and n_new.shape == of_b and n_new.is_contiguous() and
            block_tables.dtype is i32 and block_tables.shape == (B, width) and
            block_tables.is_contiguous() and free_ids.dtype is i32 and
            free_ids.is_contiguous() and num_free.dtype is i32 and num_free.shape == (1,) and
            slot_mapping.dtype is torch.int64 and slot_mapping.is_contiguous() and
            q_start.dtype is i32 and q_start.shape == (B + 1,) and q_start.is_contiguous() and
            seq_lens.dtype is i32 and seq_lens.shape == of_b and seq_lens.is_contiguous() and
            num_free_out.dtype is i32 and num_free_out.shape == (1,) and
            num_done.dtype is i32 and num_done.shape == (1,) and
            n_new.get_device() == dev and block_tables.get_device() == dev and
            free_ids.get_device() == dev and num_free.get_device() == dev and
            slot_mapping.get_device() == dev and q_start.get_device() == dev and
            seq_lens.get_device() == dev and num_free_out.get_device() == dev and
            num_done.get_device() == dev):
        _refuse((("lens", lens, i32, of_b), ("n_new", n_new, i32, of_b),
                 ("block_tables", block_tables, i32, (B, width)),
                 ("free_ids", free_ids, i32, of_n), ("num_free", num_free, i32, (1,)),
                 ("slot_mapping", slot_mapping, torch.int64, of_t),
                 ("q_start", q_start, i32, (B + 1,)), ("seq_lens", seq_lens, i32, of_b),
                 ("num_free_out", num_free_out, i32, (1,)), ("num_done", num_done, i32, (1,))))
    _call("pa_append_slots_device", dev, stream, (
        lens.data_ptr(), n_new.data_ptr(), block_tables.data_ptr(), width, free_ids.data_ptr(),
        num_free.data_ptr(), B, T, block_size, N, slot_mapping.data_ptr(), q_start.data_ptr(),
        seq_lens.data_ptr(), num_free_out.data_ptr(), num_done.data_ptr()))


def pa_trim_slots_device(lens, new_lens, block_tables, free_ids, num_free, block_size, seq_lens,
                         num_free_out, stream=None):
    """Shrink sequence b from lens[b] to new_lens[b] tokens on the GPU: its
    blocks behind the new length are pushed onto free_ids.  seq_lens may be
    lens, num_free_out may be num_free."""
    i32 = torch.int32
    of_b, of_n = lens.shape, free_ids.shape
    (B,), (N,) = of_b, of_n
    width = block_tables.shape[-1]
    dev = lens.get_device()
    if not (dev >= 0 and lens.dtype is i32 and lens.is_contiguous() and
            new_lens.dtype is i32 and new_lens.shape == of_b and new_lens.is_contiguous() and
            block_tables.dtype is i32 and block_tables.shape == (B, width) and
            block_tables.is_contiguous() and free_ids.dtype is i32 and
            free_ids.is_contiguous() and num_free.dtype is i32 and num_free.shape == (1,) and
            seq_lens.dtype is i32 and seq_lens.shape == of_b and seq_lens.is_contiguous() and
            num_free_out.dtype is i32 and num_free_out.shape == (1,) and
            new_lens.get_device() == dev and block_tables.get_device() == dev and
            free_ids.get_device() == dev and num_free.get_device() == dev and
            seq_lens.get_device() == dev and num_free_out.get_device() == dev):
        _refuse((("lens", lens, i32, of_b), ("new_lens", new_lens, i32, of_b),
                 ("block_tables", block_tables, i32, (B, width)),
                 ("free_ids", free_ids, i32, of_n), ("num_free", num_free, i32, (1,)),
                 ("seq_lens", seq_lens, i32, of_b), ("num_free_out", num_free_out, i32, (1,))))
    _call("pa_trim_slots_device", dev, stream, (
        lens.data_ptr(), new_lens.data_ptr(), block_tables.data_ptr(), width,
        free_ids.data_ptr(), num_free.data_ptr(), B, block_size, N, seq_lens.data_ptr(),
        num_free_out.data_ptr()))


def pa_attention_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                num_splits=0) -> int:
    n = _c_size(0)
    _check("pa_attention_workspace_size", lib().pa_attention_workspace_size(
        num_seqs, num_q_heads, num_kv_heads, head_dim, num_splits, ctypes.byref(n)))
    return int(n.value)


def _attention(fn, q, k_cache, v_cache, block_tables, q_start, seq_lens, scale, out, workspace,
               k_scale, v_scale, num_splits, stream):
    bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    of_q, of_kv, of_b = q.shape, k_cache.shape, seq_lens.shape
    T, hq, d = of_q
    nb, hkv, bs, d2 = of_kv
    B, = of_b
    width = block_tables.shape[-1]
    kv_type = k_cache.dtype
    kv = PA_KV_BF16 if kv_type is bf16 else _kv_dtype(k_cache)
    if d2 != d:
        raise ValueError(f"{fn}: head_dim of q is {d}, of the cache {d2}")
    dev = q.get_device()
    ok = (dev >= 0 and q.dtype is bf16 and q.is_contiguous() and
          out.dtype is bf16 and out.shape == of_q and out.is_contiguous() and
          k_cache.is_contiguous() and v_cache.dtype is kv_type and v_cache.shape == of_kv and
          v_cache.is_contiguous() and block_tables.dtype is i32 and
          block_tables.shape == (B, width) and block_tables.is_contiguous() and
          seq_lens.dtype is i32 and seq_lens.is_contiguous() and
          k_cache.get_device() == dev and v_cache.get_device() == dev and
          block_tables.get_device() == dev and seq_lens.get_device() == dev and
          out.get_device() == dev)
    starts = ks = vs = ws = None
    ws_bytes = 0
    if q_start is not None:
        ok = ok and (q_start.dtype is i32 and q_start.shape == (B + 1,) and
                     q_start.is_contiguous() and q_start.get_device() == dev)
        starts = q_start.data_ptr()
    if workspace is not None:
        ok = ok and workspace.is_contiguous() and workspace.get_device() == dev
        ws, ws_bytes = workspace.data_ptr(), workspace.nbytes
    if kv == PA_KV_FP8_E4M3:
        if k_scale is None or v_scale is None:
            raise ValueError(f"{fn}: an FP8 cache needs k_scale and v_scale")
        ok = ok and (k_scale.dtype is f32 and k_scale.shape == (nb, hkv) and
                     k_scale.is_contiguous() and k_scale.get_device() == dev and
                     v_scale.dtype is f32 and v_scale.shape == (nb, hkv) and
                     v_scale.is_contiguous() and v_scale.get_device() == dev)
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    elif k_scale is not None or v_scale is not None:
        raise ValueError(f"{fn}: a bf16 cache takes no scales")
    if not ok:
        named = [("q", q, bf16, of_q), ("k_cache", k_cache, kv_type, of_kv),
                 ("v_cache", v_cache, kv_type, of_kv),
                 ("block_tables", block_tables, i32, (B, width)),
                 ("seq_lens", seq_lens, i32, of_b), ("out", out, bf16, of_q),
                 ("q_start", q_start, i32, (B + 1,)), ("k_scale", k_scale, f32, (nb, hkv)),
                 ("v_scale", v_scale, f32, (nb, hkv))]
        if workspace is not None:
            named.append(("workspace", workspace, workspace.dtype, workspace.shape))
        _refuse(named)
    _call(fn, dev, stream, (
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, kv,
        block_tables.data_ptr(), width, starts, seq_lens.data_ptr(), B, T, hq, hkv, d, bs, nb,
        float(scale), out.data_ptr(), ws, ws_bytes, num_splits))


def pa_prefill(q, k_cache, v_cache, block_tables, q_start, seq_lens, scale, out, workspace=None,
               k_scale=None, v_scale=None, num_splits=0, stream=None):
    """Causal attention of each sequence's newest tokens over its paged
    cache: q, out [T, Hq, d] (bf16), sequence b's tokens at rows
    [q_start[b], q_start[b + 1]), the last of them at position
    seq_lens[b] - 1.  Their K and V are in the cache already."""
    _attention("pa_prefill", q, k_cache, v_cache, block_tables, q_start, seq_lens, scale, out,
               workspace, k_scale, v_scale, num_splits, stream)


def pa_cross_attention(q, k_cache, v_cache, block_tables, q_start, seq_lens, scale, out,
                       workspace=None, k_scale=None, v_scale=None, num_splits=0, stream=None):
    """Attention of a decoder's tokens to an encoder's states in a paged
    cache: every token of sequence b sees all seq_lens[b] states.  q_start
    None: one token per sequence."""
    _attention("pa_cross_attention", q, k_cache, v_cache, block_tables, q_start, seq_lens, scale,
               out, workspace, k_scale, v_scale, num_splits, stream)


# --------------------------------------------------------- block manager ---
class Allocator:
    """Handle over the native host block manager (pa_allocator)."""

    def __init__(self, num_blocks: int):
        h = ctypes.c_void_p()
        _check("pa_allocator_create", lib().pa_allocator_create(num_blocks, ctypes.byref(h)))
        self._h = h
        self.num_blocks = num_blocks

    def close(self):
        if self._h:
            lib().pa_allocator_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @staticmethod
    def _ids(ids):
        arr = (ctypes.c_int32 * max(1, len(ids)))(*ids)
        return arr, len(ids)

    def alloc(self, n: int):
        """(status, ids or None)."""
        buf = (ctypes.c_int32 * max(1, n))()
        st = lib().pa_block_alloc(self._h, n, buf)
        return st, (list(buf[:n]) if st == PA_OK else None)

    def free(self, ids) -> int:
        arr, n = self._ids(ids)
        return lib().pa_block_free(self._h, arr, n)

    def fork(self, ids) -> int:
        arr, n = self._ids(ids)
        return lib().pa_block_fork(self._h, arr, n)

    def refcount(self, bid: int):
        rc = ctypes.c_int32(0)
        st = lib().pa_block_refcount(self._h, bid, ctypes.byref(rc))
        return st, (rc.value if st == PA_OK else None)

    def num_free(self) -> int:
        return int(lib().pa_block_num_free(self._h))

    def append_slots(self, table: list, length: int, n: int, block_size: int,
                     max_blocks: int):
        """Grow a sequence; ``table`` (list) is updated in place on success.

        Returns (status, slots, cow_pairs) like the C call.
        """
        tab = (ctypes.c_int32 * max(1, max_blocks))(*([-1] * max(1, max_blocks)))
        for i, b in enumerate(table[:max_blocks]):
            tab[i] = b
        slots = (ctypes.c_int64 * max(1, n))()
        cow = (ctypes.c_int32 * 3)()
        ncow = ctypes.c_int32(0)
        st = lib().pa_seq_append_slots(self._h, tab, max_blocks, length, n, block_size,
                                       slots, cow, ctypes.byref(ncow))
        if st != PA_OK:
            return st, None, None
        # the call filled the -1 padded table up to the sequence's new end
        table[:] = list(itertools.takewhile(lambda x: x >= 0, tab))
        pairs = [tuple(cow[:3])] if ncow.value else []
        return st, list(slots[:n]), pairs


class BatchAppender:
    """One decode step's appends for a batch through pa_batch_append_slots.

    Holds host arrays sized for the batch so that each call is one native
    call with no per-sequence Python work: ``tables`` (int32 [B, max_blocks],
    -1 padded) is updated in place.
    """

    def __init__(self, alloc: "Allocator", tables, max_blocks: int):
        import numpy as np
        self.alloc = alloc
        self.max_blocks = max_blocks
        B = len(tables)
        self.tables = np.full((B, max_blocks), -1, dtype=np.int32)
        for b, t in enumerate(tables):
            self.tables[b, :len(t)] = t
        self.cow = np.zeros((B, 3), dtype=np.int32)
        self.ncow = np.zeros(B, dtype=np.int32)

    def append(self, lens, n_new, block_size: int):
        """(status, slots int64 [sum n_new], cow pairs list, num_done)."""
        import numpy as np
        lens = np.ascontiguousarray(lens, dtype=np.int32)
        n_new = np.ascontiguousarray(n_new, dtype=np.int32)
        slots = np.zeros(max(1, int(n_new.sum())), dtype=np.int64)
        done = ctypes.c_int32(0)
        fn = lib().pa_batch_append_slots
        args = (self.alloc._h, self.tables.ctypes.data, self.max_blocks, lens.ctypes.data,
                n_new.ctypes.data, len(lens), block_size, slots.ctypes.data,
                self.cow.ctypes.data, self.ncow.ctypes.data, ctypes.byref(done))
        t0 = time.perf_counter()
        st = fn(*args)
        self.last_call_us = (time.perf_counter() - t0) * 1e6  # the native call alone
        pairs = [tuple(int(x) for x in self.cow[i]) for i in np.flatnonzero(self.ncow[:done.value])]
        return st, slots[:int(n_new[:done.value].sum())], pairs, done.value


def allocator_usage(alloc: "Allocator", tables, lens, block_size: int) -> dict:
    """pa_allocator_usage over the sequences (tables: lists or an int32
    [B, max_blocks] array; lens: per-sequence lengths)."""
    import numpy as np
    if isinstance(tables, np.ndarray):
        tab = np.ascontiguousarray(tables, dtype=np.int32)
    else:
        width = max([1] + [len(t) for t in tables])
        tab = np.full((len(tables), width), -1, dtype=np.int32)
        for b, t in enumerate(tables):
            tab[b, :len(t)] = t
    ln = np.ascontiguousarray(lens, dtype=np.int32)
    out = np.zeros(4, dtype=np.int64)
    _check("pa_allocator_usage", lib().pa_allocator_usage(
        alloc._h, tab.ctypes.data, tab.shape[1], ln.ctypes.data, len(ln), block_size,
        out.ctypes.data))
    return dict(zip(("live_blocks", "slots_reserved", "tokens_stored", "tokens_logical"),
                    (int(x) for x in out)))


def replay_script(ops, num_seqs: int, block_size: int, max_blocks: int, num_blocks: int):
    """Apply a workload op script to a fresh native allocator.

    Returns (allocator, tables, lens); raises on any non-OK status.
    """
    a = Allocator(num_blocks)
    tables = [[] for _ in range(num_seqs)]
    lens = [0] * num_seqs
    for op in ops:
        kind = op[0]
        if kind == "alloc":
            st, _ = a.alloc(op[1])
            _check("pa_block_alloc", st)
        elif kind == "free_list":
            _check("pa_block_free", a.free(op[1]))
        elif kind == "append":
            _, b, n = op
            st, _, _ = a.append_slots(tables[b], lens[b], n, block_size, max_blocks)
            _check("pa_seq_append_slots", st)
            lens[b] += n
        elif kind == "fork":
            _, child, parent, ntok = op
            ids = tables[parent][:-(-ntok // block_size)]
            _check("pa_block_fork", a.fork(ids))
            tables[child] = list(ids)
            lens[child] = ntok
        else:
            raise ValueError(kind)
    return a, tables, lens
