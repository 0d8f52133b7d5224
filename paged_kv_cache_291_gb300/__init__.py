"""paged_kv_cache_291_gb300 -- Python binding of libpagedkv (GB300, sm_103a).

A thin ctypes layer over the C-ABI declared in ``include/pkv.h``: it checks
tensor dtypes, shapes and devices, passes ``data_ptr()`` values and the
current CUDA stream, and raises :class:`PKVError` on a non-OK status.  Every
step of the computation runs in the library's CUDA kernels; there is no
fallback of any kind, and the binding refuses to work when ``libpagedkv.so``
has not been built (build it with ``python -m paged_kv_cache_291_gb300.build``
or ``__graft_entry__.build()``).

Tensors: K/V pools are 2-byte (bf16) CUDA tensors
``[num_blocks][num_kv_heads][16][head_dim]``; q/k_new/v_new bf16; index
arrays int32; outputs float32.  8-bit pools are uint8 or float8_e4m3fn
(e4m3 codes) with ``k_scale`` and ``v_scale``, or, with ``block_scales``
float32 ``[num_blocks][num_kv_heads][2]``, those or int8, a scale for each
block and kv head.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import warnings
from typing import Optional, Tuple

__all__ = [
    "PKVError", "lib_path", "load", "version", "status_string", "cache_write", "cache_append", "cache_read",
    "copy_blocks",
    "decode_workspace_size", "decode_attention", "decode_step", "prefill_workspace_size",
    "chunked_prefill_attention",
    "rotary", "rotary_cache_write", "linear_decode_attention", "linear_prefill_attention",
    "linear_prefill_workspace_size",
    "get_error", "Cache", "Blocks", "prefix_keys", "swap_out", "swap_in", "test_arm_decode_stall",
    "test_arm_prefill_stall",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libpagedkv.so")
_lib = None
_calls = None

PKV_OK = 0
STATUS_NAMES = {
    0: "PKV_OK", 1: "PKV_ERR_NULL", 2: "PKV_ERR_SHAPE", 3: "PKV_ERR_HEADS", 4: "PKV_ERR_HEADDIM",
    5: "PKV_ERR_BLOCKSIZE", 6: "PKV_ERR_ALIAS", 7: "PKV_ERR_WORKSPACE", 8: "PKV_ERR_ALIGN", 9: "PKV_ERR_RANGE",
    10: "PKV_ERR_TIMEOUT", 11: "PKV_ERR_CUDA", 12: "PKV_ERR_UNSUPPORTED", 13: "PKV_ERR_SCRATCH_LIMIT",
    14: "PKV_ERR_NO_BLOCKS", 15: "PKV_ERR_HOST_MEMORY", 16: "PKV_ERR_DTYPE",
}
PKV_KV_BF16, PKV_KV_E4M3, PKV_KV_E4M3_BLOCKS, PKV_KV_INT8_BLOCKS = 0, 1, 2, 3
PKV_ROTARY_ADJACENT_PAIRS, PKV_ROTARY_INTERLEAVED_AXES = 1, 2


class PKVError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = int(status)
        msg = status_string(status) if _lib is not None else STATUS_NAMES.get(status, str(status))
        if self.status == 11 and _lib is not None:
            msg += f" ({_lib.pkv_last_cuda_error().decode()})"
        super().__init__(f"{what}: {msg}" if what else msg)


class Cache(ctypes.Structure):
    """Mirror of ``pkv_cache_t``."""
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("num_blocks", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
                ("block_scales", ctypes.c_void_p)]


class BlocksState(ctypes.Structure):
    """Mirror of ``pkv_blocks_t``."""
    _fields_ = [("block_tables", ctypes.c_void_p), ("context_lens", ctypes.c_void_p),
                ("ref_counts", ctypes.c_void_p), ("free_ring", ctypes.c_void_p), ("ring_pos", ctypes.c_void_p),
                ("free_state", ctypes.c_void_p), ("scratch", ctypes.c_void_p), ("block_keys", ctypes.c_void_p),
                ("key_table", ctypes.c_void_p), ("cached", ctypes.c_void_p), ("num_blocks", ctypes.c_int32),
                ("max_seqs", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32), ("table_size", ctypes.c_int32)]


_Sections = ctypes.c_int32 * 4


class Rotary(ctypes.Structure):
    """Mirror of ``pkv_rotary_t``."""
    _fields_ = [("inv_freq", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("num_axes", ctypes.c_int32), ("sections", _Sections), ("flags", ctypes.c_int32)]


class States(ctypes.Structure):
    """Mirror of ``pkv_states_t``."""
    _fields_ = [("states", ctypes.c_void_p), ("log_decay", ctypes.c_void_p), ("num_slots", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


def lib_path() -> str:
    return _LIB_PATH


def load():
    """Load libpagedkv.so (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"libpagedkv.so is not built ({_LIB_PATH}); run `python -m "
                           "paged_kv_cache_291_gb300.build` or __graft_entry__.build() first")
    lib = ctypes.CDLL(_LIB_PATH)
    P, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    i64 = ctypes.c_int64
    CP = ctypes.POINTER(Cache)
    sigs = {
        "pkv_cache_write": ([CP, P, P, P, i32, P], ctypes.c_int),
        "pkv_cache_append": ([CP, P, i64, P, i64, i32, P, P, i32, P, i32, P], ctypes.c_int),
        "pkv_cache_read": ([CP, P, P, i32, P, P, i32, P, i32, P], ctypes.c_int),
        "pkv_copy_blocks": ([CP, P, P, i32, P, P, P], ctypes.c_int),
        "pkv_decode_workspace_size": ([i32, i32, i32, i32, i32, i32], sz),
        "pkv_decode_attention": ([CP, P, i32, P, i32, P, i32, i32, f32, P, P, sz, i32, P], ctypes.c_int),
        "pkv_decode_step": ([CP, P, P, P, P, i32, P, i32, P, i32, i32, f32, P, P, sz, i32, P], ctypes.c_int),
        "pkv_decode_shared_prefix_workspace_size": ([i32, i32, i32, i32, i32, i32], sz),
        "pkv_decode_attention_shared_prefix": ([CP, P, i32, P, i32, P, i32, i32, i32, f32, P, P, sz, P],
                                               ctypes.c_int),
        "pkv_common_prefix_blocks": ([P, i32, P, i32], i32),
        "pkv_copy": ([P, P, sz, P], ctypes.c_int),
        "pkv_prefill_workspace_size": ([i32, i32, i32, i32, i32, i32], sz),
        "pkv_chunked_prefill_attention": ([CP, P, i32, i32, P, P, P, i32, P, i32, i32, f32, P, P, sz, P],
                                          ctypes.c_int),
        "pkv_blocks_reset": ([ctypes.POINTER(BlocksState), P], ctypes.c_int),
        "pkv_blocks_append": ([ctypes.POINTER(BlocksState), P, i32, i32, P, P, P, P, P], ctypes.c_int),
        "pkv_blocks_fork": ([ctypes.POINTER(BlocksState), P, P, i32, P], ctypes.c_int),
        "pkv_blocks_release": ([ctypes.POINTER(BlocksState), P, i32, P], ctypes.c_int),
        "pkv_blocks_match": ([ctypes.POINTER(BlocksState), P, i32, P, i32, P, P], ctypes.c_int),
        "pkv_blocks_register": ([ctypes.POINTER(BlocksState), P, i32, P, i32, P], ctypes.c_int),
        "pkv_prefix_keys": ([P, P, P, P, i32, i32, P, P], ctypes.c_int),
        "pkv_swap_blocks": ([CP, i32, P, P, i32, P, ctypes.c_int64, P], ctypes.c_int),
        "pkv_rotary": ([ctypes.POINTER(Rotary), P, i64, i32, P, i64, i32, i32, i32, P, P, P], ctypes.c_int),
        "pkv_rotary_cache_write": ([CP, ctypes.POINTER(Rotary), P, i64, i32, P, i64, P, i64, P, i32, P, P],
                                   ctypes.c_int),
        "pkv_linear_decode_attention": ([ctypes.POINTER(States), P, i64, i32, P, i64, P, i64, P, P, P, i32, f32, P,
                                         P], ctypes.c_int),
        "pkv_linear_prefill_workspace_size": ([i32, i32, i32, i32, i32], sz),
        "pkv_linear_prefill_attention": ([ctypes.POINTER(States), P, i64, i32, P, i64, P, i64, i32, P, P, P, P, P, i32,
                                          f32, P, P, sz, P], ctypes.c_int),
        "pkv_get_error": ([P, ctypes.POINTER(i32)], ctypes.c_int),
        "pkv_test_arm_decode_stall": ([i32], ctypes.c_int),
        "pkv_test_arm_prefill_stall": ([i32], ctypes.c_int),
        "pkv_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "pkv_last_cuda_error": ([], ctypes.c_char_p),
        "pkv_version": ([], ctypes.c_char_p),
    }
    for name, (argt, rest) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = argt
        fn.restype = rest
    _lib = lib
    return lib


class _NoCalls:
    """In place of the compiled calls, where they cannot be loaded."""

    @staticmethod
    def rotary(*args):
        return None

    rotary_cache_write = linear_decode = linear_prefill = rotary
    cache_append = cache_read = decode_scaled = prefill_scaled = rotary


def _fast():
    """The compiled calls (csrc/binding.cpp).  Each returns the status of a
    plain valid call it has made, or None without having launched anything:
    then the wrapper's own checks say what is wrong, or it makes the call.
    The module belongs to the torch it was built against; without it, which
    is said once, the wrappers make every call of the library themselves."""
    global _calls
    if _calls is None:
        load()
        try:
            from . import _binding
            _calls = _binding
        except ImportError as e:
            warnings.warn("the package's _binding module is not built for this torch, so calls take longer on the "
                          f"host; run `python -m paged_kv_cache_291_gb300.build` ({e})", RuntimeWarning, stacklevel=3)
            _calls = _NoCalls
    return _calls


def version() -> str:
    return load().pkv_version().decode()


def status_string(status: int) -> str:
    return load().pkv_status_string(int(status)).decode()


# ---------------------------------------------------------------- helpers

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream_handle(stream) -> ctypes.c_void_p:
    torch = _torch()
    if stream is None:
        # the raw handle of torch.cuda.current_stream(), without building the object
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()))
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


_CURRENT = contextlib.nullcontext()


def _on(stream):
    """Makes the stream a call launches on torch's current one, for what the
    call allocates and reads back: torch then hands the memory of a workspace
    that the call lets go of to later work on that stream only, and what it
    hands out is free of earlier work there."""
    if stream is None:
        return _CURRENT
    torch = _torch()
    if not isinstance(stream, torch.cuda.Stream):  # an object with a handle, or the handle
        handle = _stream_handle(stream).value
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _dev(t, name, elem_size=None, dtype=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if elem_size is not None and t.element_size() != elem_size:
        raise TypeError(f"{name} must have {elem_size}-byte elements")
    return ctypes.c_void_p(t.data_ptr())


def _out(t, name="out"):
    """An fp32 output tensor on the device or in page-locked host memory
    (``pin_memory()``), which the kernels then write directly."""
    torch = _torch()
    if isinstance(t, torch.Tensor) and not t.is_cuda:
        if not t.is_pinned():
            raise ValueError(f"{name} must be a CUDA tensor or page-locked host memory")
        if not t.is_contiguous() or t.dtype != torch.float32:
            raise ValueError(f"{name} must be contiguous float32")
        return ctypes.c_void_p(t.data_ptr())
    return _dev(t, name, dtype=torch.float32)


def _cache(k_pool, v_pool, k_scale=None, v_scale=None, need_scales=False, block_scales=None) -> Cache:
    """Descriptor of a pool pair: 2-byte elements are bf16, 1-byte elements
    (uint8 or float8_e4m3fn) e4m3 codes with one scale per pool, or, with
    block_scales, e4m3 or int8 codes with a scale per (block, kv head)."""
    if k_pool.shape != v_pool.shape or k_pool.dim() != 4:
        raise ValueError("k_pool and v_pool must both be [num_blocks][num_kv_heads][16][head_dim]")
    nb, hkv, bs, d = k_pool.shape
    es = k_pool.element_size()
    if es not in (1, 2):
        raise TypeError("pools must have 2-byte (bf16) or 1-byte (e4m3) elements")
    if block_scales is not None:
        torch = _torch()
        if k_pool.dtype not in (torch.int8, torch.uint8, torch.float8_e4m3fn) or v_pool.dtype != k_pool.dtype:
            raise TypeError("pools with block_scales must both be int8, or e4m3 codes (uint8 or float8_e4m3fn)")
        if k_scale is not None or v_scale is not None:
            raise ValueError("a pool has block_scales or k_scale and v_scale, not both")
        if tuple(block_scales.shape) != (nb, hkv, 2):
            raise ValueError("block_scales must be [num_blocks][num_kv_heads][2]")
        if not k_pool.get_device() == v_pool.get_device() == block_scales.get_device() == _device():
            raise ValueError("the pools and block_scales must be on the current device")
        return Cache(_dev(k_pool, "k_pool").value, _dev(v_pool, "v_pool").value, nb, hkv, d, bs,
                     PKV_KV_INT8_BLOCKS if k_pool.dtype == torch.int8 else PKV_KV_E4M3_BLOCKS, 1.0, 1.0,
                     _dev(block_scales, "block_scales", dtype=torch.float32).value)
    if _torch().int8 in (k_pool.dtype, v_pool.dtype):
        raise TypeError("an int8 pool needs block_scales")  # its codes are not e4m3's, and mean nothing without them
    if es == 1 and need_scales and (k_scale is None or v_scale is None):
        raise ValueError("an e4m3 pool needs k_scale and v_scale")
    return Cache(_dev(k_pool, "k_pool", es).value, _dev(v_pool, "v_pool", es).value, nb, hkv, d, bs,
                 PKV_KV_E4M3 if es == 1 else PKV_KV_BF16,
                 1.0 if k_scale is None else float(k_scale), 1.0 if v_scale is None else float(v_scale))


def _check(status, what):
    if status != PKV_OK:
        raise PKVError(status, what)


def _host_i32(x):
    import numpy as np
    a = np.ascontiguousarray(x.cpu().numpy() if hasattr(x, "cpu") else x, dtype=np.int32)
    return a, a.ctypes.data_as(ctypes.c_void_p)


# ---------------------------------------------------------------- calls

def cache_write(k_pool, v_pool, k_new, v_new, slot_mapping, stream=None, k_scale=None, v_scale=None) -> None:
    """Store rows k_new/v_new [T][Hkv][d] at ``slot_mapping`` [T] (negative = skip).
    e4m3 pools (1-byte elements) store code(x * (1/scale)) and need the scales."""
    torch = _torch()
    lib = load()
    c = _cache(k_pool, v_pool, k_scale, v_scale, need_scales=True)
    T = int(slot_mapping.shape[0])
    if k_new.shape != (T, c.num_kv_heads, c.head_dim) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [num_tokens][num_kv_heads][head_dim]")
    st = lib.pkv_cache_write(ctypes.byref(c), _dev(k_new, "k_new", 2), _dev(v_new, "v_new", 2),
                             _dev(slot_mapping, "slot_mapping", dtype=torch.int32), T, _stream_handle(stream))
    _check(st, "pkv_cache_write")


def _cache_rows(k_pool, v_pool, query_start_loc, context_lens, block_tables, k_scale, v_scale, block_scales, dev):
    """Descriptor and index arguments of cache_append and cache_read."""
    i32 = _torch().int32
    c = _cache(k_pool, v_pool, k_scale, v_scale, need_scales=True, block_scales=block_scales)
    if k_pool.get_device() != dev or v_pool.get_device() != dev:
        raise ValueError(f"the pools are on {k_pool.device} and {v_pool.device}, the current device is cuda:{dev}")
    if context_lens.dim() != 1 or block_tables.dim() != 2:
        raise ValueError("context_lens must be [num_seqs] and block_tables [num_seqs][max_blocks]")
    S, wide = context_lens.shape[0], block_tables.shape[1]
    return c, (_addr(query_start_loc, "query_start_loc", i32, dev, (S + 1,)),
               _addr(context_lens, "context_lens", i32, dev, (S,)), S,
               _addr(block_tables, "block_tables", i32, dev, (S, wide)), wide)


def cache_append(k_pool, v_pool, block_scales, k_new, v_new, query_start_loc, context_lens, block_tables,
                 stream=None) -> None:
    """Store rows k_new/v_new [T][Hkv][d] (bf16; a token's rows may be a view
    of a packed projection) in 8 bits at the ends of their sequences'
    contexts, with a scale for each (block, kv head): sequence s owns rows
    query_start_loc[s] .. query_start_loc[s+1]-1, and context_lens[s] counts
    them.  The pools are int8, or e4m3 codes (uint8 or float8_e4m3fn), and
    block_scales float32 [num_blocks][Hkv][2] (K, V).  A block whose scale has
    to grow has its earlier rows encoded again."""
    if block_scales is None:
        raise ValueError("cache_append needs block_scales; pools without them take cache_write")
    st = _fast().cache_append(k_pool, v_pool, block_scales, k_new, v_new, query_start_loc, context_lens, block_tables,
                              stream)
    if st == PKV_OK:
        return
    if st is not None:
        raise PKVError(st, "pkv_cache_append")
    torch = _torch()
    lib = load()
    dev = _device()
    c, index = _cache_rows(k_pool, v_pool, query_start_loc, context_lens, block_tables, None, None, block_scales, dev)
    shape = (k_new.shape[0], c.num_kv_heads, c.head_dim)
    kp, ks = _rows(k_new, "k_new", torch.bfloat16, dev, shape)
    vp, vs = _rows(v_new, "v_new", torch.bfloat16, dev, shape)
    st = lib.pkv_cache_append(ctypes.byref(c), kp, ks, vp, vs, shape[0], *index, _stream_handle(stream))
    if st:
        _check(st, "pkv_cache_append")


def cache_read(k_pool, v_pool, query_start_loc, context_lens, block_tables, num_tokens: int, k_out=None, v_out=None,
               k_scale=None, v_scale=None, block_scales=None, stream=None):
    """Rows of the cache back as bf16, from pools of any kind: sequence s
    takes rows query_start_loc[s] .. query_start_loc[s+1]-1 of the outputs
    [num_tokens][Hkv][d] for the last rows of its context.  Returns (k_out,
    v_out)."""
    torch = _torch()
    shape = (int(num_tokens), k_pool.shape[1], k_pool.shape[3])
    if k_out is None or v_out is None:
        with _on(stream):
            k_out = torch.empty(shape, dtype=torch.bfloat16, device=k_pool.device) if k_out is None else k_out
            v_out = torch.empty(shape, dtype=torch.bfloat16, device=k_pool.device) if v_out is None else v_out
    if block_scales is not None and k_scale is None and v_scale is None:
        st = _fast().cache_read(k_pool, v_pool, block_scales, query_start_loc, context_lens, block_tables, shape[0],
                                k_out, v_out, stream)
        if st == PKV_OK:
            return k_out, v_out
        if st is not None:
            raise PKVError(st, "pkv_cache_read")
    lib = load()
    dev = _device()
    c, index = _cache_rows(k_pool, v_pool, query_start_loc, context_lens, block_tables, k_scale, v_scale,
                           block_scales, dev)
    st = lib.pkv_cache_read(ctypes.byref(c), _addr(k_out, "k_out", torch.bfloat16, dev, shape),
                            _addr(v_out, "v_out", torch.bfloat16, dev, shape), shape[0], *index,
                            _stream_handle(stream))
    if st:
        _check(st, "pkv_cache_read")
    return k_out, v_out


def copy_blocks(k_pool, v_pool, src, dst, check_host: bool = True, src_host=None, dst_host=None,
                stream=None, block_scales=None) -> None:
    """Copy-on-write: pool[dst[i]] <- pool[src[i]] (K and V, whole blocks,
    with their block_scales where the pool has them).

    The library rejects aliasing destinations before launching when it gets
    host copies of the id lists: pass them as ``src_host``/``dst_host``, or
    leave ``check_host`` on to have them copied from the device tensors
    (which synchronises).
    """
    torch = _torch()
    lib = load()
    c = _cache(k_pool, v_pool, block_scales=block_scales)
    n = int(src.shape[0])
    if dst.shape[0] != n:
        raise ValueError("src and dst must have the same length")
    sh = dh = None
    sp = dp = None
    if src_host is not None and dst_host is not None:
        sh, sp = _host_i32(src_host)
        dh, dp = _host_i32(dst_host)
        if sh.shape[0] != n or dh.shape[0] != n:
            raise ValueError("host id lists must match the device ones")
    elif check_host:
        with _on(stream):
            sh, sp = _host_i32(src)
            dh, dp = _host_i32(dst)
    st = lib.pkv_copy_blocks(ctypes.byref(c), _dev(src, "src", dtype=torch.int32),
                             _dev(dst, "dst", dtype=torch.int32), n, sp, dp, _stream_handle(stream))
    _check(st, "pkv_copy_blocks")


def decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                          partition_blocks=0) -> int:
    n = load().pkv_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                                         partition_blocks)
    if n == 0:
        raise PKVError(2, "pkv_decode_workspace_size")
    return int(n)


def new_workspace(nbytes: int, device=None):
    """A zero-filled, 256-byte aligned workspace (torch allocations are)."""
    torch = _torch()
    return torch.zeros(max(256, (nbytes + 255) // 256 * 256), dtype=torch.uint8, device=device or "cuda")


def decode_attention(k_pool, v_pool, q, block_tables, context_lens, max_context_len: int, scale: float,
                     out=None, workspace=None, partition_blocks: int = 0, stream=None, k_scale=None,
                     v_scale=None, block_scales=None):
    """Paged decode attention; returns ``out`` float32 [B][Hq][d].  8-bit pools
    (1-byte elements) need the scales they were written with."""
    if block_scales is not None:
        return _decode_scaled(k_pool, v_pool, q, block_tables, context_lens, max_context_len, scale, out, workspace,
                              partition_blocks, stream, k_scale, v_scale, block_scales)
    torch = _torch()
    lib = load()
    c = _cache(k_pool, v_pool, k_scale, v_scale, need_scales=True)
    B, hq, d = q.shape
    if d != c.head_dim:
        raise ValueError("q head_dim does not match the pools")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("block_tables must be [B][max_blocks] and context_lens [B]")
    if out is None:
        with _on(stream):
            out = torch.empty((B, hq, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = load().pkv_decode_workspace_size(B, hq, c.num_kv_heads, d, int(max_context_len),
                                                int(partition_blocks))
        with _on(stream):
            workspace = new_workspace(need, q.device)  # a size of 0 means bad arguments: the call reports them
    st = lib.pkv_decode_attention(ctypes.byref(c), _dev(q, "q", 2), hq,
                                  _dev(block_tables, "block_tables", dtype=torch.int32), int(block_tables.shape[1]),
                                  _dev(context_lens, "context_lens", dtype=torch.int32), B, int(max_context_len),
                                  float(scale), _out(out),
                                  _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
                                  int(partition_blocks), _stream_handle(stream))
    _check(st, "pkv_decode_attention")
    return out


def _decode_scaled(k_pool, v_pool, q, block_tables, context_lens, max_context_len, scale, out, workspace,
                   partition_blocks, stream, k_scale, v_scale, block_scales):
    """:func:`decode_attention` over pools with a scale per block."""
    torch = _torch()
    if k_scale is not None or v_scale is not None:
        raise ValueError("a pool has block_scales or k_scale and v_scale, not both")
    if out is None:
        with _on(stream):
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if workspace is None:
        need = load().pkv_decode_workspace_size(q.shape[0], q.shape[1], k_pool.shape[1], q.shape[2],
                                                int(max_context_len), int(partition_blocks))
        with _on(stream):
            workspace = new_workspace(need, q.device)
    st = _fast().decode_scaled(k_pool, v_pool, block_scales, q, block_tables, context_lens, max_context_len, scale, out,
                               workspace, partition_blocks, stream)
    if st == PKV_OK:
        return out
    if st is not None:
        raise PKVError(st, "pkv_decode_attention")
    lib = load()
    dev = _device()
    c = _cache(k_pool, v_pool, block_scales=block_scales)
    B, hq, d = q.shape
    if d != c.head_dim:
        raise ValueError("q head_dim does not match the pools")
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [B][max_blocks]")
    i32, wide = torch.int32, block_tables.shape[1]
    st = lib.pkv_decode_attention(ctypes.byref(c), _addr(q, "q", torch.bfloat16, dev, (B, hq, d)), hq,
                                  _addr(block_tables, "block_tables", i32, dev, (B, wide)), wide,
                                  _addr(context_lens, "context_lens", i32, dev, (B,)), B, int(max_context_len),
                                  float(scale), _out_addr(out, dev, q.shape),
                                  _addr(workspace, "workspace", workspace.dtype, dev, workspace.shape),
                                  workspace.nbytes, int(partition_blocks), _stream_handle(stream))
    _check(st, "pkv_decode_attention")
    return out


def decode_step(k_pool, v_pool, k_new, v_new, slot_mapping, q, block_tables, context_lens, max_context_len: int,
                scale: float, out=None, workspace=None, partition_blocks: int = 0, stream=None, k_scale=None,
                v_scale=None):
    """One decode step in one launch: store row s of k_new/v_new [B][Hkv][d]
    at slot_mapping[s] (the slot of position context_lens[s] - 1; negative =
    skip) and attend over the context; returns ``out`` float32 [B][Hq][d]."""
    torch = _torch()
    lib = load()
    c = _cache(k_pool, v_pool, k_scale, v_scale, need_scales=True)
    B, hq, d = q.shape
    if d != c.head_dim:
        raise ValueError("q head_dim does not match the pools")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("block_tables must be [B][max_blocks] and context_lens [B]")
    if k_new.shape != (B, c.num_kv_heads, d) or v_new.shape != k_new.shape or slot_mapping.shape[0] != B:
        raise ValueError("k_new/v_new must be [B][num_kv_heads][head_dim] and slot_mapping [B]")
    if out is None:
        with _on(stream):
            out = torch.empty((B, hq, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = lib.pkv_decode_workspace_size(B, hq, c.num_kv_heads, d, int(max_context_len), int(partition_blocks))
        with _on(stream):
            workspace = new_workspace(need, q.device)
    st = lib.pkv_decode_step(ctypes.byref(c), _dev(k_new, "k_new", 2), _dev(v_new, "v_new", 2),
                             _dev(slot_mapping, "slot_mapping", dtype=torch.int32), _dev(q, "q", 2), hq,
                             _dev(block_tables, "block_tables", dtype=torch.int32), int(block_tables.shape[1]),
                             _dev(context_lens, "context_lens", dtype=torch.int32), B, int(max_context_len),
                             float(scale), _out(out), _dev(workspace, "workspace"),
                             workspace.numel() * workspace.element_size(), int(partition_blocks),
                             _stream_handle(stream))
    _check(st, "pkv_decode_step")
    return out


def copy(dst, src, stream=None) -> None:
    """Copy the bytes of tensor ``src`` into tensor ``dst`` (same byte size,
    contiguous) with a kernel; either may be on the device or in page-locked
    host memory (``pin_memory()``), which the GPU then reads or writes
    directly (pkv_copy)."""
    if not (dst.is_contiguous() and src.is_contiguous()):
        raise ValueError("copy needs contiguous tensors")
    nbytes = dst.numel() * dst.element_size()
    if nbytes != src.numel() * src.element_size():
        raise ValueError("copy needs tensors of the same byte size")
    st = load().pkv_copy(ctypes.c_void_p(dst.data_ptr()), ctypes.c_void_p(src.data_ptr()), nbytes,
                         _stream_handle(stream))
    _check(st, "pkv_copy")


def common_prefix_blocks(block_tables_host, context_lens_host) -> int:
    """The largest J such that every row of the host block table
    [B][max_blocks] starts with row 0's first J ids and every context holds
    16 J tokens (pkv_common_prefix_blocks; host arrays only)."""
    import numpy as np
    t = np.ascontiguousarray(block_tables_host, dtype=np.int32)
    n = np.ascontiguousarray(context_lens_host, dtype=np.int32)
    if t.ndim != 2 or n.ndim != 1 or n.shape[0] != t.shape[0]:
        raise ValueError("block_tables_host must be [B][max_blocks] and context_lens_host [B]")
    return int(load().pkv_common_prefix_blocks(t.ctypes.data, t.shape[1], n.ctypes.data, t.shape[0]))


def decode_shared_prefix_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                                        shared_blocks) -> int:
    n = load().pkv_decode_shared_prefix_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                       max_context_len, shared_blocks)
    if n == 0:
        raise PKVError(2, "pkv_decode_shared_prefix_workspace_size")
    return int(n)


def decode_attention_shared_prefix(k_pool, v_pool, q, block_tables, context_lens, max_context_len: int,
                                   shared_blocks: int, scale: float, out=None, workspace=None, stream=None,
                                   k_scale=None, v_scale=None, block_scales=None):
    """Decode attention for a batch whose block tables all start with the
    same ``shared_blocks`` full blocks: those are read once per kv head for
    every sequence (tensor cores), the rest per sequence; returns ``out``
    float32 [B][Hq][d].  8-bit pools (with their scales) attend the shared
    blocks per sequence."""
    torch = _torch()
    lib = load()
    c = _cache(k_pool, v_pool, k_scale, v_scale, need_scales=True, block_scales=block_scales)
    B, hq, d = q.shape
    if d != c.head_dim:
        raise ValueError("q head_dim does not match the pools")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("block_tables must be [B][max_blocks] and context_lens [B]")
    if out is None:
        with _on(stream):
            out = torch.empty((B, hq, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = lib.pkv_decode_shared_prefix_workspace_size(B, hq, c.num_kv_heads, d, int(max_context_len),
                                                           int(shared_blocks))
        with _on(stream):
            workspace = new_workspace(need, q.device)
    st = lib.pkv_decode_attention_shared_prefix(
        ctypes.byref(c), _dev(q, "q", 2), hq, _dev(block_tables, "block_tables", dtype=torch.int32),
        int(block_tables.shape[1]), _dev(context_lens, "context_lens", dtype=torch.int32), B, int(max_context_len),
        int(shared_blocks), float(scale), _out(out), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream_handle(stream))
    _check(st, "pkv_decode_attention_shared_prefix")
    return out


def prefill_workspace_size(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, max_context_len) -> int:
    n = load().pkv_prefill_workspace_size(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim,
                                          max_context_len)
    if n == 0:
        raise PKVError(2, "pkv_prefill_workspace_size")
    return int(n)


def chunked_prefill_attention(k_pool, v_pool, q, query_start_loc, context_lens, block_tables,
                              max_context_len: int, scale: float, out=None, workspace=None,
                              query_start_loc_host=None, stream=None, block_scales=None):
    """Mixed batch of causal prefill chunks and decode rows; returns ``out``
    float32 [Tq][Hq][d].  Pools are bf16, or 8-bit with ``block_scales``."""
    if block_scales is not None:
        return _prefill_scaled(k_pool, v_pool, q, query_start_loc, context_lens, block_tables, max_context_len, scale,
                               out, workspace, query_start_loc_host, stream, block_scales)
    torch = _torch()
    lib = load()
    c = _cache(k_pool, v_pool)
    T, hq, d = q.shape
    S = int(context_lens.shape[0])
    if query_start_loc.shape[0] != S + 1:
        raise ValueError("query_start_loc must have num_seqs + 1 entries")
    if query_start_loc_host is None:
        query_start_loc_host = query_start_loc
    with _on(stream):
        qh, qhp = _host_i32(query_start_loc_host)
    if out is None:
        with _on(stream):
            out = torch.empty((T, hq, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = load().pkv_prefill_workspace_size(S, T, hq, c.num_kv_heads, d, int(max_context_len))
        with _on(stream):
            workspace = new_workspace(need, q.device)
    st = lib.pkv_chunked_prefill_attention(
        ctypes.byref(c), _dev(q, "q", 2), hq, T, _dev(query_start_loc, "query_start_loc", dtype=torch.int32), qhp,
        _dev(context_lens, "context_lens", dtype=torch.int32), S,
        _dev(block_tables, "block_tables", dtype=torch.int32), int(block_tables.shape[1]), int(max_context_len),
        float(scale), _out(out), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream_handle(stream))
    _check(st, "pkv_chunked_prefill_attention")
    return out


def _prefill_scaled(k_pool, v_pool, q, query_start_loc, context_lens, block_tables, max_context_len, scale, out,
                    workspace, query_start_loc_host, stream, block_scales):
    """:func:`chunked_prefill_attention` over pools with a scale per block."""
    torch = _torch()
    qh = query_start_loc if query_start_loc_host is None else query_start_loc_host
    if not isinstance(qh, torch.Tensor) or qh.is_cuda or qh.dtype is not torch.int32:
        with _on(stream):
            qh = torch.from_numpy(_host_i32(qh)[0])
    if out is None:
        with _on(stream):
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if workspace is None:
        need = load().pkv_prefill_workspace_size(context_lens.shape[0], q.shape[0], q.shape[1], k_pool.shape[1],
                                                 q.shape[2], int(max_context_len))
        with _on(stream):
            workspace = new_workspace(need, q.device)
    st = _fast().prefill_scaled(k_pool, v_pool, block_scales, q, query_start_loc, qh, context_lens, block_tables,
                                max_context_len, scale, out, workspace, stream)
    if st == PKV_OK:
        return out
    if st is not None:
        raise PKVError(st, "pkv_chunked_prefill_attention")
    lib = load()
    dev = _device()
    c = _cache(k_pool, v_pool, block_scales=block_scales)
    T, hq, d = q.shape
    S = context_lens.shape[0]
    if d != c.head_dim:
        raise ValueError("q head_dim does not match the pools")
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [num_seqs][max_blocks]")
    if tuple(qh.shape) != (S + 1,) or not qh.is_contiguous():
        raise ValueError("query_start_loc_host must have num_seqs + 1 entries")
    i32, wide = torch.int32, block_tables.shape[1]
    st = lib.pkv_chunked_prefill_attention(
        ctypes.byref(c), _addr(q, "q", torch.bfloat16, dev, (T, hq, d)), hq, T,
        _addr(query_start_loc, "query_start_loc", i32, dev, (S + 1,)), qh.data_ptr(),
        _addr(context_lens, "context_lens", i32, dev, (S,)), S,
        _addr(block_tables, "block_tables", i32, dev, (S, wide)), wide, int(max_context_len), float(scale),
        _out_addr(out, dev, q.shape), _addr(workspace, "workspace", workspace.dtype, dev, workspace.shape),
        workspace.nbytes, _stream_handle(stream))
    _check(st, "pkv_chunked_prefill_attention")
    return out


# The rotary and linear-attention calls, and those on pools with a scale per
# block, go through the compiled binding; what it hands back is checked and
# called here.

def _device() -> int:
    """The current device's index: the library launches there, so every
    tensor of a call has to be on it."""
    return _torch()._C._cuda_getDevice()


def _refuse(t, name, dtype, dev):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


def _addr(t, name, dtype, dev, shape) -> int:
    """Address of a contiguous CUDA tensor of the current device."""
    if not hasattr(t, "data_ptr") or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _rows(t, name, dtype, dev, shape):
    """Address and token stride (in elements) of rows [tokens][heads][d] whose
    tokens may lie further apart than their rows need (a view of a packed
    projection)."""
    if not hasattr(t, "data_ptr") or t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    tokens, heads, d = shape
    st, sh, sd = t.stride()
    if tokens and (sd != 1 or (sh != d and heads > 1)):
        raise ValueError(f"{name}: a token's heads and dims must be contiguous")
    return t.data_ptr(), st if tokens > 1 else heads * d


def _out_addr(t, dev, shape) -> int:
    """An fp32 output on the device or in page-locked host memory."""
    if t.shape != shape:
        raise ValueError(f"out must be {list(shape)}, got {list(t.shape)}")
    if t.get_device() != dev:
        if t.is_cuda:
            _refuse(t, "out", _torch().float32, dev)
        return _out(t)
    return _addr(t, "out", _torch().float32, dev, shape)


def _rotary(positions, inv_freq, sections, interleaved_axes, adjacent_pairs, tokens, dev) -> Rotary:
    torch = _torch()
    shape = positions.shape
    if len(shape) not in (1, 2):
        raise ValueError("positions must be [num_tokens] or [num_axes][num_tokens]")
    axes = 1 if len(shape) == 1 else shape[0]
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be [rot_dim / 2]")
    pairs = inv_freq.shape[0]
    if sections is None:
        if axes != 1:
            raise ValueError("several axes need sections")
        sections = (pairs,)
    if len(sections) != axes or axes > 4:
        raise ValueError("sections must name the pairs of each of at most 4 axes")
    flags = (PKV_ROTARY_ADJACENT_PAIRS if adjacent_pairs else 0) | (
        PKV_ROTARY_INTERLEAVED_AXES if interleaved_axes else 0)
    return Rotary(_addr(inv_freq, "inv_freq", torch.float32, dev, (pairs,)),
                  _addr(positions, "positions", torch.int32, dev, (tokens,) if len(shape) == 1 else (axes, tokens)),
                  2 * pairs, axes, _Sections(*sections), flags)


def rotary(q, k, positions, inv_freq, sections=None, interleaved_axes: bool = False, adjacent_pairs: bool = False,
           q_out=None, k_out=None, stream=None):
    """Turn q [T][Hq][d] and k [T][Hkv][d] (bf16; a token's rows may be a view
    of a packed projection) by positions int32 [T] or [axes][T]: pair i by
    positions[axis(i)] * inv_freq[i] (fp32 [rot_dim/2]).  ``sections`` names
    the pairs of each axis, in order or (``interleaved_axes``) dealt in turn;
    pairs are (i, i + rot_dim/2), or (2i, 2i + 1) with ``adjacent_pairs``.
    Returns (q_out, k_out), contiguous; q_out may be q and k_out k."""
    torch = _torch()
    if q_out is None:
        with _on(stream):
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if k_out is None:
        with _on(stream):
            k_out = torch.empty(k.shape, dtype=torch.bfloat16, device=k.device)
    st = _fast().rotary(q, k, positions, inv_freq, sections, interleaved_axes, adjacent_pairs, q_out, k_out, stream)
    if st == PKV_OK:
        return q_out, k_out
    if st is not None:
        raise PKVError(st, "pkv_rotary")
    lib = load()
    dev = _device()
    bf16 = torch.bfloat16
    qshape = T, hq, d = q.shape
    kshape = (T, k.shape[1], d)
    qp, qs = _rows(q, "q", bf16, dev, qshape)
    kp, ks = _rows(k, "k", bf16, dev, kshape)
    r = _rotary(positions, inv_freq, sections, interleaved_axes, adjacent_pairs, T, dev)
    st = lib.pkv_rotary(ctypes.byref(r), qp, qs, hq, kp, ks, kshape[1], d, T,
                        _addr(q_out, "q_out", bf16, dev, qshape), _addr(k_out, "k_out", bf16, dev, kshape),
                        _stream_handle(stream))
    if st:
        _check(st, "pkv_rotary")
    return q_out, k_out


def rotary_cache_write(k_pool, v_pool, q, k, v, slot_mapping, positions, inv_freq, sections=None,
                       interleaved_axes: bool = False, adjacent_pairs: bool = False, q_out=None, stream=None,
                       k_scale=None, v_scale=None):
    """:func:`rotary` and :func:`cache_write` in one launch: turned q to
    ``q_out`` (returned), turned k and v to their slots.  e4m3 pools need the
    scales; their codes come from the unrounded turned k."""
    torch = _torch()
    if q_out is None:
        with _on(stream):
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    st = _fast().rotary_cache_write(k_pool, v_pool, q, k, v, slot_mapping, positions, inv_freq, sections,
                                    interleaved_axes, adjacent_pairs, q_out, k_scale, v_scale, stream)
    if st == PKV_OK:
        return q_out
    if st is not None:
        raise PKVError(st, "pkv_rotary_cache_write")
    lib = load()
    dev = _device()
    bf16 = torch.bfloat16
    c = _cache(k_pool, v_pool, k_scale, v_scale, need_scales=True)
    if k_pool.get_device() != dev or v_pool.get_device() != dev:
        raise ValueError(f"the pools are on {k_pool.device} and {v_pool.device}, the current device is cuda:{dev}")
    qshape = T, hq, d = q.shape
    if d != c.head_dim:
        raise ValueError("q head_dim does not match the pools")
    kshape = (T, c.num_kv_heads, d)
    qp, qs = _rows(q, "q", bf16, dev, qshape)
    kp, ks = _rows(k, "k", bf16, dev, kshape)
    vp, vs = _rows(v, "v", bf16, dev, kshape)
    r = _rotary(positions, inv_freq, sections, interleaved_axes, adjacent_pairs, T, dev)
    st = lib.pkv_rotary_cache_write(ctypes.byref(c), ctypes.byref(r), qp, qs, hq, kp, ks, vp, vs,
                                    _addr(slot_mapping, "slot_mapping", torch.int32, dev, (T,)), T,
                                    _addr(q_out, "q_out", bf16, dev, qshape), _stream_handle(stream))
    if st:
        _check(st, "pkv_rotary_cache_write")
    return q_out


def _states(states, log_decay, d, dev) -> States:
    f32 = _torch().float32
    shape = states.shape
    if len(shape) != 4 or shape[2] != d or shape[3] != d:
        raise ValueError(f"states must be [num_slots][num_kv_heads][{d}][{d}] for q's head_dim, got {list(shape)}")
    return States(_addr(states, "states", f32, dev, shape), _addr(log_decay, "log_decay", f32, dev, (shape[1],)),
                  shape[0], shape[1], d)


def linear_decode_attention(states, log_decay, q, k, v, state_slots, context_lens, scale: float, new_slots=None,
                            out=None, stream=None):
    """Linear attention of one token per sequence: S <- exp(log_decay) S +
    k v^T in slot ``state_slots[s]`` of states float32 [slots][Hkv][d][d]
    (stored to ``new_slots[s]`` when given), out = scale q^T S, float32
    [B][Hq][d].  context_lens counts the token: 1 starts from a zero state,
    0 marks padding."""
    torch = _torch()
    if out is None:
        with _on(stream):
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    st = _fast().linear_decode(states, log_decay, q, k, v, state_slots, context_lens, scale, new_slots, out, stream)
    if st == PKV_OK:
        return out
    if st is not None:
        raise PKVError(st, "pkv_linear_decode_attention")
    lib = load()
    dev = _device()
    bf16, i32 = torch.bfloat16, torch.int32
    qshape = B, hq, d = q.shape
    s = _states(states, log_decay, d, dev)
    kshape, per_seq = (B, s.num_kv_heads, d), (B,)
    qp, qs = _rows(q, "q", bf16, dev, qshape)
    kp, ks = _rows(k, "k", bf16, dev, kshape)
    vp, vs = _rows(v, "v", bf16, dev, kshape)
    st = lib.pkv_linear_decode_attention(
        ctypes.byref(s), qp, qs, hq, kp, ks, vp, vs, _addr(state_slots, "state_slots", i32, dev, per_seq),
        None if new_slots is None else _addr(new_slots, "new_slots", i32, dev, per_seq),
        _addr(context_lens, "context_lens", i32, dev, per_seq), B, scale, _out_addr(out, dev, qshape),
        _stream_handle(stream))
    if st:
        _check(st, "pkv_linear_decode_attention")
    return out


def linear_prefill_workspace_size(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim) -> int:
    n = load().pkv_linear_prefill_workspace_size(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim)
    if n == 0:
        raise PKVError(2, "pkv_linear_prefill_workspace_size")
    return int(n)


def linear_prefill_attention(states, log_decay, q, k, v, query_start_loc, state_slots, context_lens, scale: float,
                             new_slots=None, out=None, workspace=None, query_start_loc_host=None, stream=None):
    """Linear attention of a mixed batch of prompt chunks and single tokens
    over their states (see :func:`linear_decode_attention`); returns ``out``
    float32 [T][Hq][d].  context_lens counts the call's tokens: a sequence
    starts from zero when it has no others."""
    torch = _torch()
    qh = query_start_loc if query_start_loc_host is None else query_start_loc_host
    if not isinstance(qh, torch.Tensor) or qh.is_cuda or qh.dtype is not torch.int32:
        with _on(stream):
            qh = torch.from_numpy(_host_i32(qh)[0])
    if out is None:
        with _on(stream):
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    if workspace is None:
        need = load().pkv_linear_prefill_workspace_size(context_lens.shape[0], q.shape[0], q.shape[1], k.shape[1],
                                                        q.shape[2])
        with _on(stream):
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    st = _fast().linear_prefill(states, log_decay, q, k, v, state_slots, context_lens, scale, new_slots, out, stream,
                                query_start_loc, qh, workspace)
    if st == PKV_OK:
        return out
    if st is not None:
        raise PKVError(st, "pkv_linear_prefill_attention")
    lib = load()
    dev = _device()
    bf16, i32 = torch.bfloat16, torch.int32
    qshape = T, hq, d = q.shape
    s = _states(states, log_decay, d, dev)
    S = context_lens.shape[0]
    kshape, per_seq = (T, s.num_kv_heads, d), (S,)
    qp, qs = _rows(q, "q", bf16, dev, qshape)
    kp, ks = _rows(k, "k", bf16, dev, kshape)
    vp, vs = _rows(v, "v", bf16, dev, kshape)
    if qh.shape != (S + 1,) or not qh.is_contiguous():
        raise ValueError("query_start_loc_host must have num_seqs + 1 entries")
    st = lib.pkv_linear_prefill_attention(
        ctypes.byref(s), qp, qs, hq, kp, ks, vp, vs, T,
        _addr(query_start_loc, "query_start_loc", i32, dev, (S + 1,)), qh.data_ptr(),
        _addr(state_slots, "state_slots", i32, dev, per_seq),
        None if new_slots is None else _addr(new_slots, "new_slots", i32, dev, per_seq),
        _addr(context_lens, "context_lens", i32, dev, per_seq), S, scale, _out_addr(out, dev, qshape),
        _addr(workspace, "workspace", workspace.dtype, dev, workspace.shape), workspace.nbytes, _stream_handle(stream))
    if st:
        _check(st, "pkv_linear_prefill_attention")
    return out


def _swap(direction, k_pool, v_pool, blocks, slots, host, stream, block_scales):
    torch = _torch()
    lib = load()
    c = _cache(k_pool, v_pool, block_scales=block_scales)
    n = int(blocks.shape[0])
    if slots.shape[0] != n:
        raise ValueError("blocks and slots must have the same length")
    if not isinstance(host, torch.Tensor) or host.is_cuda or not host.is_contiguous():
        raise ValueError("host must be a contiguous CPU tensor in page-locked memory")
    slab = 2 * c.num_kv_heads * 16 * c.head_dim * k_pool.element_size()
    if block_scales is not None:
        slab += (8 * c.num_kv_heads + 15) // 16 * 16
    if host.numel() * host.element_size() % slab:
        raise ValueError("host must hold whole slabs of [2][num_kv_heads][16][head_dim] pool elements, each followed "
                         "by the block's scales [num_kv_heads][2] up to 16 bytes where the pool has them")
    num_slots = host.numel() * host.element_size() // slab
    st = lib.pkv_swap_blocks(ctypes.byref(c), int(direction), _dev(blocks, "blocks", dtype=torch.int32),
                             _dev(slots, "slots", dtype=torch.int32), n, ctypes.c_void_p(host.data_ptr()),
                             num_slots, _stream_handle(stream))
    _check(st, "pkv_swap_blocks")


def swap_out(k_pool, v_pool, blocks, slots, host, stream=None, block_scales=None) -> None:
    """host slab slots[i] <- pool block blocks[i] (K then V); ``host`` is a
    pinned CPU tensor of whole [2][Hkv][16][d] slabs of the pools' elements,
    each followed by the block's scales, fp32 [Hkv][2], up to a multiple of 16
    bytes, where the pool has block_scales."""
    _swap(0, k_pool, v_pool, blocks, slots, host, stream, block_scales)


def swap_in(k_pool, v_pool, blocks, slots, host, stream=None, block_scales=None) -> None:
    """pool block blocks[i] <- host slab slots[i]."""
    _swap(1, k_pool, v_pool, blocks, slots, host, stream, block_scales)


def prefix_keys(token_ids, token_start_loc, max_blocks: int, extra=None, parent_keys=None, keys=None,
                stream=None):
    """Prefix-cache keys (uint8 [S][max_blocks][32]) of the full blocks of each
    token list: key_i = SHA-256(key_{i-1} || 16 token ids (<i4) || extra (<i8))."""
    torch = _torch()
    S = int(token_start_loc.shape[0]) - 1
    if keys is None:
        with _on(stream):
            keys = torch.zeros((max(S, 1), max(max_blocks, 1), 32), dtype=torch.uint8, device=token_ids.device)
    ep = _dev(extra, "extra", dtype=torch.int64) if extra is not None else None
    pp = _dev(parent_keys, "parent_keys", dtype=torch.uint8) if parent_keys is not None else None
    st = load().pkv_prefix_keys(_dev(token_ids, "token_ids", dtype=torch.int32),
                                _dev(token_start_loc, "token_start_loc", dtype=torch.int32), ep, pp, S,
                                int(max_blocks), _dev(keys, "keys", dtype=torch.uint8), _stream_handle(stream))
    _check(st, "pkv_prefix_keys")
    return keys


class Blocks:
    """Block bookkeeping state on one GPU (``pkv_blocks_t``): block tables,
    context lengths, reference counts and the ring of free blocks, as int32
    CUDA tensors owned by this object.  ``block_tables`` and ``context_lens``
    are the arrays the attention calls read.  Every method is one launch on
    the current stream; device-side errors are read with :func:`get_error`."""

    def __init__(self, num_blocks: int, max_seqs: int, max_blocks_per_seq: int, device=None,
                 prefix_cache: bool = False):
        torch = _torch()
        device = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        i32 = dict(dtype=torch.int32, device=device)
        self.num_blocks, self.max_seqs, self.max_blocks_per_seq = num_blocks, max_seqs, max_blocks_per_seq
        n1 = max(num_blocks, 1)
        self.block_tables = torch.empty((max_seqs, max_blocks_per_seq), **i32)
        self.context_lens = torch.empty((max_seqs,), **i32)
        self.ref_counts = torch.empty((n1,), **i32)
        self.free_ring = torch.empty((2 * n1,), **i32)
        self.ring_pos = torch.empty((n1,), **i32)
        self.free_state = torch.empty((3,), **i32)
        self.scratch = torch.empty((3 * n1,), **i32)
        self.table_size = 0
        self.block_keys = self.key_table = self.cached = None
        if prefix_cache:
            self.table_size = 1 << max(1, (2 * n1 - 1).bit_length())
            self.block_keys = torch.zeros((n1, 32), dtype=torch.uint8, device=device)
            self.key_table = torch.empty((self.table_size,), **i32)
            self.cached = torch.empty((n1,), **i32)
        self.reset()

    def _state(self) -> BlocksState:
        ptr = lambda t: t.data_ptr() if t is not None else None
        return BlocksState(self.block_tables.data_ptr(), self.context_lens.data_ptr(), self.ref_counts.data_ptr(),
                           self.free_ring.data_ptr(), self.ring_pos.data_ptr(), self.free_state.data_ptr(),
                           self.scratch.data_ptr(), ptr(self.block_keys), ptr(self.key_table), ptr(self.cached),
                           self.num_blocks, self.max_seqs, self.max_blocks_per_seq, self.table_size)

    def free_queue(self) -> list:
        """The free block ids, least recently freed first (synchronises)."""
        ring, pos = self.free_ring.cpu().tolist(), self.ring_pos.cpu().tolist()
        head, entries, _ = self.free_state.cpu().tolist()
        cap = 2 * self.num_blocks
        out = []
        for e in range(entries):
            idx = (head + e) % cap
            b = ring[idx]
            if 0 <= b < self.num_blocks and pos[b] == idx:
                out.append(b)
        return out

    def match(self, keys, num_keys, matched=None, stream=None):
        """Prefix-cache hits for empty rows: returns matched [S] (int32 CUDA)."""
        torch = _torch()
        S = int(num_keys.shape[0])
        if matched is None:
            with _on(stream):
                matched = torch.empty((max(S, 1),), dtype=torch.int32, device=self.block_tables.device)
        st = load().pkv_blocks_match(ctypes.byref(self._state()), _dev(keys, "keys", dtype=torch.uint8),
                                     int(keys.shape[1]), _dev(num_keys, "num_keys", dtype=torch.int32), S,
                                     _dev(matched, "matched", dtype=torch.int32), _stream_handle(stream))
        _check(st, "pkv_blocks_match")
        return matched

    def register(self, keys, num_keys, stream=None) -> None:
        """Give rows' full blocks their prefix-cache keys."""
        torch = _torch()
        st = load().pkv_blocks_register(ctypes.byref(self._state()), _dev(keys, "keys", dtype=torch.uint8),
                                        int(keys.shape[1]), _dev(num_keys, "num_keys", dtype=torch.int32),
                                        int(num_keys.shape[0]), _stream_handle(stream))
        _check(st, "pkv_blocks_register")

    def reset(self, stream=None) -> None:
        """Every row empty, every block free (queued 0, 1, 2, ...)."""
        _check(load().pkv_blocks_reset(ctypes.byref(self._state()), _stream_handle(stream)), "pkv_blocks_reset")

    def append(self, query_start_loc, num_tokens: int, slot_mapping=None, cow_src=None, cow_dst=None,
               cow_count=None, stream=None):
        """Row s gains query_start_loc[s+1] - query_start_loc[s] tokens.

        Returns (slot_mapping [num_tokens], cow_src [S], cow_dst [S],
        cow_count [1]) as int32 CUDA tensors (allocated when not given)."""
        torch = _torch()
        S = int(query_start_loc.shape[0]) - 1
        dev = self.block_tables.device
        i32 = dict(dtype=torch.int32, device=dev)
        with _on(stream):
            slot_mapping = slot_mapping if slot_mapping is not None else torch.empty((num_tokens,), **i32)
            cow_src = cow_src if cow_src is not None else torch.empty((max(S, 1),), **i32)
            cow_dst = cow_dst if cow_dst is not None else torch.empty((max(S, 1),), **i32)
            cow_count = cow_count if cow_count is not None else torch.empty((1,), **i32)
        if slot_mapping.shape[0] < num_tokens or cow_src.shape[0] < S or cow_dst.shape[0] < S:
            raise ValueError("output tensors are too small")
        sp = _dev(slot_mapping, "slot_mapping", dtype=torch.int32) if num_tokens > 0 else None
        st = load().pkv_blocks_append(ctypes.byref(self._state()),
                                      _dev(query_start_loc, "query_start_loc", dtype=torch.int32), S,
                                      int(num_tokens), sp, _dev(cow_src, "cow_src", dtype=torch.int32),
                                      _dev(cow_dst, "cow_dst", dtype=torch.int32),
                                      _dev(cow_count, "cow_count", dtype=torch.int32), _stream_handle(stream))
        _check(st, "pkv_blocks_append")
        return slot_mapping, cow_src, cow_dst, cow_count

    def fork(self, parents, children, stream=None) -> None:
        """Row children[i] takes row parents[i]'s blocks and length."""
        torch = _torch()
        n = int(parents.shape[0])
        if children.shape[0] != n:
            raise ValueError("parents and children must have the same length")
        st = load().pkv_blocks_fork(ctypes.byref(self._state()), _dev(parents, "parents", dtype=torch.int32),
                                    _dev(children, "children", dtype=torch.int32), n, _stream_handle(stream))
        _check(st, "pkv_blocks_fork")

    def release(self, rows, stream=None) -> None:
        """Rows drop their blocks (each row last block first) and end empty."""
        torch = _torch()
        st = load().pkv_blocks_release(ctypes.byref(self._state()), _dev(rows, "rows", dtype=torch.int32),
                                       int(rows.shape[0]), _stream_handle(stream))
        _check(st, "pkv_blocks_release")


def test_arm_decode_stall(launches: int) -> None:
    """Test hook: the next ``launches`` decode launches time out on purpose
    (their producer warp issues nothing; the bounded waits of the other warps
    expire after 2 s and record PKV_ERR_TIMEOUT).  0 disarms."""
    _check(load().pkv_test_arm_decode_stall(int(launches)), "pkv_test_arm_decode_stall")


def test_arm_prefill_stall(launches: int) -> None:
    """Test hook: the same for the next ``launches`` prefill launches (their
    tensor-core warp issues nothing)."""
    _check(load().pkv_test_arm_prefill_stall(int(launches)), "pkv_test_arm_prefill_stall")


def get_error(stream=None) -> Tuple[int, int]:
    """Synchronise the stream and return (status, detail) of the first
    device-side error since the last call, clearing it."""
    detail = ctypes.c_int32(0)
    st = load().pkv_get_error(_stream_handle(stream), ctypes.byref(detail))
    return int(st), int(detail.value)
