"""Paged KV-pool attention for GB300 (sm_103a): Python binding of libminisgl.so.

The C library (include/minisgl.h) does all the work in hand-written CUDA
kernels; this module only marshals torch tensors into pointers, sizes and the
current CUDA stream.  There is no fallback: if the library is not built, or a
call fails, an exception is raised.

Entry points (same names as the C ABI):
    minisgl_store_kv(pool, layer, k, v, out_loc)
    minisgl_decode_attn(pool, layer, q, page_table, seq_lens, sm_scale, ...)
    minisgl_extend_attn(pool, layer, q, page_table, cached_lens, extend_lens, q_offsets, sm_scale, ...)
    minisgl_rope_store_kv(pool, layer, q, k, v, positions, cos_sin_cache, out_loc)
    minisgl_check_indices(page_table, lens, num_rows, out_loc)   (debugging aid)
    minisgl_build_slots(cached_lens, extend_lens, page_table, free_pages, page_size, dummy_row, total_tokens)
    minisgl_store_kv_fp4(pool, layer, k, v, out_loc)                    (pool: a KVPoolFP4)
    minisgl_load_kv_fp4(pool, layer, page_table, lens, offsets, total_tokens)
    minisgl_decode_attn_fp4(pool, layer, q, page_table, seq_lens, sm_scale, ...)
"""
from __future__ import annotations

import ctypes
import operator
import os
from typing import List, NamedTuple, Optional, Sequence, Tuple, Union

import torch

from .build import LIB_PATH

__all__ = [
    "KVPool", "minisgl_store_kv", "minisgl_decode_attn", "minisgl_extend_attn",
    "minisgl_decode_workspace_bytes", "minisgl_device_sm_count", "minisgl_debug_timeout_count",
    "kv_pool_bytes", "load_library", "MinisglError", "EXPORTED_SYMBOLS",
    "minisgl_decode_attn_noalloc", "minisgl_rope_store_kv", "minisgl_cascade_decode_attn",
    "minisgl_cascade_workspace_bytes", "minisgl_store_decode_attn", "minisgl_check_indices",
    "minisgl_debug_set_pdl", "extend_work_counter", "minisgl_cascade_extend_attn",
    "minisgl_cascade_extend_workspace_bytes", "minisgl_check_shared_prefix",
    "KVPoolFP4", "Slots", "minisgl_build_slots", "minisgl_store_kv_fp4", "minisgl_load_kv_fp4",
    "minisgl_decode_attn_fp4", "decode_workspace_fp4", "kv_pool_fp4_bytes",
]

EXPORTED_SYMBOLS = [
    "minisgl_store_kv", "minisgl_decode_workspace_bytes", "minisgl_decode_attn",
    "minisgl_extend_attn", "minisgl_last_error", "minisgl_device_sm_count",
    "minisgl_debug_timeout_count", "minisgl_decode_attn_noalloc", "minisgl_rope_store_kv",
    "minisgl_cascade_decode_attn", "minisgl_cascade_workspace_bytes", "minisgl_store_decode_attn",
    "minisgl_check_indices", "minisgl_debug_set_pdl", "minisgl_cascade_extend_attn",
    "minisgl_cascade_extend_workspace_bytes", "minisgl_check_shared_prefix",
    "minisgl_build_slots", "minisgl_store_kv_fp4", "minisgl_load_kv_fp4", "minisgl_decode_attn_fp4",
]

MINISGL_BF16 = 1
MINISGL_FP4 = 2


class MinisglError(RuntimeError):
    pass


class _PoolDesc(ctypes.Structure):
    _fields_ = [
        ("k_base", ctypes.c_void_p), ("v_base", ctypes.c_void_p),
        ("layer_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
        ("num_layers", ctypes.c_int32), ("num_rows", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("dtype", ctypes.c_int32),
    ]


class _PoolFP4Desc(ctypes.Structure):
    _fields_ = [
        ("k_data", ctypes.c_void_p), ("v_data", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("data_layer_stride", ctypes.c_int64), ("data_row_stride", ctypes.c_int64),
        ("scale_layer_stride", ctypes.c_int64), ("scale_row_stride", ctypes.c_int64),
        ("num_layers", ctypes.c_int32), ("num_rows", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("k_exp", ctypes.c_int32), ("v_exp", ctypes.c_int32),
    ]


_lib: Optional[ctypes.CDLL] = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libminisgl.so (built by paged_kv_cache_row_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m paged_kv_cache_row_gb300.build`"
                          " (or __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    P = ctypes.POINTER(_PoolDesc)
    lib.minisgl_store_kv.argtypes = [P, i32, vp, vp, i64, i64, vp, i32, vp]
    lib.minisgl_store_kv.restype = ctypes.c_int
    lib.minisgl_decode_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.minisgl_decode_workspace_bytes.restype = sz
    lib.minisgl_decode_attn.argtypes = [P, i32, vp, i32, vp, i32, i64, i32, vp, f32, vp, vp, sz, i32, vp]
    lib.minisgl_decode_attn.restype = ctypes.c_int
    lib.minisgl_decode_attn_noalloc.argtypes = [P, i32, vp, i32, vp, i32, i64, i32, vp, f32, vp, i32, vp]
    lib.minisgl_decode_attn_noalloc.restype = ctypes.c_int
    lib.minisgl_extend_attn.argtypes = [P, i32, vp, i32, vp, i32, i64, i32, vp, vp, vp, i32, f32, vp, vp,
                                        vp]
    lib.minisgl_extend_attn.restype = ctypes.c_int
    lib.minisgl_rope_store_kv.argtypes = [P, i32, vp, i32, i64, vp, vp, i64, i64, vp, vp, i32, vp,
                                          i32, vp]
    lib.minisgl_rope_store_kv.restype = ctypes.c_int
    lib.minisgl_cascade_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.minisgl_cascade_workspace_bytes.restype = sz
    lib.minisgl_cascade_decode_attn.argtypes = [P, i32, vp, i32, vp, i32, i64, i32, vp, i32, f32, vp,
                                                vp, sz, vp]
    lib.minisgl_cascade_decode_attn.restype = ctypes.c_int
    lib.minisgl_store_decode_attn.argtypes = [P, i32, vp, vp, i64, i64, vp, vp, i32, vp, i32, i64, i32,
                                              vp, f32, vp, vp, sz, i32, vp]
    lib.minisgl_store_decode_attn.restype = ctypes.c_int
    lib.minisgl_check_indices.argtypes = [vp, i32, i64, i32, vp, vp, i32, i32, vp, vp]
    lib.minisgl_check_indices.restype = ctypes.c_int
    lib.minisgl_last_error.argtypes = []
    lib.minisgl_last_error.restype = ctypes.c_char_p
    lib.minisgl_device_sm_count.argtypes = []
    lib.minisgl_device_sm_count.restype = i32
    lib.minisgl_debug_timeout_count.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    lib.minisgl_debug_timeout_count.restype = ctypes.c_int
    lib.minisgl_cascade_extend_workspace_bytes.argtypes = [i32, i32, i32]
    lib.minisgl_cascade_extend_workspace_bytes.restype = sz
    lib.minisgl_cascade_extend_attn.argtypes = [P, i32, vp, i32, vp, i32, i64, i32, vp, vp, vp, i32, i32,
                                                f32, vp, vp, sz, vp]
    lib.minisgl_cascade_extend_attn.restype = ctypes.c_int
    lib.minisgl_check_shared_prefix.argtypes = [vp, i32, i64, i32, i32, vp, vp, vp]
    lib.minisgl_check_shared_prefix.restype = ctypes.c_int
    lib.minisgl_debug_set_pdl.argtypes = [ctypes.c_int]
    lib.minisgl_debug_set_pdl.restype = ctypes.c_int
    P4 = ctypes.POINTER(_PoolFP4Desc)
    lib.minisgl_build_slots.argtypes = [vp, vp, i32, vp, i64, i32, vp, i32, i32, i32, vp, vp, vp, vp, vp,
                                        i32, vp]
    lib.minisgl_build_slots.restype = ctypes.c_int
    lib.minisgl_store_kv_fp4.argtypes = [P4, i32, vp, vp, i64, i64, vp, i32, vp]
    lib.minisgl_store_kv_fp4.restype = ctypes.c_int
    lib.minisgl_load_kv_fp4.argtypes = [P4, i32, vp, i32, i64, i32, vp, vp, i32, vp, vp, i64, i64, vp]
    lib.minisgl_load_kv_fp4.restype = ctypes.c_int
    lib.minisgl_decode_attn_fp4.argtypes = [P4, i32, vp, i32, vp, i32, i64, i32, vp, f32, vp, vp, sz, i32,
                                            vp]
    lib.minisgl_decode_attn_fp4.restype = ctypes.c_int
    _lib = lib
    return lib


def _check(rc: int, what: str) -> None:
    if rc != 0:
        msg = load_library().minisgl_last_error().decode(errors="replace")
        raise MinisglError(f"{what} failed ({rc}): {msg}")


def _stream(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _rows_ok(t: torch.Tensor, n: int, row: int) -> bool:
    """True when t is [n, ...] and each t[i] is `row` contiguous elements
    (read from the shape and strides alone: indexing a tensor costs several
    microseconds of host time per call)."""
    if t.dim() < 2 or t.shape[0] != n:
        return False
    expect = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != expect:
            return False
        expect *= size
    return expect == row


def _need(t: torch.Tensor, name: str, dtype: torch.dtype) -> None:
    if not t.is_cuda:
        raise MinisglError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise MinisglError(f"{name} must be {dtype}, got {t.dtype}")


class KVPool:
    """A paged KV pool: one bf16 tensor of logical shape (2, L, R, H_kv, d).

    `tensor` may be LayerFirst (contiguous (2, L, R, H_kv, d)) or a permuted
    PageFirst view; only strides are read.  The pool is caller-owned device
    memory; the library keeps no reference to it."""

    def __init__(self, tensor: torch.Tensor, page_size: int = 1):
        if tensor.dim() != 5 or tensor.shape[0] != 2:
            raise MinisglError("pool tensor must have shape (2, L, R, H_kv, d)")
        _need(tensor, "pool", torch.bfloat16)
        if tensor.stride(4) != 1 or tensor.stride(3) != tensor.shape[4]:
            raise MinisglError("pool rows must be (H_kv, d) contiguous")
        self.tensor = tensor
        self.page_size = page_size
        _, L, R, H, d = tensor.shape
        self.num_layers, self.num_rows, self.num_kv_heads, self.head_dim = L, R, H, d
        self.desc = _PoolDesc(
            k_base=tensor[0].data_ptr(), v_base=tensor[1].data_ptr(),
            layer_stride=tensor.stride(1), row_stride=tensor.stride(2),
            num_layers=L, num_rows=R, num_kv_heads=H, head_dim=d, page_size=page_size,
            dtype=MINISGL_BF16)

    def k(self, layer: int) -> torch.Tensor:
        return self.tensor[0, layer]

    def v(self, layer: int) -> torch.Tensor:
        return self.tensor[1, layer]


def kv_pool_bytes(num_layers: int, num_kv_heads: int, head_dim: int, num_tokens: int,
                  elem_bytes: int = 2) -> int:
    """Bytes the pool needs to hold num_tokens token rows in every layer, K and V."""
    return 2 * num_layers * num_kv_heads * head_dim * num_tokens * elem_bytes


def minisgl_store_kv(pool: KVPool, layer: int, k: torch.Tensor, v: torch.Tensor,
                     out_loc: torch.Tensor, stream=None) -> None:
    """pool[K|V][layer][out_loc[i]] = k[i] | v[i] for every new token i (bit-exact)."""
    lib = load_library()
    _need(k, "k", torch.bfloat16)
    _need(v, "v", torch.bfloat16)
    _need(out_loc, "out_loc", torch.int32)
    n = out_loc.numel()
    row = pool.num_kv_heads * pool.head_dim
    for t, nm in ((k, "k"), (v, "v")):
        if not _rows_ok(t, n, row):
            raise MinisglError(f"{nm} must be [n_tokens, H_kv, d] with contiguous rows")
    if not out_loc.is_contiguous():
        raise MinisglError("out_loc must be contiguous")
    _check(lib.minisgl_store_kv(ctypes.byref(pool.desc), layer, _ptr(k), _ptr(v), k.stride(0),
                                v.stride(0), _ptr(out_loc), n, _stream(stream)), "store_kv")


def minisgl_decode_workspace_bytes(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                   max_splits: int = 16) -> int:
    return int(load_library().minisgl_decode_workspace_bytes(batch, num_q_heads, num_kv_heads,
                                                             head_dim, max_splits))


_ws_cache = {}


def decode_workspace(batch: int, num_q_heads: int, pool: KVPool, max_splits: int = 16,
                     device=None) -> torch.Tensor:
    """A workspace tensor for minisgl_decode_attn, cached per shape and device."""
    device = torch.device(device or pool.tensor.device)
    nbytes = minisgl_decode_workspace_bytes(batch, num_q_heads, pool.num_kv_heads, pool.head_dim,
                                            max_splits)
    key = (device, nbytes)
    ws = _ws_cache.get(key)
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    return ws


def minisgl_decode_attn(pool: KVPool, layer: int, q: torch.Tensor, page_table: torch.Tensor,
                        seq_lens: torch.Tensor, sm_scale: float, out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, split_tokens: int = 0,
                        max_splits: int = 16, stream=None) -> torch.Tensor:
    """Decode attention of q [B, H_q, d] over each request's page_table row."""
    lib = load_library()
    _need(q, "q", torch.bfloat16)
    _need(page_table, "page_table", torch.int32)
    _need(seq_lens, "seq_lens", torch.int32)
    B, Hq, d = q.shape
    if not q.is_contiguous() or d != pool.head_dim:
        raise MinisglError("q must be contiguous [B, H_q, head_dim]")
    if page_table.dim() != 2 or page_table.shape[0] != B or page_table.stride(1) != 1:
        raise MinisglError("page_table must be [B, W] with unit column stride")
    if seq_lens.numel() != B or not seq_lens.is_contiguous():
        raise MinisglError("seq_lens must be contiguous [B]")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16)
    if workspace is None:
        workspace = decode_workspace(B, Hq, pool, max_splits)
    _check(lib.minisgl_decode_attn(ctypes.byref(pool.desc), layer, _ptr(q), Hq, _ptr(page_table), B,
                                   page_table.stride(0), page_table.shape[1], _ptr(seq_lens),
                                   float(sm_scale), _ptr(out), _ptr(workspace), workspace.numel(),
                                   split_tokens, _stream(stream)), "decode_attn")
    return out


def minisgl_decode_attn_noalloc(pool: KVPool, layer: int, q: torch.Tensor, page_table: torch.Tensor,
                                seq_lens: torch.Tensor, sm_scale: float,
                                out: Optional[torch.Tensor] = None, split_tokens: int = 0,
                                stream=None) -> torch.Tensor:
    """minisgl_decode_attn without a workspace, for callers that cannot allocate
    device memory: the split-KV scratch comes from a fixed 32 MiB array inside
    the library (one per GPU, shared by all calls, so calls must not overlap on
    the GPU).  `out` must be given by a caller that cannot allocate; when it is
    None this wrapper allocates it with torch for convenience."""
    lib = load_library()
    _need(q, "q", torch.bfloat16)
    _need(page_table, "page_table", torch.int32)
    _need(seq_lens, "seq_lens", torch.int32)
    B, Hq, d = q.shape
    if not q.is_contiguous() or d != pool.head_dim:
        raise MinisglError("q must be contiguous [B, H_q, head_dim]")
    if page_table.dim() != 2 or page_table.shape[0] != B or page_table.stride(1) != 1:
        raise MinisglError("page_table must be [B, W] with unit column stride")
    if seq_lens.numel() != B or not seq_lens.is_contiguous():
        raise MinisglError("seq_lens must be contiguous [B]")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16)
    _check(lib.minisgl_decode_attn_noalloc(ctypes.byref(pool.desc), layer, _ptr(q), Hq,
                                           _ptr(page_table), B, page_table.stride(0),
                                           page_table.shape[1], _ptr(seq_lens), float(sm_scale),
                                           _ptr(out), split_tokens, _stream(stream)),
           "decode_attn_noalloc")
    return out


def minisgl_extend_attn(pool: KVPool, layer: int, q: torch.Tensor, page_table: torch.Tensor,
                        cached_lens: torch.Tensor, extend_lens: torch.Tensor,
                        q_offsets: torch.Tensor, sm_scale: float,
                        out: Optional[torch.Tensor] = None, work_counter: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """Causal extend attention of the packed new tokens q [T, H_q, d].
    work_counter: optional int32 CUDA tensor of 2 elements, zero before its
    first use (see extend_work_counter); calls that may run concurrently on
    different streams need different counters."""
    lib = load_library()
    _need(q, "q", torch.bfloat16)
    for t, nm in ((page_table, "page_table"), (cached_lens, "cached_lens"),
                  (extend_lens, "extend_lens"), (q_offsets, "q_offsets")):
        _need(t, nm, torch.int32)
    T, Hq, d = q.shape
    B = cached_lens.numel()
    if not q.is_contiguous() or d != pool.head_dim:
        raise MinisglError("q must be contiguous [T, H_q, head_dim]")
    if page_table.dim() != 2 or page_table.shape[0] != B or page_table.stride(1) != 1:
        raise MinisglError("page_table must be [B, W] with unit column stride")
    if extend_lens.numel() != B or q_offsets.numel() != B + 1:
        raise MinisglError("extend_lens must be [B] and q_offsets [B+1]")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16)
    if work_counter is not None:
        _need(work_counter, "work_counter", torch.int32)
        if work_counter.numel() < 2 or not work_counter.is_contiguous():
            raise MinisglError("work_counter must be a contiguous int32 tensor of 2 elements")
    _check(lib.minisgl_extend_attn(ctypes.byref(pool.desc), layer, _ptr(q), Hq, _ptr(page_table), B,
                                   page_table.stride(0), page_table.shape[1], _ptr(cached_lens),
                                   _ptr(extend_lens), _ptr(q_offsets), T, float(sm_scale), _ptr(out),
                                   _ptr(work_counter), _stream(stream)), "extend_attn")
    return out


def extend_work_counter(device=None) -> torch.Tensor:
    """A zeroed work counter for minisgl_extend_attn (8 bytes of device memory)."""
    return torch.zeros(2, dtype=torch.int32, device=device or "cuda")


def minisgl_device_sm_count() -> int:
    return int(load_library().minisgl_device_sm_count())


def minisgl_check_indices(page_table: torch.Tensor, lens: torch.Tensor, num_rows: int,
                          out_loc: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """Count, on the device, the index values a decode or extend call over
    these tensors would read that lie outside the pool: returns an int32 CUDA
    tensor [page-table entries, out_loc entries, lengths outside
    [0, page_table width]] (read it after the stream).  lens is seq_lens for
    decode, cached_lens + extend_lens for extend."""
    lib = load_library()
    _need(page_table, "page_table", torch.int32)
    _need(lens, "lens", torch.int32)
    if page_table.dim() != 2 or page_table.stride(1) != 1:
        raise MinisglError("page_table must be [B, W] with unit column stride")
    if lens.numel() != page_table.shape[0] or not lens.is_contiguous():
        raise MinisglError("lens must be a contiguous [B] tensor")
    n_out = 0
    if out_loc is not None:
        _need(out_loc, "out_loc", torch.int32)
        if not out_loc.is_contiguous():
            raise MinisglError("out_loc must be contiguous")
        n_out = out_loc.numel()
    if counts is None:
        counts = torch.empty(3, dtype=torch.int32, device=page_table.device)
    _need(counts, "counts", torch.int32)
    if counts.numel() < 3:
        raise MinisglError("counts needs 3 elements")
    _check(lib.minisgl_check_indices(_ptr(page_table), page_table.shape[0], page_table.stride(0),
                                     page_table.shape[1], _ptr(lens), _ptr(out_loc), n_out,
                                     num_rows, _ptr(counts), _stream(stream)), "check_indices")
    return counts


def minisgl_debug_timeout_count() -> int:
    c = ctypes.c_uint32(0)
    _check(load_library().minisgl_debug_timeout_count(ctypes.byref(c)), "debug_timeout_count")
    return int(c.value)


def minisgl_debug_set_pdl(enabled: bool) -> bool:
    """Turn programmatic dependent launch on or off for the library's later
    launches (a measurement aid); returns the previous setting."""
    return bool(load_library().minisgl_debug_set_pdl(1 if enabled else 0))


def minisgl_rope_store_kv(pool: KVPool, layer: int, q: torch.Tensor, k: torch.Tensor,
                          v: torch.Tensor, positions: torch.Tensor, cos_sin_cache: torch.Tensor,
                          out_loc: torch.Tensor, stream=None) -> torch.Tensor:
    """Rotate q [N, H_q, d] in place and k [N, H_kv, d] into the pool by each
    token's position, and store v; returns q.  k is left unrotated."""
    lib = load_library()
    _need(q, "q", torch.bfloat16)
    _need(k, "k", torch.bfloat16)
    _need(v, "v", torch.bfloat16)
    _need(positions, "positions", torch.int32)
    _need(out_loc, "out_loc", torch.int32)
    _need(cos_sin_cache, "cos_sin_cache", torch.float32)
    n = out_loc.numel()
    d = pool.head_dim
    if q.dim() != 3 or q.shape[0] != n or q.shape[2] != d or q.stride(2) != 1 or q.stride(1) != d:
        raise MinisglError("q must be [n_tokens, H_q, head_dim] with contiguous rows")
    for t, nm in ((k, "k"), (v, "v")):
        if (t.dim() != 3 or t.shape[0] != n or t.shape[1] != pool.num_kv_heads or t.shape[2] != d
                or t.stride(2) != 1 or t.stride(1) != d):
            raise MinisglError(f"{nm} must be [n_tokens, H_kv, d] with contiguous rows")
    if positions.numel() != n or not positions.is_contiguous() or not out_loc.is_contiguous():
        raise MinisglError("positions and out_loc must be contiguous [n_tokens]")
    if cos_sin_cache.dim() != 2 or cos_sin_cache.shape[1] != d or not cos_sin_cache.is_contiguous():
        raise MinisglError("cos_sin_cache must be contiguous [max_positions, head_dim] float32")
    _check(lib.minisgl_rope_store_kv(ctypes.byref(pool.desc), layer, _ptr(q), q.shape[1], q.stride(0),
                                     _ptr(k), _ptr(v), k.stride(0), v.stride(0), _ptr(positions),
                                     _ptr(cos_sin_cache), cos_sin_cache.shape[0], _ptr(out_loc), n,
                                     _stream(stream)), "rope_store_kv")
    return q


def minisgl_cascade_workspace_bytes(batch: int, num_q_heads: int, num_kv_heads: int,
                                    head_dim: int) -> int:
    return int(load_library().minisgl_cascade_workspace_bytes(batch, num_q_heads, num_kv_heads,
                                                              head_dim))


def minisgl_cascade_decode_attn(pool: KVPool, layer: int, q: torch.Tensor, page_table: torch.Tensor,
                                seq_lens: torch.Tensor, shared_len: int, sm_scale: float,
                                out: Optional[torch.Tensor] = None,
                                workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode attention of q [B, H_q, d] for requests whose first shared_len
    page-table entries are the same rows; the shared rows are read once."""
    lib = load_library()
    _need(q, "q", torch.bfloat16)
    _need(page_table, "page_table", torch.int32)
    _need(seq_lens, "seq_lens", torch.int32)
    B, Hq, d = q.shape
    if not q.is_contiguous() or d != pool.head_dim:
        raise MinisglError("q must be contiguous [B, H_q, head_dim]")
    if page_table.dim() != 2 or page_table.shape[0] != B or page_table.stride(1) != 1:
        raise MinisglError("page_table must be [B, W] with unit column stride")
    if seq_lens.numel() != B or not seq_lens.is_contiguous():
        raise MinisglError("seq_lens must be contiguous [B]")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16)
    if workspace is None:
        nbytes = minisgl_cascade_workspace_bytes(B, Hq, pool.num_kv_heads, d)
        key = ("cascade", q.device, nbytes)
        workspace = _ws_cache.get(key)
        if workspace is None:
            # the first 256 bytes (a work counter) must start at zero
            workspace = torch.zeros(nbytes, dtype=torch.uint8, device=q.device)
            _ws_cache[key] = workspace
    _check(lib.minisgl_cascade_decode_attn(ctypes.byref(pool.desc), layer, _ptr(q), Hq, _ptr(page_table),
                                           B, page_table.stride(0), page_table.shape[1], _ptr(seq_lens),
                                           int(shared_len), float(sm_scale), _ptr(out), _ptr(workspace),
                                           workspace.numel(), _stream(stream)), "cascade_decode_attn")
    return out


def minisgl_store_decode_attn(pool: KVPool, layer: int, k: torch.Tensor, v: torch.Tensor,
                              out_loc: torch.Tensor, q: torch.Tensor, page_table: torch.Tensor,
                              seq_lens: torch.Tensor, sm_scale: float,
                              out: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None, split_tokens: int = 0,
                              max_splits: int = 16, stream=None) -> torch.Tensor:
    """minisgl_store_kv(k, v, out_loc) and minisgl_decode_attn in one pass
    (k, v: [B, H_kv, d], one new row per request)."""
    lib = load_library()
    for t, nm in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, nm, torch.bfloat16)
    for t, nm in ((page_table, "page_table"), (seq_lens, "seq_lens"), (out_loc, "out_loc")):
        _need(t, nm, torch.int32)
    B, Hq, d = q.shape
    if not q.is_contiguous() or d != pool.head_dim:
        raise MinisglError("q must be contiguous [B, H_q, head_dim]")
    row = pool.num_kv_heads * d
    for t, nm in ((k, "k"), (v, "v")):
        if not _rows_ok(t, B, row):
            raise MinisglError(f"{nm} must be [B, H_kv, d] with contiguous rows")
    if page_table.dim() != 2 or page_table.shape[0] != B or page_table.stride(1) != 1:
        raise MinisglError("page_table must be [B, W] with unit column stride")
    if seq_lens.numel() != B or not seq_lens.is_contiguous() or out_loc.numel() != B \
            or not out_loc.is_contiguous():
        raise MinisglError("seq_lens and out_loc must be contiguous [B]")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16)
    if workspace is None:
        workspace = decode_workspace(B, Hq, pool, max_splits)
    _check(lib.minisgl_store_decode_attn(ctypes.byref(pool.desc), layer, _ptr(k), _ptr(v), k.stride(0),
                                         v.stride(0), _ptr(out_loc), _ptr(q), Hq, _ptr(page_table), B,
                                         page_table.stride(0), page_table.shape[1], _ptr(seq_lens),
                                         float(sm_scale), _ptr(out), _ptr(workspace), workspace.numel(),
                                         split_tokens, _stream(stream)), "store_decode_attn")
    return out


def minisgl_cascade_extend_workspace_bytes(total_q_tokens: int, num_q_heads: int, head_dim: int) -> int:
    return int(load_library().minisgl_cascade_extend_workspace_bytes(total_q_tokens, num_q_heads,
                                                                     head_dim))


def minisgl_cascade_extend_attn(pool: KVPool, layer: int, q: torch.Tensor, page_table: torch.Tensor,
                                cached_lens: torch.Tensor, extend_lens: torch.Tensor,
                                q_offsets: torch.Tensor, shared_len: int, sm_scale: float,
                                out: Optional[torch.Tensor] = None,
                                workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal extend attention of q [T, H_q, d] for requests whose first
    shared_len page-table entries are the same rows: a pass of all new tokens
    against the shared rows, then each request's own rows with that pass's
    partial folded in."""
    lib = load_library()
    _need(q, "q", torch.bfloat16)
    for t, nm in ((page_table, "page_table"), (cached_lens, "cached_lens"),
                  (extend_lens, "extend_lens"), (q_offsets, "q_offsets")):
        _need(t, nm, torch.int32)
    T, Hq, d = q.shape
    B = cached_lens.numel()
    if not q.is_contiguous() or d != pool.head_dim:
        raise MinisglError("q must be contiguous [T, H_q, head_dim]")
    if page_table.dim() != 2 or page_table.shape[0] != B or page_table.stride(1) != 1:
        raise MinisglError("page_table must be [B, W] with unit column stride")
    if extend_lens.numel() != B or q_offsets.numel() != B + 1:
        raise MinisglError("extend_lens must be [B] and q_offsets [B+1]")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16)
    if workspace is None:
        nbytes = minisgl_cascade_extend_workspace_bytes(T, Hq, d)
        key = ("cascade_extend", q.device, nbytes)
        workspace = _ws_cache.get(key)
        if workspace is None:
            # the first 256 bytes (a work counter) must start at zero
            workspace = torch.zeros(nbytes, dtype=torch.uint8, device=q.device)
            _ws_cache[key] = workspace
    _check(lib.minisgl_cascade_extend_attn(ctypes.byref(pool.desc), layer, _ptr(q), Hq, _ptr(page_table), B,
                                           page_table.stride(0), page_table.shape[1], _ptr(cached_lens),
                                           _ptr(extend_lens), _ptr(q_offsets), T, int(shared_len),
                                           float(sm_scale), _ptr(out), _ptr(workspace), workspace.numel(),
                                           _stream(stream)), "cascade_extend_attn")
    return out


def minisgl_check_shared_prefix(page_table: torch.Tensor, lens: torch.Tensor, shared_len: int,
                                counts: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Count, on the device, the shared-prefix page-table entries that differ
    from the first request's and the requests shorter than shared_len:
    returns an int32 CUDA tensor [differing entries, short requests] (read it
    after the stream).  lens: seq_lens for decode, cached_lens for extend."""
    lib = load_library()
    _need(page_table, "page_table", torch.int32)
    _need(lens, "lens", torch.int32)
    if page_table.dim() != 2 or page_table.stride(1) != 1:
        raise MinisglError("page_table must be [B, W] with unit column stride")
    if lens.numel() != page_table.shape[0] or not lens.is_contiguous():
        raise MinisglError("lens must be a contiguous [B] tensor")
    if counts is None:
        counts = torch.empty(2, dtype=torch.int32, device=page_table.device)
    _need(counts, "counts", torch.int32)
    if counts.numel() < 2:
        raise MinisglError("counts needs 2 elements")
    _check(lib.minisgl_check_shared_prefix(_ptr(page_table), page_table.shape[0], page_table.stride(0),
                                           page_table.shape[1], int(shared_len), _ptr(lens), _ptr(counts),
                                           _stream(stream)), "check_shared_prefix")
    return counts


# --------------------------------------------------------------------------- #
# the 4-bit pool
# --------------------------------------------------------------------------- #
FP4_BLOCK = 16  # channels that share a scale


# The quick forms of torch.cuda.current_stream(i).cuda_stream (which builds a
# Stream object first and takes longer than a kernel launch), current_device()
# and empty_strided(device="cuda"), where torch has them: a call that allocates
# 5 outputs takes 15 us instead of 22.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_quick_new = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)


def _new(shape, strides, dtype):
    """A new tensor on the current device.  The quick form goes past torch's
    own function, which fills new memory where deterministic algorithms are
    asked for."""
    if _quick_new is None or torch.are_deterministic_algorithms_enabled():
        return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")
    return _quick_new(shape, strides, dtype)


def _on(stream, index: int):
    """The context in which tensors on cuda:index are current: their device,
    and the stream if the caller named one."""
    if stream is None:
        return torch.cuda.device(index)
    if stream.device.index != index:
        raise MinisglError(f"stream on {stream.device}, tensors on cuda:{index}")
    return torch.cuda.stream(stream)


_I32, _BF16 = torch.int32, torch.bfloat16


def _at(t: torch.Tensor, name: str, dtype: torch.dtype, index: Optional[int] = None) -> int:
    """The CUDA device index of t, a tensor of this type (on device `index` if given)."""
    i = t.get_device()
    if i < 0 or t.dtype is not dtype:
        _need(t, name, dtype)
    if index is not None and i != index:
        raise MinisglError(f"tensors on different devices: {name} on cuda:{i}, others on cuda:{index}")
    return i


# The checks below look at a tensor themselves and leave it to _at to say what
# is wrong: a call less for each argument.
def _vec(t: torch.Tensor, name: str, n: Optional[int], index: int) -> None:
    if t.get_device() != index or t.dtype is not _I32:
        _at(t, name, _I32, index)
    if (n is not None and t.numel() != n) or not t.is_contiguous():
        raise MinisglError(f"{name} must be a contiguous int32 tensor" + (f" of {n} elements" if n is not None else ""))


def _table(t: torch.Tensor, n: int, index: int) -> Tuple[int, int]:
    """Row stride and width of a page table of n rows."""
    if t.get_device() != index or t.dtype is not _I32:
        _at(t, "page_table", _I32, index)
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or shape[0] != n or (shape[1] > 1 and strides[1] != 1):
        raise MinisglError("page_table must be [B, W] with unit column stride")
    # the stride of a table of one row means nothing and can be anything
    return (strides[0] if n > 1 else max(strides[0], shape[1])), shape[1]


def _kv_rows(t: torch.Tensor, name: str, n: int, row: int, index: int, what: str = "n_tokens") -> int:
    """Token stride of n contiguous rows of `row` bf16 elements."""
    if t.get_device() != index or t.dtype is not _BF16:
        _at(t, name, _BF16, index)
    shape, strides = t.shape, t.stride()
    usual = (len(shape) == 3 and shape[0] == n and shape[1] * shape[2] == row and strides[2] == 1
             and strides[1] == shape[2])
    if not usual and not _rows_ok(t, n, row):
        raise MinisglError(f"{name} must be [{what}, H_kv, d] with contiguous rows")
    return strides[0] if n > 1 else row


def _exponents(e, layers: int, name: str) -> List[int]:
    """One exponent per layer from one integer (of any kind) or one per layer."""
    try:
        try:
            e = [operator.index(e)] * layers
        except TypeError:
            e = list(e)
        out = [int(x) for x in e]
        if len(out) == layers and all(o == x and -64 <= o <= 64 for o, x in zip(out, e)):
            return out
    except (TypeError, ValueError, OverflowError):
        pass
    raise MinisglError(f"{name} must be one int or one per layer, in [-64, 64]")


class KVPoolFP4:
    """A paged KV pool in 4 bits (the format is in include/minisgl.h): `data`
    uint8 (2, L, R, H_kv, d/2), two e2m1 elements to a byte, and `scales`
    (2, L, R, H_kv, d/16), e4m3 scales as float8_e4m3fn or their uint8 bytes.
    The rows of a layer are contiguous (H_kv, ..); the axes before them may have
    any strides.  k_exp, v_exp: the power of two that K and V values are
    multiplied with, one int or one per layer.  Caller-owned device memory; a
    new pool's bytes should be zero (KVPoolFP4.zeros makes one).  With one KV
    head use pages of 16 rows or more: a row's 64 and 8 bytes from anywhere take
    longer to read than when their neighbours are used too (200 requests of 1k
    to 8k tokens, 8 query heads: 50 us instead of 36)."""

    def __init__(self, data: torch.Tensor, scales: torch.Tensor, page_size: int = 1,
                 k_exp: Union[int, Sequence[int]] = 0, v_exp: Union[int, Sequence[int]] = 0):
        if data.dim() != 5 or data.shape[0] != 2:
            raise MinisglError("pool data must have shape (2, L, R, H_kv, d/2)")
        _need(data, "pool data", torch.uint8)
        if scales.dtype == torch.float8_e4m3fn:
            scales = scales.view(torch.uint8)
        _need(scales, "pool scales", torch.uint8)
        _, L, R, H, half = data.shape
        d = 2 * half
        if tuple(scales.shape) != (2, L, R, H, d // FP4_BLOCK):
            raise MinisglError("pool scales must have shape (2, L, R, H_kv, d/16)")
        if scales.device != data.device:
            raise MinisglError("pool data and scales on different devices")
        for t in (data, scales):
            if t.stride(4) != 1 or (H > 1 and t.stride(3) != t.shape[4]):
                raise MinisglError("pool rows must be (H_kv, ..) contiguous")
        self.data, self.scales, self.page_size = data, scales, page_size
        self.num_layers, self.num_rows, self.num_kv_heads, self.head_dim = L, R, H, d
        exps = _exponents(k_exp, L, "k_exp"), _exponents(v_exp, L, "v_exp")
        self.k_exp, self.v_exp = exps
        at = {p: _PoolFP4Desc(
            k_data=data.data_ptr(), v_data=data.data_ptr() + data.stride(0),
            k_scale=scales.data_ptr(), v_scale=scales.data_ptr() + scales.stride(0),
            data_layer_stride=data.stride(1), data_row_stride=data.stride(2),
            scale_layer_stride=scales.stride(1), scale_row_stride=scales.stride(2),
            num_layers=L, num_rows=R, num_kv_heads=H, head_dim=d, page_size=page_size,
            dtype=MINISGL_FP4, k_exp=p[0], v_exp=p[1]) for p in set(zip(*exps))}
        self._by_layer = [ctypes.byref(at[p]) for p in zip(*exps)]
        self._index = data.get_device()

    @classmethod
    def zeros(cls, num_layers: int, num_rows: int, num_kv_heads: int, head_dim: int, page_size: int = 1,
              k_exp: Union[int, Sequence[int]] = 0, v_exp: Union[int, Sequence[int]] = 0,
              device=None) -> "KVPoolFP4":
        shape = (2, num_layers, num_rows, num_kv_heads)
        device = device or "cuda"
        return cls(torch.zeros(shape + (head_dim // 2,), dtype=torch.uint8, device=device),
                   torch.zeros(shape + (head_dim // FP4_BLOCK,), dtype=torch.uint8, device=device),
                   page_size, k_exp, v_exp)

    def _desc(self, layer: int):
        if not 0 <= layer < self.num_layers:
            raise MinisglError(f"layer {layer} outside [0, {self.num_layers})")
        return self._by_layer[layer]


def kv_pool_fp4_bytes(num_layers: int, num_kv_heads: int, head_dim: int, num_tokens: int) -> int:
    """Bytes a 4-bit pool needs to hold num_tokens token rows in every layer, K and V."""
    return 2 * num_layers * num_kv_heads * (head_dim // 2 + head_dim // FP4_BLOCK) * num_tokens


class Slots(NamedTuple):
    """What minisgl_build_slots writes besides the page table (int32 CUDA tensors)."""
    out_loc: torch.Tensor     # [total_tokens] row of each new token
    positions: torch.Tensor   # [total_tokens] position of each new token
    q_offsets: torch.Tensor   # [B + 1] exclusive prefix sum of extend_lens
    seq_lens: torch.Tensor    # [B] cached_lens + extend_lens
    pages_used: torch.Tensor  # [1] new pages the batch needs

    @staticmethod
    def empty(batch: int, total_tokens: int, device=None) -> "Slots":
        return Slots(*(torch.empty(n, dtype=torch.int32, device=device or "cuda")
                       for n in (total_tokens, total_tokens, batch + 1, batch, 1)))


def minisgl_build_slots(cached_lens: torch.Tensor, extend_lens: torch.Tensor, page_table: torch.Tensor,
                        free_pages: torch.Tensor, page_size: int, dummy_row: int, total_tokens: int,
                        out: Optional[Slots] = None, stream=None) -> Slots:
    """Give every new token of the batch a row: requests with cached_lens[r]
    tokens in the pool get extend_lens[r] more, in pages taken from free_pages
    in order.  Writes page_table [B, W] in place and returns the step's Slots
    (into `out` if given).  cached_lens[r] < 0 marks a padding request, whose
    rows are dummy_row, a row that no request holds.  pages_used >
    len(free_pages) says that pages ran out (the tokens without one are on
    dummy_row, and so are the later ones of the same page)."""
    B, total = cached_lens.numel(), int(total_tokens)
    if total < 0:
        raise MinisglError("total_tokens must not be negative")
    dev = _at(cached_lens, "cached_lens", _I32)
    if stream is not None or _device() != dev:
        with _on(stream, dev):
            return minisgl_build_slots(cached_lens, extend_lens, page_table, free_pages, page_size, dummy_row,
                                       total, out)
    _vec(cached_lens, "cached_lens", None, dev)
    _vec(extend_lens, "extend_lens", B, dev)
    _vec(free_pages, "free_pages", None, dev)
    stride, width = _table(page_table, B, dev)
    if out is not None:
        for t, nm, n in zip(out, Slots._fields, (total, total, B + 1, B, 1)):
            _vec(t, nm, n, dev)
    else:
        one = (1,)
        out = Slots(_new((total,), one, _I32), _new((total,), one, _I32), _new((B + 1,), one, _I32),
                    _new((B,), one, _I32), _new(one, one, _I32))
    loc, pos, off, lens, used = out
    _check(load_library().minisgl_build_slots(
        cached_lens.data_ptr(), extend_lens.data_ptr(), B, page_table.data_ptr(), stride, width,
        free_pages.data_ptr(), free_pages.numel(), page_size, dummy_row, loc.data_ptr(), pos.data_ptr(),
        off.data_ptr(), lens.data_ptr(), used.data_ptr(), total, _raw_stream(dev)), "build_slots")
    return out


def minisgl_store_kv_fp4(pool: KVPoolFP4, layer: int, k: torch.Tensor, v: torch.Tensor,
                         out_loc: torch.Tensor, stream=None) -> None:
    """Quantise k[i], v[i] ([n_tokens, H_kv, d] bf16) into row out_loc[i] of the 4-bit pool."""
    dev, row = pool._index, pool.num_kv_heads * pool.head_dim
    if stream is not None or _device() != dev:
        with _on(stream, dev):
            return minisgl_store_kv_fp4(pool, layer, k, v, out_loc)
    n = out_loc.numel()
    _vec(out_loc, "out_loc", None, dev)
    ks, vs = _kv_rows(k, "k", n, row, dev), _kv_rows(v, "v", n, row, dev)
    _check(load_library().minisgl_store_kv_fp4(pool._desc(layer), layer, k.data_ptr(), v.data_ptr(), ks, vs,
                                               out_loc.data_ptr(), n, _raw_stream(dev)), "store_kv_fp4")


def minisgl_load_kv_fp4(pool: KVPoolFP4, layer: int, page_table: torch.Tensor, lens: torch.Tensor,
                        offsets: torch.Tensor, total_tokens: int, k_out: Optional[torch.Tensor] = None,
                        v_out: Optional[torch.Tensor] = None,
                        stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Rows page_table[r, :lens[r]] of the 4-bit pool as bf16, request r's from
    row offsets[r] of k_out and v_out ([total_tokens, H_kv, d], made here if
    not given; rows that no request fills are not written)."""
    dev, H, d = pool._index, pool.num_kv_heads, pool.head_dim
    if stream is not None or _device() != dev:
        with _on(stream, dev):
            return minisgl_load_kv_fp4(pool, layer, page_table, lens, offsets, total_tokens, k_out, v_out)
    B, total = lens.numel(), int(total_tokens)
    if total < 0:
        raise MinisglError("total_tokens must not be negative")
    stride, width = _table(page_table, B, dev)
    _vec(lens, "lens", None, dev)
    _vec(offsets, "offsets", B + 1, dev)
    row = H * d
    ks = row if k_out is None else _kv_rows(k_out, "k_out", total, row, dev, "total_tokens")
    vs = row if v_out is None else _kv_rows(v_out, "v_out", total, row, dev, "total_tokens")
    if k_out is None:
        k_out = _new((total, H, d), (row, d, 1), _BF16)
    if v_out is None:
        v_out = _new((total, H, d), (row, d, 1), _BF16)
    _check(load_library().minisgl_load_kv_fp4(pool._desc(layer), layer, page_table.data_ptr(), B, stride, width,
                                              lens.data_ptr(), offsets.data_ptr(), total, k_out.data_ptr(),
                                              v_out.data_ptr(), ks, vs, _raw_stream(dev)), "load_kv_fp4")
    return k_out, v_out


def decode_workspace_fp4(batch: int, num_q_heads: int, pool: KVPoolFP4, max_splits: int = 32) -> torch.Tensor:
    """A new workspace for minisgl_decode_attn_fp4 on the pool's device.  Calls
    that may run at the same time need different ones.  For one or two requests
    of many tokens more splits let more of the GPU work (256 at most)."""
    return torch.empty(minisgl_decode_workspace_bytes(batch, num_q_heads, pool.num_kv_heads, pool.head_dim,
                                                      max_splits), dtype=torch.uint8, device=pool.data.device)


def minisgl_decode_attn_fp4(pool: KVPoolFP4, layer: int, q: torch.Tensor, page_table: torch.Tensor,
                            seq_lens: torch.Tensor, sm_scale: float, out: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, split_tokens: int = 0,
                            max_splits: int = 32, stream=None) -> torch.Tensor:
    """Decode attention of q [B, H_q, d] over each request's page_table row of
    the 4-bit pool.  Without a workspace the call allocates its own."""
    dev = _at(q, "q", _BF16, pool._index)
    if stream is not None or _device() != dev:
        with _on(stream, dev):
            return minisgl_decode_attn_fp4(pool, layer, q, page_table, seq_lens, sm_scale, out, workspace,
                                           split_tokens, max_splits)
    shape = q.shape
    if len(shape) != 3 or shape[2] != pool.head_dim or not q.is_contiguous():
        raise MinisglError("q must be contiguous [B, H_q, head_dim]")
    B, Hq, d = shape
    stride, width = _table(page_table, B, dev)
    _vec(seq_lens, "seq_lens", B, dev)
    if out is None:
        out = _new((B, Hq, d), (Hq * d, d, 1), _BF16)
    else:
        _at(out, "out", _BF16, dev)
        if out.shape != shape or not out.is_contiguous():
            raise MinisglError("out must be contiguous with the shape of q")
    if workspace is None:
        workspace = decode_workspace_fp4(B, Hq, pool, max_splits)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise MinisglError("workspace must be a contiguous CUDA tensor on the pool's device")
    _check(load_library().minisgl_decode_attn_fp4(
        pool._desc(layer), layer, q.data_ptr(), Hq, page_table.data_ptr(), B, stride, width, seq_lens.data_ptr(),
        float(sm_scale), out.data_ptr(), workspace.data_ptr(), workspace.nbytes, split_tokens,
        _raw_stream(dev)), "decode_attn_fp4")
    return out
