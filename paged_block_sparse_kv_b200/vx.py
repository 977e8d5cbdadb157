"""Python binding of libvx (include/vx.h): argument marshalling only.

Every function has the name of the C entry point it calls and does nothing but turn
torch tensors into pointers and sizes, call the library on the current CUDA stream and
raise VxError on a non-zero status.  All computation runs in libvx's CUDA kernels; there
is no fallback: if libvx.so is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvx.so")

VX_OK, VX_ERR_INVALID_ARG, VX_ERR_UNSUPPORTED, VX_ERR_WORKSPACE, VX_ERR_CUDA = range(5)
VX_DATA_BAD_PAGE_ID, VX_DATA_BAD_SEQ_LEN, VX_DATA_BAD_SELECTION, VX_DATA_TIMEOUT = 1, 2, 4, 8
VX_DATA_BAD_VALUE, VX_DATA_BAD_ROW, VX_DATA_NO_PAGES, VX_DATA_BAD_COPY = 16, 32, 64, 128
VX_QUANT_INT8, VX_QUANT_E4M3 = 1, 2  # code types of an 8-bit cache
NOALLOC_SCRATCH_BYTES = 16 << 20  # VX_NOALLOC_SCRATCH_BYTES of include/vx.h
VX_TABLE_READY = 0x100  # mode flag of the chained steps: the table and lengths are not the previous kernel's output

# every symbol include/vx.h declares
EXPORTS = ["vx_centroid_update", "vx_score_pages", "vx_topk_pages", "vx_sparse_decode",
           "vx_sparse_decode_noalloc", "vx_block_topk_decode", "vx_block_topk_decode_append",
           "vx_block_topk_decode_persistent", "vx_quant_update", "vx_sparse_decode_quant",
           "vx_block_topk_decode_quant", "vx_block_topk_decode_append_quant", "vx_copy_pages", "vx_update_table",
           "vx_compact_pages", "vx_page_workspace_size", "vx_workspace_size", "vx_planned_splits", "vx_status_string",
           "vx_last_error", "vx_version"]


class VxError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


class vx_geometry(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim_qk", ctypes.c_int32), ("head_dim_v", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("mla_shared_kv", ctypes.c_int32), ("num_pool_pages", ctypes.c_int64)]


class vx_page_table(ctypes.Structure):
    _fields_ = [("page_ptr", ctypes.c_void_p), ("page_indices", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("max_pages", ctypes.c_int32)]


class vx_quant_cache(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class vx_page_pool(ctypes.Structure):
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("centroids", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("elem_bytes", ctypes.c_int32),
                ("num_pages", ctypes.c_int64)]


_lib = None


def lib():
    """The loaded libvx.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libvx.so is not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        p, i32, i64, u64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64,
                                     ctypes.c_float, ctypes.c_size_t)
        G, T = ctypes.POINTER(vx_geometry), ctypes.POINTER(vx_page_table)
        L.vx_centroid_update.argtypes = [G, T, p, p, p, p, p, p, p, p]
        L.vx_score_pages.argtypes = [G, T, p, p, i32, p, p, p]
        L.vx_topk_pages.argtypes = [G, T, p, i32, i32, u64, p, p, p]
        L.vx_sparse_decode.argtypes = [G, T, p, p, p, p, i32, f32, i32, p, p, p, sz, p, p]
        L.vx_sparse_decode_noalloc.argtypes = [G, T, p, p, p, p, i32, f32, i32, p, p, p, p]
        L.vx_block_topk_decode_persistent.argtypes = [G, T, p, p, p, p, i32, f32, p, p, p, p, p, sz, p, p]
        L.vx_block_topk_decode.argtypes = [G, T, p, p, p, p, i32, i32, u64, f32, i32, i32, p, p, p, p, p, sz,
                                           p, p]
        L.vx_block_topk_decode_append.argtypes = [G, T, p, p, p, p, p, p, i32, i32, u64, f32, i32, i32, p, p, p, p,
                                                  p, sz, p, p]
        Q, O = ctypes.POINTER(vx_quant_cache), ctypes.POINTER(vx_page_pool)
        L.vx_quant_update.argtypes = [G, T, Q, p, p, p, p, p, p]
        L.vx_sparse_decode_quant.argtypes = [G, T, p, Q, p, i32, f32, i32, p, p, p, sz, p, p]
        L.vx_block_topk_decode_quant.argtypes = [G, T, p, Q, p, i32, i32, u64, f32, i32, i32, p, p, p, p, p, sz, p, p]
        L.vx_block_topk_decode_append_quant.argtypes = [G, T, p, Q, p, p, p, i32, i32, u64, f32, i32, i32, p, p, p, p,
                                                        p, sz, p, p]
        L.vx_copy_pages.argtypes = [G, O, O, p, p, i32, p, sz, p, p]
        L.vx_update_table.argtypes = [G, O, T, p, p, p, i32, p, p, i64, p, i32, p, p, sz, p, p]
        L.vx_compact_pages.argtypes = [G, O, T, p, p, p, p, p, p, sz, p, p]
        L.vx_page_workspace_size.argtypes = [G, i32]
        L.vx_page_workspace_size.restype = sz
        L.vx_workspace_size.argtypes = [G, i32, i32, i32]
        L.vx_workspace_size.restype = sz
        L.vx_planned_splits.argtypes = [G, i32, i32]
        L.vx_planned_splits.restype = i32
        L.vx_status_string.argtypes = [i32]
        L.vx_status_string.restype = ctypes.c_char_p
        L.vx_last_error.restype = ctypes.c_char_p
        L.vx_version.restype = ctypes.c_char_p
        for name in ("vx_centroid_update", "vx_score_pages", "vx_topk_pages", "vx_sparse_decode",
                     "vx_sparse_decode_noalloc", "vx_block_topk_decode", "vx_block_topk_decode_append",
                     "vx_block_topk_decode_persistent", "vx_quant_update", "vx_sparse_decode_quant",
                     "vx_block_topk_decode_quant", "vx_block_topk_decode_append_quant", "vx_copy_pages",
                     "vx_update_table", "vx_compact_pages"):
            getattr(L, name).restype = i32
        _lib = L
    return _lib


@dataclass
class Geometry:
    batch: int
    num_q_heads: int
    num_kv_heads: int
    head_dim_qk: int
    head_dim_v: int
    page_size: int
    mla_shared_kv: bool
    num_pool_pages: int

    def c(self) -> vx_geometry:
        return vx_geometry(self.batch, self.num_q_heads, self.num_kv_heads, self.head_dim_qk, self.head_dim_v,
                           self.page_size, int(self.mla_shared_kv), self.num_pool_pages)

    @staticmethod
    def of(k_cache: torch.Tensor, num_q_heads: int, batch: int, mla_shared_kv: bool = False,
           head_dim_v: Optional[int] = None) -> "Geometry":
        """Geometry of a cache [Npool][Hkv][P][Dqk]."""
        npool, hkv, P, dqk = k_cache.shape
        dv = head_dim_v if head_dim_v is not None else (512 if mla_shared_kv else dqk)
        return Geometry(batch, num_q_heads, hkv, dqk, dv, P, mla_shared_kv, npool)


@dataclass
class PageTable:
    page_ptr: torch.Tensor      # int32 [B] (device)
    page_indices: torch.Tensor  # int32 (device)
    seq_lens: torch.Tensor      # int32 [B] (device)
    max_pages: int

    def c(self) -> vx_page_table:
        for t in (self.page_ptr, self.page_indices, self.seq_lens):
            _check(t, torch.int32)
        return vx_page_table(self.page_ptr.data_ptr(), self.page_indices.data_ptr(), self.seq_lens.data_ptr(),
                             self.max_pages)


def _check(t: Optional[torch.Tensor], dtype=None):
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError("tensors passed to libvx must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"expected {dtype}, got {t.dtype}")


def _ptr(t: Optional[torch.Tensor], dtype=None):
    if t is None:
        return None
    _check(t, dtype)
    return t.data_ptr()


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _ok(status: int):
    if status != VX_OK:
        L = lib()
        raise VxError(status, f"{L.vx_status_string(status).decode()}: {L.vx_last_error().decode()}")


def vx_workspace_size(geo: Geometry, max_pages: int, k: int, num_splits: int = 0) -> int:
    n = lib().vx_workspace_size(ctypes.byref(geo.c()), max_pages, k, num_splits)
    if n == 0:
        raise VxError(VX_ERR_INVALID_ARG, lib().vx_last_error().decode())
    return n


def vx_planned_splits(geo: Geometry, max_pages: int, k: int) -> int:
    return int(lib().vx_planned_splits(ctypes.byref(geo.c()), max_pages, k))


def vx_centroid_update(geo: Geometry, table: PageTable, k_cache, centroids, v_cache=None, k_new=None, v_new=None,
                       first_pos=None, err=None, stream=None):
    """Rebuild (k_new None), append one token per request (k_new [B][Hkv][Dqk]) or write a
    prefill chunk (k_new [N][Hkv][Dqk] packed in request order, with first_pos)."""
    _ok(lib().vx_centroid_update(ctypes.byref(geo.c()), ctypes.byref(table.c()), _ptr(k_cache, torch.bfloat16),
                                 _ptr(v_cache, torch.bfloat16), _ptr(centroids, torch.bfloat16),
                                 _ptr(k_new, torch.bfloat16), _ptr(v_new, torch.bfloat16),
                                 _ptr(first_pos, torch.int32), _ptr(err, torch.int32), _stream(stream)))


def vx_score_pages(geo: Geometry, table: PageTable, q, centroids, scores, score_dims=0, err=None, stream=None):
    _ok(lib().vx_score_pages(ctypes.byref(geo.c()), ctypes.byref(table.c()), _ptr(q, torch.bfloat16),
                             _ptr(centroids, torch.bfloat16), score_dims, _ptr(scores, torch.float32),
                             _ptr(err, torch.int32), _stream(stream)))


def vx_topk_pages(geo: Geometry, table: PageTable, scores, k: int, sel, mode=0, seed=0, err=None, stream=None):
    _ok(lib().vx_topk_pages(ctypes.byref(geo.c()), ctypes.byref(table.c()), _ptr(scores, torch.float32), k, mode,
                            seed & (2 ** 64 - 1), _ptr(sel, torch.int32), _ptr(err, torch.int32), _stream(stream)))


def vx_sparse_decode(geo: Geometry, table: PageTable, q, k_cache, v_cache, sel, k: int, out, ws, lse=None,
                     sm_scale=0.0, num_splits=0, err=None, stream=None):
    _ok(lib().vx_sparse_decode(ctypes.byref(geo.c()), ctypes.byref(table.c()), _ptr(q, torch.bfloat16),
                               _ptr(k_cache, torch.bfloat16), _ptr(v_cache, torch.bfloat16), _ptr(sel, torch.int32),
                               k, float(sm_scale), num_splits, _ptr(out, torch.bfloat16), _ptr(lse, torch.float32),
                               _ptr(ws), ws.numel() * ws.element_size(), _ptr(err, torch.int32), _stream(stream)))


def vx_sparse_decode_noalloc(geo: Geometry, table: PageTable, q, k_cache, v_cache, sel, k: int, out, lse=None,
                             sm_scale=0.0, num_splits=0, err=None, stream=None):
    """vx_sparse_decode for callers that cannot allocate device memory: the split partials
    live in a fixed scratch array inside the library (see include/vx.h)."""
    _ok(lib().vx_sparse_decode_noalloc(ctypes.byref(geo.c()), ctypes.byref(table.c()), _ptr(q, torch.bfloat16),
                                       _ptr(k_cache, torch.bfloat16), _ptr(v_cache, torch.bfloat16),
                                       _ptr(sel, torch.int32), k, float(sm_scale), num_splits,
                                       _ptr(out, torch.bfloat16), _ptr(lse, torch.float32), _ptr(err, torch.int32),
                                       _stream(stream)))


def vx_block_topk_decode(geo: Geometry, table: PageTable, q, k_cache, v_cache, centroids, k: int, out, ws,
                         lse=None, mode=0, seed=0, sm_scale=0.0, score_dims=0, num_splits=0, scores_out=None,
                         sel_out=None, err=None, stream=None):
    _ok(lib().vx_block_topk_decode(ctypes.byref(geo.c()), ctypes.byref(table.c()), _ptr(q, torch.bfloat16),
                                   _ptr(k_cache, torch.bfloat16), _ptr(v_cache, torch.bfloat16),
                                   _ptr(centroids, torch.bfloat16), k, mode, seed & (2 ** 64 - 1), float(sm_scale),
                                   score_dims, num_splits, _ptr(out, torch.bfloat16), _ptr(lse, torch.float32),
                                   _ptr(scores_out, torch.float32), _ptr(sel_out, torch.int32), _ptr(ws),
                                   ws.numel() * ws.element_size(), _ptr(err, torch.int32), _stream(stream)))


def vx_block_topk_decode_append(geo: Geometry, table: PageTable, q, k_cache, v_cache, centroids, k_new, v_new,
                                k: int, out, ws, lse=None, mode=0, seed=0, sm_scale=0.0, score_dims=0, num_splits=0,
                                scores_out=None, sel_out=None, err=None, stream=None):
    """One appending decode step: write each request's new token (k_new [B][Hkv][Dqk], v_new
    [B][Hkv][Dv]) into its page and update the page centroid, then score, select and attend."""
    _ok(lib().vx_block_topk_decode_append(ctypes.byref(geo.c()), ctypes.byref(table.c()), _ptr(q, torch.bfloat16),
                                          _ptr(k_cache, torch.bfloat16), _ptr(v_cache, torch.bfloat16),
                                          _ptr(centroids, torch.bfloat16), _ptr(k_new, torch.bfloat16),
                                          _ptr(v_new, torch.bfloat16), k, mode, seed & (2 ** 64 - 1),
                                          float(sm_scale), score_dims, num_splits, _ptr(out, torch.bfloat16),
                                          _ptr(lse, torch.float32), _ptr(scores_out, torch.float32),
                                          _ptr(sel_out, torch.int32), _ptr(ws), ws.numel() * ws.element_size(),
                                          _ptr(err, torch.int32), _stream(stream)))


def vx_block_topk_decode_persistent(geo: Geometry, table: PageTable, q, k_cache, v_cache, centroids, k: int, out,
                                    ws, lse=None, sm_scale=0.0, scores_out=None, sel_out=None, err=None,
                                    stream=None):
    """The decode step as one persistent kernel (see include/vx.h).  `ws` (uint8,
    vx_workspace_size bytes) must be zero-filled once before its first use here (torch.zeros);
    every call leaves its counters zero again."""
    _ok(lib().vx_block_topk_decode_persistent(ctypes.byref(geo.c()), ctypes.byref(table.c()), _ptr(q, torch.bfloat16),
                                              _ptr(k_cache, torch.bfloat16), _ptr(v_cache, torch.bfloat16),
                                              _ptr(centroids, torch.bfloat16), k, float(sm_scale),
                                              _ptr(out, torch.bfloat16), _ptr(lse, torch.float32),
                                              _ptr(scores_out, torch.float32), _ptr(sel_out, torch.int32), _ptr(ws),
                                              ws.numel() * ws.element_size(), _ptr(err, torch.int32), _stream(stream)))


# ---------------------------------------------------------------------- 8-bit caches and pages
#
# These calls also check shapes and devices, and run on the device their tensors lie on (the
# stream given, or that device's current one), whatever the current device is.

_CODES = {torch.int8: VX_QUANT_INT8, torch.float8_e4m3fn: VX_QUANT_E4M3}


@dataclass
class QuantCache:
    """A cache held in 8 bits: element = code * scale of its page and KV head."""
    k_cache: torch.Tensor  # int8 or float8_e4m3fn [Npool][Hkv][P][D]
    v_cache: torch.Tensor  # the same type and shape
    k_scale: torch.Tensor  # float32 [Npool][Hkv]
    v_scale: torch.Tensor  # float32 [Npool][Hkv]

    def c(self, geo: Geometry) -> vx_quant_cache:
        if self.k_cache.dtype not in _CODES:
            raise TypeError(f"k_cache must be int8 or float8_e4m3fn, got {self.k_cache.dtype}")
        codes = (geo.num_pool_pages, geo.num_kv_heads, geo.page_size, geo.head_dim_qk)
        scales = codes[:2]
        return vx_quant_cache(_CODES[self.k_cache.dtype], _shaped(self.k_cache, "k_cache", codes, self.k_cache.dtype),
                              _shaped(self.v_cache, "v_cache", codes, self.k_cache.dtype),
                              _shaped(self.k_scale, "k_scale", scales, torch.float32),
                              _shaped(self.v_scale, "v_scale", scales, torch.float32))

    def tensors(self):
        return [self.k_cache, self.v_cache, self.k_scale, self.v_scale]


@dataclass
class PagePool:
    """The arrays of a page pool (see include/vx.h); a page is one entry of each."""
    k_cache: torch.Tensor                       # bf16, int8 or float8_e4m3fn [Npool][Hkv][P][Dqk]
    v_cache: Optional[torch.Tensor] = None      # the same type [Npool][Hkv][P][Dv]; None for MLA
    centroids: Optional[torch.Tensor] = None    # bf16 [Npool][Hkv][Dqk]
    k_scale: Optional[torch.Tensor] = None      # float32 [Npool][Hkv], 8-bit pools only
    v_scale: Optional[torch.Tensor] = None

    def c(self, geo: Geometry) -> vx_page_pool:
        dtype = self.k_cache.dtype
        if dtype != torch.bfloat16 and dtype not in _CODES:
            raise TypeError(f"k_cache must be bfloat16, int8 or float8_e4m3fn, got {dtype}")
        n, h = self.k_cache.shape[0], geo.num_kv_heads
        return vx_page_pool(_shaped(self.k_cache, "k_cache", (n, h, geo.page_size, geo.head_dim_qk), dtype),
                            _shaped(self.v_cache, "v_cache", (n, h, geo.page_size, geo.head_dim_v), dtype),
                            _shaped(self.centroids, "centroids", (n, h, geo.head_dim_qk), torch.bfloat16),
                            _shaped(self.k_scale, "k_scale", (n, h), torch.float32),
                            _shaped(self.v_scale, "v_scale", (n, h), torch.float32),
                            1 if dtype in _CODES else 2, n)

    def tensors(self):
        return [t for t in (self.k_cache, self.v_cache, self.centroids, self.k_scale, self.v_scale) if t is not None]


def _shaped(t: Optional[torch.Tensor], name: str, shape, dtype):
    """Pointer of an optional contiguous tensor; None in `shape` stands for any extent."""
    if t is None:
        return None
    _check(t, dtype)
    if t.dim() != len(shape) or any(want is not None and have != want for have, want in zip(t.shape, shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _table_c(geo: Geometry, table: PageTable) -> vx_page_table:
    for name in ("page_ptr", "seq_lens"):
        _shaped(getattr(table, name), name, (geo.batch,), torch.int32)
    return table.c()


def _run(fn, tensors, stream, *args):
    """Call a C entry point on the device that every tensor lies on."""
    device = tensors[0].device
    if device.type != "cuda":
        raise ValueError("libvx works on CUDA tensors")
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"tensors on {device} and on {t.device} in one call")
    if stream is not None and stream.device != device:
        raise ValueError(f"tensors on {device}, stream on {stream.device}")
    with torch.cuda.device(device):
        _ok(fn(*args, (torch.cuda.current_stream() if stream is None else stream).cuda_stream))


def _table_tensors(table: PageTable):
    return [table.page_ptr, table.page_indices, table.seq_lens]


def vx_quant_update(geo: Geometry, table: PageTable, cache: QuantCache, centroids, k_new, v_new, first_pos=None,
                    err=None, stream=None):
    """Quantise one new token per request (k_new, v_new [B][Hkv][D]), or a prefill chunk (k_new,
    v_new [N][Hkv][D] packed in request order, with first_pos), into an 8-bit cache; scales and
    centroids of the pages touched follow.  N is the sum of seq_lens - first_pos."""
    n, h, d = (None if first_pos is not None else geo.batch), geo.num_kv_heads, geo.head_dim_qk
    ptrs = [_shaped(centroids, "centroids", (geo.num_pool_pages, h, d), torch.bfloat16),
            _shaped(k_new, "k_new", (n, h, d), torch.bfloat16), _shaped(v_new, "v_new", (n, h, d), torch.bfloat16),
            _shaped(first_pos, "first_pos", (geo.batch,), torch.int32), _ptr(err, torch.int32)]
    _run(lib().vx_quant_update, [k_new, v_new, centroids, first_pos, err] + cache.tensors() + _table_tensors(table),
         stream, ctypes.byref(geo.c()), ctypes.byref(_table_c(geo, table)), ctypes.byref(cache.c(geo)), *ptrs)


def _query_out(geo: Geometry, q, out, lse):
    rows = (geo.batch, geo.num_q_heads)
    return (_shaped(q, "q", rows + (geo.head_dim_qk,), torch.bfloat16),
            _shaped(out, "out", rows + (geo.head_dim_v,), torch.bfloat16), _shaped(lse, "lse", rows, torch.float32))


def vx_sparse_decode_quant(geo: Geometry, table: PageTable, q, cache: QuantCache, sel, k: int, out, ws, lse=None,
                           sm_scale=0.0, num_splits=0, err=None, stream=None):
    """vx_sparse_decode over an 8-bit cache."""
    pq, po, pl = _query_out(geo, q, out, lse)
    _run(lib().vx_sparse_decode_quant, [q, sel, out, lse, ws, err] + cache.tensors() + _table_tensors(table), stream,
         ctypes.byref(geo.c()), ctypes.byref(_table_c(geo, table)), pq, ctypes.byref(cache.c(geo)),
         _shaped(sel, "sel", (geo.batch, geo.num_kv_heads, k), torch.int32), k, float(sm_scale), num_splits, po, pl,
         _ptr(ws), ws.numel() * ws.element_size(), _ptr(err, torch.int32))


def _chained(geo, table, q, cache, centroids, new, k, out, ws, lse, mode, seed, sm_scale, score_dims, num_splits,
             scores_out, sel_out, err, stream):
    pq, po, pl = _query_out(geo, q, out, lse)
    rows = (geo.batch, geo.num_kv_heads)
    fn = lib().vx_block_topk_decode_append_quant if new else lib().vx_block_topk_decode_quant
    tensors = [q, centroids, *new, out, lse, scores_out, sel_out, ws, err] + cache.tensors() + _table_tensors(table)
    _run(fn, tensors, stream, ctypes.byref(geo.c()), ctypes.byref(_table_c(geo, table)), pq,
         ctypes.byref(cache.c(geo)),
         _shaped(centroids, "centroids", (geo.num_pool_pages, geo.num_kv_heads, geo.head_dim_qk), torch.bfloat16),
         *[_shaped(x, name, rows + (geo.head_dim_qk,), torch.bfloat16) for name, x in zip(("k_new", "v_new"), new)],
         k, mode, seed & (2 ** 64 - 1), float(sm_scale), score_dims, num_splits, po, pl,
         _shaped(scores_out, "scores_out", rows + (table.max_pages,), torch.float32),
         _shaped(sel_out, "sel_out", rows + (k,), torch.int32), _ptr(ws), ws.numel() * ws.element_size(),
         _ptr(err, torch.int32))


def vx_block_topk_decode_quant(geo: Geometry, table: PageTable, q, cache: QuantCache, centroids, k: int, out, ws,
                               lse=None, mode=0, seed=0, sm_scale=0.0, score_dims=0, num_splits=0, scores_out=None,
                               sel_out=None, err=None, stream=None):
    """vx_block_topk_decode over an 8-bit cache: score, select, attend."""
    _chained(geo, table, q, cache, centroids, (), k, out, ws, lse, mode, seed, sm_scale, score_dims, num_splits,
             scores_out, sel_out, err, stream)


def vx_block_topk_decode_append_quant(geo: Geometry, table: PageTable, q, cache: QuantCache, centroids, k_new, v_new,
                                      k: int, out, ws, lse=None, mode=0, seed=0, sm_scale=0.0, score_dims=0,
                                      num_splits=0, scores_out=None, sel_out=None, err=None, stream=None):
    """One appending decode step over an 8-bit cache: quantise each request's new token into its
    page, then score, select and attend."""
    _chained(geo, table, q, cache, centroids, (k_new, v_new), k, out, ws, lse, mode, seed, sm_scale, score_dims,
             num_splits, scores_out, sel_out, err, stream)


def vx_page_workspace_size(geo: Geometry, rows: int) -> int:
    n = lib().vx_page_workspace_size(ctypes.byref(geo.c()), rows)
    if n == 0:
        raise VxError(VX_ERR_INVALID_ARG, lib().vx_last_error().decode())
    return n


def vx_copy_pages(geo: Geometry, src: PagePool, dst: PagePool, src_pages, dst_pages, ws, err=None, stream=None):
    """Page src_pages[i] of `src` to page dst_pages[i] of `dst` (which may be the same pool)."""
    n = src_pages.numel()
    if src.k_cache.dtype != dst.k_cache.dtype:
        raise TypeError("the pools must hold the same type")
    _run(lib().vx_copy_pages, [src_pages, dst_pages, ws, err] + src.tensors() + dst.tensors(), stream,
         ctypes.byref(geo.c()), ctypes.byref(src.c(geo)), ctypes.byref(dst.c(geo)),
         _shaped(src_pages, "src_pages", (n,), torch.int32), _shaped(dst_pages, "dst_pages", (n,), torch.int32), n,
         _ptr(ws), ws.numel() * ws.element_size(), _ptr(err, torch.int32))


def vx_update_table(geo: Geometry, pool: PagePool, table: PageTable, ref, parent, grow, new_table: PageTable, new_ref,
                    ws, err=None, stream=None):
    """New rows of a page table: row i takes over the tokens of row parent[i] (-1: none) and gets
    room for grow[i] more; new_table.page_ptr is an input, its page_indices and seq_lens and
    new_ref (which may be ref) are written."""
    rows, pages = parent.numel(), (geo.num_pool_pages,)
    _run(lib().vx_update_table,
         [ref, new_ref, parent, grow, ws, err] + pool.tensors() + _table_tensors(table) + _table_tensors(new_table),
         stream, ctypes.byref(geo.c()), ctypes.byref(pool.c(geo)), ctypes.byref(_table_c(geo, table)),
         _shaped(ref, "ref", pages, torch.int32), _shaped(parent, "parent", (rows,), torch.int32),
         _shaped(grow, "grow", (rows,), torch.int32), rows,
         _shaped(new_table.page_ptr, "new page_ptr", (rows,), torch.int32), _ptr(new_table.page_indices, torch.int32),
         new_table.page_indices.numel(), _shaped(new_table.seq_lens, "new seq_lens", (rows,), torch.int32),
         new_table.max_pages, _shaped(new_ref, "new_ref", pages, torch.int32), _ptr(ws),
         ws.numel() * ws.element_size(), _ptr(err, torch.int32))


def vx_compact_pages(geo: Geometry, pool: PagePool, table: PageTable, ref, new_indices, new_ref, remap, num_live, ws,
                     err=None, stream=None):
    """Move every live page (ref > 0) into the lowest ids; new_indices and new_ref may be
    table.page_indices and ref."""
    pages = (geo.num_pool_pages,)
    _run(lib().vx_compact_pages,
         [ref, new_indices, new_ref, remap, num_live, ws, err] + pool.tensors() + _table_tensors(table), stream,
         ctypes.byref(geo.c()), ctypes.byref(pool.c(geo)), ctypes.byref(_table_c(geo, table)),
         _shaped(ref, "ref", pages, torch.int32),
         _shaped(new_indices, "new_indices", tuple(table.page_indices.shape), torch.int32),
         _shaped(new_ref, "new_ref", pages, torch.int32), _shaped(remap, "remap", pages, torch.int32),
         _shaped(num_live, "num_live", (1,), torch.int32), _ptr(ws), ws.numel() * ws.element_size(),
         _ptr(err, torch.int32))
