"""Binding of the attention layers' entry points (``include/gdn.h``): the
tables of a step, the paged 8-bit K / V cache and the attention that reads it.
Imported into the package's namespace, like the GDN layers' functions."""
from __future__ import annotations

import ctypes
from functools import lru_cache
from typing import Optional

import torch

from . import _check, _dev, _P, _Pool, _stream, _stream_object, load_library, workspace_for
from .inputs import AttnShape

ATTN_DECODE_ROWS = 32    # GDN_ATTN_DECODE_ROWS
KV_BLOCK = 16            # GDN_KV_BLOCK

_i32, _i64 = ctypes.c_int32, ctypes.c_int64


class _AttnDesc(ctypes.Structure):
    _fields_ = [("num_q_heads", _i32), ("num_kv_heads", _i32), ("head_dim", _i32), ("page_tokens", _i32),
                ("dtype", _i32), ("scale", ctypes.c_float), ("reserved", _i32)]


class _KvTablesArgs(ctypes.Structure):
    _fields_ = [("num_seqs", _i32), ("max_pages", _i32), ("num_free", _i32), ("num_pages", _i32),
                ("total_tokens", _i64), ("kv_len", _P), ("new_len", _P), ("free_pages", _P), ("block_table", _P),
                ("cu_seqlens", _P), ("cu_kv", _P), ("kv_len_out", _P), ("positions", _P), ("slot_map", _P),
                ("pages_taken", _P), ("dev_error", _P)]


class _KvAppendArgs(ctypes.Structure):
    _fields_ = [("total_tokens", _i64), ("k_stride", _i64), ("v_stride", _i64), ("k", _P), ("v", _P),
                ("slot_map", _P), ("dev_error", _P)]


class _KvGatherArgs(ctypes.Structure):
    _fields_ = [("num_seqs", _i32), ("max_pages", _i32), ("total_tokens", _i64), ("cu_kv", _P), ("block_table", _P),
                ("k", _P), ("v", _P), ("dev_error", _P)]


class _AttnDecodeArgs(ctypes.Structure):
    _fields_ = [("num_seqs", _i32), ("max_pages", _i32), ("max_q_len", _i32), ("max_kv_len", _i32),
                ("total_tokens", _i64), ("q_stride", _i64), ("cu_seqlens", _P), ("kv_len", _P), ("block_table", _P),
                ("q", _P), ("o", _P), ("lse", _P), ("dev_error", _P), ("wait_cycles", _i64)]


class _AttnPrefillArgs(ctypes.Structure):
    _fields_ = [("num_seqs", _i32), ("max_q_len", _i32), ("max_kv_len", _i32), ("reserved", _i32), ("total_q", _i64),
                ("total_kv", _i64), ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64), ("cu_seqlens", _P),
                ("cu_kv", _P), ("q", _P), ("k", _P), ("v", _P), ("o", _P), ("lse", _P), ("dev_error", _P),
                ("wait_cycles", _i64)]


def _signatures() -> dict:
    D, PL, ptr, sz = ctypes.POINTER(_AttnDesc), ctypes.POINTER(_Pool), ctypes.POINTER, ctypes.c_size_t
    return {
        "gdn_kv_page_bytes": ([D], _i64),
        "gdn_kv_tables": ([D, ptr(_KvTablesArgs), _P], _i32),
        "gdn_kv_append": ([D, PL, ptr(_KvAppendArgs), _P], _i32),
        "gdn_kv_gather": ([D, PL, ptr(_KvGatherArgs), _P], _i32),
        "gdn_attn_decode_workspace_size": ([D, _i32, _i64, _i32], sz),
        "gdn_attn_decode": ([D, PL, ptr(_AttnDecodeArgs), _P, sz, _P], _i32),
        "gdn_attn_prefill": ([D, ptr(_AttnPrefillArgs), _P], _i32),
    }


@lru_cache(maxsize=256)
def make_attn_desc(shape: AttnShape) -> _AttnDesc:
    return _AttnDesc(shape.num_q_heads, shape.num_kv_heads, shape.head_dim, shape.page_tokens, shape.dtype,
                     shape.softmax_scale, 0)


def gdn_kv_page_bytes(shape: AttnShape) -> int:
    return int(load_library().gdn_kv_page_bytes(ctypes.byref(make_attn_desc(shape))))


class KVPool:
    """A pool of KV pages in one device tensor (PyTorch owns the memory).

    ``buf`` takes an existing uint8 tensor of num_pages x page_bytes instead
    of allocating one; ``page_bytes`` may exceed the shape's own, so that KV
    pages share a pool with GDN state pages."""

    def __init__(self, shape: AttnShape, num_pages: int, device="cuda", fill: Optional[int] = None,
                 page_bytes: int = 0, buf: Optional[torch.Tensor] = None):
        self.shape = shape
        self.num_pages = int(num_pages)
        self.page_bytes = int(page_bytes) or shape.page_bytes
        if buf is None:
            size = self.num_pages * self.page_bytes
            self.storage = torch.empty(size + 256, dtype=torch.uint8, device=device)
            if fill is not None:
                self.storage.fill_(fill)
            off = (-self.storage.data_ptr()) % 256
            buf = self.storage[off:off + size]
        if buf.dtype != torch.uint8 or not buf.is_contiguous() or buf.numel() != self.num_pages * self.page_bytes:
            raise ValueError("buf: expected a contiguous uint8 tensor of num_pages x page_bytes")
        self.buf = buf.view(self.num_pages, self.page_bytes)
        self._abi = _Pool(self.buf.data_ptr(), self.page_bytes, self.num_pages, 0)

    def abi(self) -> _Pool:
        return self._abi

    def _blocks(self):
        return self.shape.num_kv_heads, self.shape.page_tokens // KV_BLOCK

    def k_codes(self) -> torch.Tensor:
        """e4m3 [pages][Hkv][blocks][2][d/16][8][16]"""
        n, d = self.shape.codes_bytes, self.shape.head_dim
        return self.buf[:, :n].unflatten(1, self._blocks() + (2, d // 16, 8, 16)).view(torch.float8_e4m3fn)

    def v_codes(self) -> torch.Tensor:
        """e4m3 [pages][Hkv][blocks][d][16]"""
        n, d = self.shape.codes_bytes, self.shape.head_dim
        return self.buf[:, n:2 * n].unflatten(1, self._blocks() + (d, KV_BLOCK)).view(torch.float8_e4m3fn)

    def _scales(self, i: int) -> torch.Tensor:
        o, n = self.shape.codes_bytes // 2, self._blocks()[0] * self._blocks()[1]
        return self.buf.view(torch.float32)[:, o + i * n:o + (i + 1) * n].unflatten(1, self._blocks())

    def k_scales(self) -> torch.Tensor:
        """fp32 [pages][Hkv][blocks]"""
        return self._scales(0)

    def v_scales(self) -> torch.Tensor:
        return self._scales(1)


# the current stream of a device as an integer (the public call makes a Stream object: 3 us of a 13 us call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(stream, t: torch.Tensor) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(t.get_device())
    return _stream(stream)


def _rows(t: torch.Tensor, heads: int, shape: AttnShape, name: str):
    """(pointer, elements between rows) of [T, heads, d] rows that may be slices of wider ones."""
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.dtype != shape.torch_dtype():
        raise ValueError(f"{name}: expected {shape.torch_dtype()}, got {t.dtype}")
    d = shape.head_dim
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != d:
        raise ValueError(f"{name}: expected [T, {heads}, {d}], got {tuple(t.shape)}")
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != d):
        raise ValueError(f"{name}: a row's heads must be dense")
    return t.data_ptr(), (s[0] if t.shape[0] > 1 else heads * d)


def _table(t: Optional[torch.Tensor], n: int):
    """(pointer, columns) of a block table [N, max_pages]."""
    if t is None or t.numel() == 0:
        return None, 0
    if t.dim() != 2 or t.shape[0] != n:
        raise ValueError(f"block_table: expected [{n}, max_pages], got {tuple(t.shape)}")
    return _dev(t, torch.int32, "block_table"), int(t.shape[1])


def _ints(t: torch.Tensor, n: int, name: str, dtype=torch.int32):
    if t.numel() != n:
        raise ValueError(f"{name}: expected {n} entries, got {t.numel()}")
    return _dev(t, dtype, name)


def _out(t: Optional[torch.Tensor], shape, dtype, name: str):
    if t is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name}: expected {shape}, got {tuple(t.shape)}")
    return _dev(t, dtype, name)


def gdn_kv_tables(shape: AttnShape, num_pages: int, *, kv_len, new_len, free_pages, block_table, cu_seqlens, cu_kv,
                  kv_len_out, positions, slot_map, pages_taken, dev_error, stream=None,
                  raise_on_error: bool = True) -> int:
    """Block tables, slot map and positions of a step from request lengths
    (gdn.h: gdn_kv_tables).  slot_map and positions may have more rows than
    the step has tokens: the rest get slot -1.  A step without requests gives
    sums of 0, no pages taken and only such rows (the C entry launches nothing
    for it and leaves the outputs alone)."""
    n, T = int(kv_len.numel()), int(slot_map.numel())
    bt, cols = _table(block_table, n)
    a = _KvTablesArgs(n, cols, int(free_pages.numel()), int(num_pages), T, _dev(kv_len, torch.int32, "kv_len"),
                      _ints(new_len, n, "new_len"), _dev(free_pages, torch.int32, "free_pages"), bt,
                      _ints(cu_seqlens, n + 1, "cu_seqlens"), _ints(cu_kv, n + 1, "cu_kv"),
                      _ints(kv_len_out, n, "kv_len_out"), _ints(positions, T, "positions", torch.int64),
                      _dev(slot_map, torch.int64, "slot_map"), _ints(pages_taken, 1, "pages_taken"),
                      _ints(dev_error, 1, "dev_error"))
    if n == 0:
        with torch.cuda.stream(_stream_object(stream, slot_map.device)):
            for t in (cu_seqlens, cu_kv, pages_taken, positions):
                t.zero_()
            slot_map.fill_(-1)
    st = load_library().gdn_kv_tables(make_attn_desc(shape), a, _on(stream, kv_len))
    return _check(st, "gdn_kv_tables") if raise_on_error else st


def gdn_kv_append(shape: AttnShape, pool: KVPool, *, k, v, slot_map, dev_error, stream=None,
                  raise_on_error: bool = True) -> int:
    """New K and V rows [T, Hkv, d] (slices of wider rows are fine) into the
    8-bit cache at slot_map's slots (gdn.h: gdn_kv_append)."""
    kp, ks = _rows(k, shape.num_kv_heads, shape, "k")
    vp, vs = _rows(v, shape.num_kv_heads, shape, "v")
    T = int(k.shape[0])
    if v.shape[0] != T:
        raise ValueError(f"v: expected {T} rows, got {v.shape[0]}")
    a = _KvAppendArgs(T, ks, vs, kp, vp, _ints(slot_map, T, "slot_map", torch.int64), _ints(dev_error, 1, "dev_error"))
    st = load_library().gdn_kv_append(make_attn_desc(shape), pool.abi(), a, _on(stream, k))
    return _check(st, "gdn_kv_append") if raise_on_error else st


def gdn_kv_gather(shape: AttnShape, pool: KVPool, *, cu_kv, block_table, k, v, dev_error, stream=None,
                  raise_on_error: bool = True) -> int:
    """Cached tokens 0 .. L_s - 1 of every sequence back as rows of k and v
    [T, Hkv, d] (gdn.h: gdn_kv_gather)."""
    n, T = int(cu_kv.numel()) - 1, int(k.shape[0])
    bt, cols = _table(block_table, n)
    rows = (T, shape.num_kv_heads, shape.head_dim)
    a = _KvGatherArgs(n, cols, T, _dev(cu_kv, torch.int32, "cu_kv"), bt, _out(k, rows, shape.torch_dtype(), "k"),
                      _out(v, rows, shape.torch_dtype(), "v"), _ints(dev_error, 1, "dev_error"))
    st = load_library().gdn_kv_gather(make_attn_desc(shape), pool.abi(), a, _on(stream, k))
    return _check(st, "gdn_kv_gather") if raise_on_error else st


def gdn_attn_decode_workspace_size(shape: AttnShape, num_seqs: int, total_tokens: int, max_kv_len: int) -> int:
    return int(load_library().gdn_attn_decode_workspace_size(make_attn_desc(shape), num_seqs, total_tokens, max_kv_len))


def gdn_attn_decode(shape: AttnShape, pool: KVPool, *, q, cu_seqlens, kv_len, block_table, o, dev_error, lse=None,
                    max_q_len: int = 1, max_kv_len: Optional[int] = None, workspace=None, wait_cycles: int = 0,
                    stream=None, raise_on_error: bool = True) -> int:
    """Attention of 1 to 32 new rows a sequence over the 8-bit cache (gdn.h:
    gdn_attn_decode).  max_kv_len bounds kv_len (None: what the block table
    can hold).  Without `workspace` one of gdn_attn_decode_workspace_size
    bytes is taken from PyTorch's allocator for the call.  wait_cycles bounds
    the device-side waits (gdn.h)."""
    lib = load_library()
    n = int(kv_len.numel())
    qp, qs = _rows(q, shape.num_q_heads, shape, "q")
    T = int(q.shape[0])
    bt, cols = _table(block_table, n)
    if max_kv_len is None:
        max_kv_len = min(cols * shape.page_tokens, 0x7fffffff)
    desc = make_attn_desc(shape)
    if workspace is None:
        size = lib.gdn_attn_decode_workspace_size(desc, n, T, max_kv_len)
        workspace = workspace_for(size, q.device, stream)
    a = _AttnDecodeArgs(n, cols, int(max_q_len), int(max_kv_len), T, qs, _ints(cu_seqlens, n + 1, "cu_seqlens"),
                        _dev(kv_len, torch.int32, "kv_len"), bt, qp,
                        _out(o, (T, shape.num_q_heads, shape.head_dim), shape.torch_dtype(), "o"),
                        _out(lse, (T, shape.num_q_heads), torch.float32, "lse"), _ints(dev_error, 1, "dev_error"),
                        int(wait_cycles))
    st = lib.gdn_attn_decode(desc, pool.abi(), a, _dev(workspace, None, "workspace"),
                             workspace.numel() * workspace.element_size(), _on(stream, q))
    return _check(st, "gdn_attn_decode") if raise_on_error else st


def gdn_attn_prefill(shape: AttnShape, *, q, k, v, cu_seqlens, cu_kv, o, dev_error, lse=None, max_q_len: int = 0,
                     max_kv_len: int = 0, wait_cycles: int = 0, stream=None, raise_on_error: bool = True) -> int:
    """Causal attention of packed rows q [Tq, Hq, d] over k, v [Tk, Hkv, d]
    (slices of wider rows are fine; gdn.h: gdn_attn_prefill).  max_q_len and
    max_kv_len (the longest sequence; 0: the call's totals) bound a sequence;
    with the longest one's rows the launch starts the tiles with the most keys
    first."""
    n = int(cu_seqlens.numel()) - 1
    qp, qs = _rows(q, shape.num_q_heads, shape, "q")
    kp, ks = _rows(k, shape.num_kv_heads, shape, "k")
    vp, vs = _rows(v, shape.num_kv_heads, shape, "v")
    Tq, Tk = int(q.shape[0]), int(k.shape[0])
    if v.shape[0] != Tk:
        raise ValueError(f"v: expected {Tk} rows, got {v.shape[0]}")
    a = _AttnPrefillArgs(n, int(max_q_len), int(max_kv_len), 0, Tq, Tk, qs, ks, vs,
                         _dev(cu_seqlens, torch.int32, "cu_seqlens"), _ints(cu_kv, n + 1, "cu_kv"), qp, kp, vp,
                         _out(o, (Tq, shape.num_q_heads, shape.head_dim), shape.torch_dtype(), "o"),
                         _out(lse, (Tq, shape.num_q_heads), torch.float32, "lse"), _ints(dev_error, 1, "dev_error"),
                         int(wait_cycles))
    st = load_library().gdn_attn_prefill(make_attn_desc(shape), a, _on(stream, q))
    return _check(st, "gdn_attn_prefill") if raise_on_error else st
