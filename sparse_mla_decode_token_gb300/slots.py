"""Slot maps of a step, built on the GPU from request lengths (argument marshalling
only): offsets, positions and physical slots of the new tokens, and the index
tables of ``sparse_mla_decode`` from page tables.  The calls are
``smla_token_slots`` and ``smla_sparse_slots`` of ``include/smla.h``, which
defines them; plain tensors go through the extension module.

    step = token_slots(lens, new_lens, tables, max_tokens=T, page_size=64)
    indices, topk_lens = sparse_slots(new_lens, tables, T, page_size=64, cum_seq_lens_q=step.cum_seq_lens_q,
                                      selected=picks, compressed_tables=comp_tables, compressed_page_size=64,
                                      compress_ratio=4)
    out, lse = sparse_mla_decode(q, swa_kv, ws, indices, compressed_kv, topk_lens, new_lens,
                                 cum_seq_lens_q=step.cum_seq_lens_q)
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import binding as _b
from . import cache as _cache
from .binding import SWA_COLS, _c_void_p, _ptr
from .cache import _call, _int32, _on, _table, _words

_i32, _i64 = ctypes.c_int32, ctypes.c_int64


class SmlaTokenSlotsArgs(ctypes.Structure):
    _fields_ = [
        ("lens", _c_void_p), ("new_lens", _c_void_p), ("batch", _i32), ("max_tokens", _i32),
        ("block_tables", _c_void_p), ("block_table_stride", _i64), ("max_pages", _i32), ("page_size", _i32),
        ("cum_seq_lens_q", _c_void_p), ("requests", _c_void_p), ("positions", _c_void_p), ("slots", _c_void_p),
        ("error_word", _c_void_p),
    ]


class SmlaSparseSlotsArgs(ctypes.Structure):
    _fields_ = [
        ("sum_q", _i32), ("batch", _i32), ("seq_lens", _c_void_p), ("cum_seq_lens_q", _c_void_p),
        ("swa_tables", _c_void_p), ("swa_table_stride", _i64), ("swa_max_pages", _i32), ("swa_page_size", _i32),
        ("comp_tables", _c_void_p), ("comp_table_stride", _i64), ("comp_max_pages", _i32), ("comp_page_size", _i32),
        ("compress_ratio", _i32), ("num_selected", _i32), ("selected", _c_void_p), ("selected_stride", _i64),
        ("sparse_indices", _c_void_p), ("indices_row_stride", _i64), ("topk_lens", _c_void_p), ("error_word", _c_void_p),
    ]


class StepSlots(NamedTuple):
    """A step's tokens: offsets ``[B + 1]``, and of each token its request,
    position and physical slot (int64, as indexing takes them; None without
    tables); -1 behind the last one."""
    cum_seq_lens_q: torch.Tensor
    requests: torch.Tensor
    positions: torch.Tensor
    slots: Optional[torch.Tensor]


def token_slots(lens: torch.Tensor, new_lens: torch.Tensor, block_tables: Optional[torch.Tensor] = None, *, max_tokens: int,
                page_size: int = 1, out: Optional[StepSlots] = None, error_word: Optional[torch.Tensor] = None,
                stream: Optional[int] = None) -> StepSlots:
    """Offsets, requests, positions and slots of the tokens that take each request
    from ``lens`` to ``new_lens`` (allocated when ``out`` is not given)."""
    done = (_cache._extension or _cache.extension()).token_slots(lens, new_lens, block_tables, max_tokens, page_size, out,
                                                                 error_word, stream)
    if done.__class__ is tuple:
        return StepSlots._make(done)
    if done is not None:
        _b._check(done)
    max_tokens, batch = _int32("max_tokens", max_tokens), lens.numel()
    if max_tokens < 0:
        raise ValueError(f"max_tokens {max_tokens} is negative")
    _words("lens", lens, 0)
    _words("new_lens", new_lens, batch)
    index = lens.get_device()
    if out is None:
        with _b._allocate_for(stream, index):
            new = lambda n, dtype: torch.empty(n, dtype=dtype, device=lens.device)
            out = StepSlots(new(batch + 1, torch.int32), new(max_tokens, torch.int32), new(max_tokens, torch.int32),
                            None if block_tables is None else new(max_tokens, torch.int64))
    _words("cum_seq_lens_q", out.cum_seq_lens_q, batch + 1)
    _words("requests", out.requests, max_tokens)
    _words("positions", out.positions, max_tokens)
    _words("slots", out.slots, max_tokens, torch.int64)
    _words("error_word", error_word, 1)
    a = SmlaTokenSlotsArgs(lens.data_ptr(), new_lens.data_ptr(), batch, max_tokens)
    if block_tables is None:
        if out.slots is not None:
            raise ValueError("slots need block_tables")
    else:
        _table("block_tables", block_tables)
        if block_tables.shape[0] < batch:
            raise ValueError(f"block_tables has {block_tables.shape[0]} rows for {batch} requests")
        a.block_tables, a.max_pages, a.page_size = block_tables.data_ptr(), block_tables.shape[1], _int32("page_size", page_size)
        a.block_table_stride = block_tables.stride(0) if block_tables.shape[0] > 1 else a.max_pages
    a.cum_seq_lens_q, a.requests, a.positions = out.cum_seq_lens_q.data_ptr(), _ptr(out.requests), _ptr(out.positions)
    a.slots, a.error_word = _ptr(out.slots), _ptr(error_word)
    _on(index, (lens, new_lens, block_tables, *out, error_word),
        ("lens", "new_lens", "block_tables", "cum_seq_lens_q", "requests", "positions", "slots", "error_word"))
    _call(_b.lib().smla_token_slots, index, stream, ctypes.byref(a))
    return out


def sparse_slots(seq_lens: torch.Tensor, swa_tables: torch.Tensor, num_tokens: int, *, page_size: int,
                 cum_seq_lens_q: Optional[torch.Tensor] = None, selected: Optional[torch.Tensor] = None, num_selected: int = 0,
                 compressed_tables: Optional[torch.Tensor] = None, compressed_page_size: int = 1, compress_ratio: int = 1,
                 sparse_indices: Optional[torch.Tensor] = None, topk_lens: Optional[torch.Tensor] = None,
                 error_word: Optional[torch.Tensor] = None, stream: Optional[int] = None):
    """The combined index table ``[num_tokens, 128 + K]`` of ``sparse_mla_decode``
    and its ``sparse_topk_lens``: each token's last 128 positions through
    ``swa_tables``, then the compressed positions ``selected`` ``[num_tokens, K]``
    (-1: none), or without them the first ``num_selected``, through
    ``compressed_tables``; returns both, allocated when not given."""
    done = (_cache._extension or _cache.extension()).sparse_slots(
        seq_lens, swa_tables, num_tokens, page_size, cum_seq_lens_q, selected, num_selected, compressed_tables,
        compressed_page_size, compress_ratio, sparse_indices, topk_lens, error_word, stream)
    if done.__class__ is tuple:
        return done
    if done is not None:
        _b._check(done)
    _table("swa_tables", swa_tables)
    batch, T = swa_tables.shape[0], _int32("num_tokens", num_tokens)
    if T < 0:
        raise ValueError(f"num_tokens {T} is negative")
    _words("seq_lens", seq_lens, batch)
    if cum_seq_lens_q is not None:
        _words("cum_seq_lens_q", cum_seq_lens_q, batch + 1)
    a = SmlaSparseSlotsArgs(T, batch, seq_lens.data_ptr(), _ptr(cum_seq_lens_q), swa_tables.data_ptr(),
                            swa_tables.stride(0) if batch > 1 else 0, swa_tables.shape[1], _int32("page_size", page_size))
    a.compress_ratio, a.num_selected = _int32("compress_ratio", compress_ratio), _int32("num_selected", num_selected)
    if selected is not None:
        if selected.dtype != torch.int32:
            raise TypeError("selected must be int32")
        if selected.dim() != 2 or selected.shape[0] != T or (selected.shape[1] > 1 and selected.stride(1) != 1):
            raise ValueError(f"selected must be [{T}, K] with contiguous rows; got {tuple(selected.shape)}")
        if T > 1 and selected.stride(0) < selected.shape[1]:
            raise ValueError("selected: rows overlap")
        a.num_selected = selected.shape[1]
        a.selected, a.selected_stride = selected.data_ptr(), selected.stride(0) if T > 1 else 0
    if a.num_selected < 0:
        raise ValueError(f"num_selected {a.num_selected} is negative")
    if compressed_tables is not None:
        _table("compressed_tables", compressed_tables)
        if compressed_tables.shape[0] != batch:
            raise ValueError(f"compressed_tables has {compressed_tables.shape[0]} rows for {batch} requests")
        a.comp_tables, a.comp_max_pages = compressed_tables.data_ptr(), compressed_tables.shape[1]
        a.comp_table_stride = compressed_tables.stride(0) if batch > 1 else 0
        a.comp_page_size = _int32("compressed_page_size", compressed_page_size)
    elif a.num_selected > 0:
        raise ValueError("compressed columns need compressed_tables")
    columns, index = SWA_COLS + a.num_selected, swa_tables.get_device()
    with _b._allocate_for(stream, index):
        if sparse_indices is None:
            sparse_indices = torch.empty((T, columns), dtype=torch.int32, device=swa_tables.device)
        if topk_lens is None:
            topk_lens = torch.empty(T, dtype=torch.int32, device=swa_tables.device)
    if sparse_indices.dtype != torch.int32:
        raise TypeError("sparse_indices must be int32")
    if sparse_indices.dim() != 2 or tuple(sparse_indices.shape) != (T, columns) or sparse_indices.stride(1) != 1 or \
            (T > 1 and sparse_indices.stride(0) < columns):
        raise ValueError(f"sparse_indices must be [{T}, {columns}] with contiguous rows; got {tuple(sparse_indices.shape)}")
    _words("topk_lens", topk_lens, T)
    _words("error_word", error_word, 1)
    a.sparse_indices, a.indices_row_stride = sparse_indices.data_ptr(), sparse_indices.stride(0) if T > 1 else columns
    a.topk_lens, a.error_word = topk_lens.data_ptr(), _ptr(error_word)
    _on(index, (seq_lens, swa_tables, cum_seq_lens_q, selected, compressed_tables, sparse_indices, topk_lens, error_word),
        ("seq_lens", "swa_tables", "cum_seq_lens_q", "selected", "compressed_tables", "sparse_indices", "topk_lens", "error_word"))
    _call(_b.lib().smla_sparse_slots, index, stream, ctypes.byref(a))
    return sparse_indices, topk_lens
