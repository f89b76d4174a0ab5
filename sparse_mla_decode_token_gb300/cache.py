"""The paged latent cache: tensor-level calls (argument marshalling only).

A cache is what the caller owns: E4M3 rows ``[num_pages, page_size, 512]``,
float32 scales ``[num_pages, page_size // block_rows]`` (one per block of
tokens), int32 page tables ``[requests, max_pages]``, lengths ``[requests]``
and, for the page calls, a count per page (0 = free).  The calls are the
``smla_window_*``, ``smla_cache_*`` and ``smla_pages_*`` entry points of
``include/smla.h``, which defines them; all work on the device, on the current
stream unless ``stream`` is given, and none waits.

    pages_resize(tables, refs, lens, new_lens, ws, page_size=64, moves=moves)   # pages for the new tokens
    pages_copy([rows, scales], moves)                                           # shared pages about to be written
    append(latent, rows, scales, tables, new_lens, cum_seq_lens_q=cum)          # quantise them in
    out, lse = window_attention(q, rows, scales, tables, new_lens, ws2, window=1024, first_tokens=4,
                                cum_seq_lens_q=cum, bmm1_scale=scale)
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Sequence

import torch

from . import binding as _b
from .binding import HEAD_DIM, _c_void_p, _check, _ptr

_i32, _i64, _size = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class SmlaCache(ctypes.Structure):
    _fields_ = [
        ("rows", _c_void_p), ("row_stride", _i64), ("page_stride", _i64),
        ("scales", _c_void_p), ("scale_stride", _i64),
        ("num_pages", _i64), ("page_size", _i32), ("block_rows", _i32),
        ("block_tables", _c_void_p), ("block_table_stride", _i64), ("max_pages", _i32), ("batch", _i32),
        ("seq_lens", _c_void_p), ("cum_seq_lens_q", _c_void_p),
    ]


class SmlaWindowArgs(ctypes.Structure):
    _fields_ = [
        ("cache", SmlaCache),
        ("sum_q", _i32), ("num_heads", _i32), ("window", _i32), ("first_tokens", _i32),
        ("q", _c_void_p), ("q_stride_token", _i64), ("sinks", _c_void_p),
        ("bmm1_scale", ctypes.c_float), ("bmm2_scale", ctypes.c_float),
        ("bmm1_scale_dev", _c_void_p), ("bmm2_scale_dev", _c_void_p),
        ("out", _c_void_p), ("out_lse", _c_void_p),
        ("workspace", _c_void_p), ("workspace_bytes", _size),
        ("num_splits", _i32), ("error_word", _c_void_p),
    ]


class SmlaAppendArgs(ctypes.Structure):
    _fields_ = [
        ("cache", SmlaCache),
        ("sum_q", _i32), ("latent", _c_void_p), ("latent_stride", _i64), ("error_word", _c_void_p),
    ]


class SmlaPagesArgs(ctypes.Structure):
    _fields_ = [
        ("block_tables", _c_void_p), ("block_table_stride", _i64),
        ("rows", _i32), ("max_pages", _i32), ("page_size", _i32),
        ("ref_counts", _c_void_p), ("num_pages", _i64),
        ("lens", _c_void_p), ("new_lens", _c_void_p), ("parents", _c_void_p), ("out_lens", _c_void_p),
        ("move_src", _c_void_p), ("move_dst", _c_void_p), ("move_count", _c_void_p), ("move_capacity", _i64),
        ("workspace", _c_void_p), ("workspace_bytes", _size), ("error_word", _c_void_p),
    ]


class SmlaPool(ctypes.Structure):
    _fields_ = [("base", _c_void_p), ("page_bytes", _i64), ("page_stride", _i64)]


class PageMoves(NamedTuple):
    """Pairs of pages to copy: ``src[i]`` to ``dst[i]`` for ``i < count[0]`` (all on the device)."""
    src: torch.Tensor
    dst: torch.Tensor
    count: torch.Tensor


def new_moves(capacity: int, device) -> PageMoves:
    """Moves for ``pages_resize`` (capacity >= requests) or ``pages_compact`` (>= num_pages // 2)."""
    return PageMoves(torch.full((capacity,), -1, dtype=torch.int32, device=device),
                     torch.full((capacity,), -1, dtype=torch.int32, device=device),
                     torch.zeros(1, dtype=torch.int32, device=device))


def _words(name: str, t: Optional[torch.Tensor], need: int, dtype=torch.int32) -> None:
    """An array that the kernels index: its type, contiguous, long enough."""
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < need:
        raise ValueError(f"{name} has {t.numel()} entries; the call reads {need}")


def _placed(device, **tensors) -> None:
    for name, t in tensors.items():
        if isinstance(t, torch.Tensor) and (t.device.type != "cuda" or t.device != device):
            raise ValueError(f"{name} is on {t.device}; every tensor must be on one CUDA device ({device})")


def _table(name: str, t: torch.Tensor) -> None:
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if t.dim() != 2 or t.shape[1] < 1 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [requests, max_pages] with a contiguous last dim")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: rows overlap")


def _row_stride(t: torch.Tensor) -> int:
    """Stride of the leading dim (a single row has none that matters: the dense one)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _stream(stream: Optional[int]):
    return _c_void_p(torch.cuda.current_stream().cuda_stream if stream is None else stream)


def _cache(rows: torch.Tensor, scales: torch.Tensor, tables: torch.Tensor, seq_lens: torch.Tensor,
           cum: Optional[torch.Tensor]) -> SmlaCache:
    if rows.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError(f"cache rows are float8_e4m3fn (or its bytes); got {rows.dtype}")
    if rows.dim() != 3 or rows.shape[2] != HEAD_DIM or rows.stride(2) != 1:
        raise ValueError(f"cache rows must be [num_pages, page_size, {HEAD_DIM}] with contiguous rows; "
                         f"got {tuple(rows.shape)}")
    if scales.dtype != torch.float32:
        raise TypeError("cache scales must be float32")
    if scales.dim() != 2 or scales.shape[0] != rows.shape[0] or scales.shape[1] < 1 or \
            (scales.shape[1] > 1 and scales.stride(1) != 1):
        raise ValueError("cache scales must be [num_pages, page_size // block_rows] with a contiguous last dim")
    if rows.shape[0] < 1 or rows.shape[1] % scales.shape[1] != 0:
        raise ValueError(f"{scales.shape[1]} scales do not divide a page of {rows.shape[1]} rows")
    if (rows.shape[0] > 1 and rows.stride(0) <= 0) or (rows.shape[1] > 1 and rows.stride(1) <= 0) or \
            (scales.shape[0] > 1 and scales.stride(0) <= 0):
        raise ValueError("cache pages must not share memory")
    _table("block_tables", tables)
    if tables.shape[0] < 1:
        raise ValueError("block_tables has no rows")
    batch = tables.shape[0]
    _words("seq_lens", seq_lens, batch)
    _words("cum_seq_lens_q", cum, batch + 1)
    c = SmlaCache()
    c.num_pages, c.page_size = rows.shape[0], rows.shape[1]
    c.block_rows = rows.shape[1] // scales.shape[1]
    c.rows = rows.data_ptr()
    c.row_stride = rows.stride(1) if rows.shape[1] > 1 else HEAD_DIM
    c.page_stride = rows.stride(0) if rows.shape[0] > 1 else 0
    c.scales, c.scale_stride = scales.data_ptr(), _row_stride(scales)
    c.block_tables, c.block_table_stride = tables.data_ptr(), _row_stride(tables)
    c.max_pages, c.batch = tables.shape[1], batch
    c.seq_lens, c.cum_seq_lens_q = seq_lens.data_ptr(), _ptr(cum)
    return c


def _window_args(q, rows, scales, tables, seq_lens, cum, sinks, window, first_tokens, num_splits) -> SmlaWindowArgs:
    if q.dtype != torch.bfloat16:
        raise TypeError(f"q must be bfloat16; got {q.dtype}")
    if q.dim() != 3 or q.shape[2] != HEAD_DIM or q.stride(2) != 1 or (q.shape[1] > 1 and q.stride(1) != HEAD_DIM):
        raise ValueError(f"q must be [T, H, {HEAD_DIM}] with contiguous heads; got {tuple(q.shape)}")
    a = SmlaWindowArgs()
    a.cache = _cache(rows, scales, tables, seq_lens, cum)
    a.sum_q, a.num_heads = q.shape[0], q.shape[1]
    a.window, a.first_tokens, a.num_splits = int(window), int(first_tokens), int(num_splits)
    a.q, a.q_stride_token = q.data_ptr(), q.stride(0) if q.shape[0] > 1 else 0
    _words("sinks", sinks, a.num_heads, torch.float32)
    a.sinks = _ptr(sinks)
    return a


def window_workspace_size(q: torch.Tensor, rows: torch.Tensor, scales: torch.Tensor, block_tables: torch.Tensor,
                          seq_lens: torch.Tensor, *, window: int, first_tokens: int = 0,
                          cum_seq_lens_q: Optional[torch.Tensor] = None, num_splits: int = 0,
                          device: int = 0) -> int:
    """Workspace bytes of ``window_attention`` for these shapes (no device memory is read)."""
    a = _window_args(q, rows, scales, block_tables, seq_lens, cum_seq_lens_q, None, window, first_tokens, num_splits)
    n = ctypes.c_size_t(0)
    _check(_b.lib().smla_window_workspace_size(ctypes.byref(a), device, ctypes.byref(n)))
    return int(n.value)


def window_attention(q: torch.Tensor, rows: torch.Tensor, scales: torch.Tensor, block_tables: torch.Tensor,
                     seq_lens: torch.Tensor, workspace_buffer: Optional[torch.Tensor], *, window: int,
                     first_tokens: int = 0, cum_seq_lens_q: Optional[torch.Tensor] = None,
                     sinks: Optional[torch.Tensor] = None, bmm1_scale=1.0, bmm2_scale=1.0,
                     out: Optional[torch.Tensor] = None, out_lse: Optional[torch.Tensor] = None,
                     num_splits: int = 0, error_word: Optional[torch.Tensor] = None,
                     stream: Optional[int] = None):
    """Attention of BF16 queries ``[T, H, 512]`` over the last ``window`` cached
    tokens of their request up to their own position, and its first
    ``first_tokens``; returns ``(out, out_lse)``, allocated when not given."""
    a = _window_args(q, rows, scales, block_tables, seq_lens, cum_seq_lens_q, sinks, window, first_tokens, num_splits)
    T, H = a.sum_q, a.num_heads
    if out is None:
        out = torch.empty((T, H, HEAD_DIM), dtype=torch.bfloat16, device=q.device)
    if out_lse is None:
        out_lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    if out.dtype != torch.bfloat16 or not out.is_contiguous() or out.numel() != T * H * HEAD_DIM:
        raise ValueError("out must be a contiguous bfloat16 tensor of T*H*512 elements")
    if out_lse.dtype != torch.float32 or not out_lse.is_contiguous() or out_lse.numel() != T * H:
        raise ValueError("out_lse must be a contiguous float32 tensor of T*H elements")
    _words("error_word", error_word, 1)
    for name, val in (("bmm1", bmm1_scale), ("bmm2", bmm2_scale)):
        if isinstance(val, torch.Tensor):
            _words(f"{name}_scale", val, 1, torch.float32)
            setattr(a, f"{name}_scale_dev", val.data_ptr())
            setattr(a, f"{name}_scale", 1.0)
        else:
            setattr(a, f"{name}_scale", float(val))
    a.out, a.out_lse, a.error_word = out.data_ptr(), out_lse.data_ptr(), _ptr(error_word)
    if workspace_buffer is not None:
        if not workspace_buffer.is_contiguous():
            raise ValueError("workspace must be contiguous")
        a.workspace = workspace_buffer.data_ptr()
        a.workspace_bytes = workspace_buffer.numel() * workspace_buffer.element_size()
    _placed(q.device, q=q, rows=rows, scales=scales, block_tables=block_tables, seq_lens=seq_lens,
            workspace=workspace_buffer, cum_seq_lens_q=cum_seq_lens_q, sinks=sinks, bmm1_scale=bmm1_scale,
            bmm2_scale=bmm2_scale, out=out, out_lse=out_lse, error_word=error_word)
    with torch.cuda.device(q.device):
        _check(_b.lib().smla_window_attention(ctypes.byref(a), _stream(stream)))
    return out, out_lse


def append(latent: torch.Tensor, rows: torch.Tensor, scales: torch.Tensor, block_tables: torch.Tensor,
           seq_lens: torch.Tensor, *, cum_seq_lens_q: Optional[torch.Tensor] = None,
           error_word: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> None:
    """Quantises the new latent rows ``[T, 512]`` (BF16) into the cache, at the
    last positions of their requests (``seq_lens`` counts them)."""
    if latent.dtype != torch.bfloat16:
        raise TypeError(f"latent must be bfloat16; got {latent.dtype}")
    if latent.dim() != 2 or latent.shape[1] != HEAD_DIM or latent.stride(1) != 1:
        raise ValueError(f"latent must be [T, {HEAD_DIM}] with contiguous rows; got {tuple(latent.shape)}")
    a = SmlaAppendArgs()
    a.cache = _cache(rows, scales, block_tables, seq_lens, cum_seq_lens_q)
    a.sum_q, a.latent = latent.shape[0], latent.data_ptr()
    a.latent_stride = latent.stride(0) if latent.shape[0] > 1 else HEAD_DIM
    _words("error_word", error_word, 1)
    a.error_word = _ptr(error_word)
    _placed(latent.device, latent=latent, rows=rows, scales=scales, block_tables=block_tables, seq_lens=seq_lens,
            cum_seq_lens_q=cum_seq_lens_q, error_word=error_word)
    with torch.cuda.device(latent.device):
        _check(_b.lib().smla_cache_append(ctypes.byref(a), _stream(stream)))


def _pages_args(tables, ref_counts, lens, page_size, error_word) -> SmlaPagesArgs:
    _table("block_tables", tables)
    _words("ref_counts", ref_counts, 1)
    _words("lens", lens, tables.shape[0])
    _words("error_word", error_word, 1)
    a = SmlaPagesArgs()
    a.block_tables, a.block_table_stride = tables.data_ptr(), _row_stride(tables)
    a.rows, a.max_pages, a.page_size = tables.shape[0], tables.shape[1], int(page_size)
    a.ref_counts, a.num_pages = ref_counts.data_ptr(), ref_counts.numel()
    a.lens, a.error_word = lens.data_ptr(), _ptr(error_word)
    return a


def _with_moves(a: SmlaPagesArgs, moves, workspace: torch.Tensor) -> None:
    src, dst, count = moves
    _words("moves.src", src, 0)
    _words("moves.dst", dst, src.numel())
    _words("moves.count", count, 1)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    a.move_src, a.move_dst, a.move_count, a.move_capacity = src.data_ptr(), dst.data_ptr(), count.data_ptr(), src.numel()
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()


def pages_workspace_size(block_tables: torch.Tensor, ref_counts: torch.Tensor, page_size: int) -> int:
    """Workspace bytes of ``pages_resize`` and ``pages_compact`` (no device memory is read)."""
    a = SmlaPagesArgs()
    a.rows, a.max_pages, a.page_size = block_tables.shape[0], block_tables.shape[1], int(page_size)
    a.num_pages = ref_counts.numel()
    n = ctypes.c_size_t(0)
    _check(_b.lib().smla_pages_workspace_size(ctypes.byref(a), ctypes.byref(n)))
    return int(n.value)


def pages_resize(block_tables: torch.Tensor, ref_counts: torch.Tensor, lens: torch.Tensor, new_lens: torch.Tensor,
                 workspace_buffer: torch.Tensor, *, page_size: int, moves,
                 error_word: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> None:
    """Takes each request from ``lens`` to ``new_lens`` tokens: pages dropped,
    then the lowest free pages handed out; ``moves`` receives the shared pages
    that a growing request got a copy of (``pages_copy`` them)."""
    a = _pages_args(block_tables, ref_counts, lens, page_size, error_word)
    _words("new_lens", new_lens, a.rows)
    a.new_lens = new_lens.data_ptr()
    _with_moves(a, moves, workspace_buffer)
    _placed(block_tables.device, block_tables=block_tables, ref_counts=ref_counts, lens=lens, new_lens=new_lens,
            workspace=workspace_buffer, move_src=moves[0], move_dst=moves[1], move_count=moves[2],
            error_word=error_word)
    with torch.cuda.device(block_tables.device):
        _check(_b.lib().smla_pages_resize(ctypes.byref(a), _stream(stream)))


def pages_fork(block_tables: torch.Tensor, ref_counts: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor,
               out_lens: torch.Tensor, *, page_size: int, error_word: Optional[torch.Tensor] = None,
               stream: Optional[int] = None) -> None:
    """Requests with ``parents[b] >= 0`` (which hold nothing) share their
    parent's pages; ``out_lens`` receives every request's length after it."""
    a = _pages_args(block_tables, ref_counts, lens, page_size, error_word)
    _words("parents", parents, a.rows)
    _words("out_lens", out_lens, a.rows)
    a.parents, a.out_lens = parents.data_ptr(), out_lens.data_ptr()
    _placed(block_tables.device, block_tables=block_tables, ref_counts=ref_counts, lens=lens, parents=parents,
            out_lens=out_lens, error_word=error_word)
    with torch.cuda.device(block_tables.device):
        _check(_b.lib().smla_pages_fork(ctypes.byref(a), _stream(stream)))


def pages_compact(block_tables: torch.Tensor, ref_counts: torch.Tensor, lens: torch.Tensor,
                  workspace_buffer: torch.Tensor, *, page_size: int, moves,
                  error_word: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> None:
    """Renumbers the pages in use to the front of the pool; ``moves`` receives
    the pages to copy (``pages_copy``) before the cache is used again."""
    a = _pages_args(block_tables, ref_counts, lens, page_size, error_word)
    _with_moves(a, moves, workspace_buffer)
    _placed(block_tables.device, block_tables=block_tables, ref_counts=ref_counts, lens=lens,
            workspace=workspace_buffer, move_src=moves[0], move_dst=moves[1], move_count=moves[2],
            error_word=error_word)
    with torch.cuda.device(block_tables.device):
        _check(_b.lib().smla_pages_compact(ctypes.byref(a), _stream(stream)))


def pages_copy(pools: Sequence[torch.Tensor], moves, *, error_word: Optional[torch.Tensor] = None,
               stream: Optional[int] = None) -> None:
    """Copies the pages of ``moves`` within every pool: tensors ``[num_pages,
    ...]`` of any type whose pages are contiguous (rows and scales of all
    layers in one call)."""
    src, dst, count = moves
    _words("moves.src", src, 0)
    _words("moves.dst", dst, src.numel())
    _words("moves.count", count, 1)
    _words("error_word", error_word, 1)
    array = (SmlaPool * max(1, len(pools)))()
    for i, t in enumerate(pools):
        if t.dim() < 1 or t.shape[0] != pools[0].shape[0]:
            raise ValueError(f"pool {i} must be [num_pages, ...] with the first pool's {pools[0].shape[0]} pages")
        if t.shape[0] < 1 or t.numel() == 0 or not t[0].is_contiguous():
            raise ValueError(f"pool {i}: pages must be contiguous and not empty")
        page = t[0].numel() * t.element_size()
        array[i].base, array[i].page_bytes = t.data_ptr(), page
        array[i].page_stride = t.stride(0) * t.element_size() if t.shape[0] > 1 else page
        _placed(src.device, **{f"pool {i}": t})
    if not pools:
        return
    _placed(src.device, move_src=src, move_dst=dst, move_count=count, error_word=error_word)
    with torch.cuda.device(src.device):
        _check(_b.lib().smla_pages_copy(ctypes.byref(array), len(pools), pools[0].shape[0], src.data_ptr(),
                                        dst.data_ptr(), count.data_ptr(), src.numel(), _ptr(error_word),
                                        _stream(stream)))
