"""The paged latent cache: tensor-level calls (argument marshalling only).

A call whose tensors are plain goes through the extension module of
``csrc/cache_torch.cpp``; the functions below take the others: they name what is
wrong, or handle what is legal but unusual.

A cache is what the caller owns: E4M3 rows ``[num_pages, page_size, 512]``,
float32 scales ``[num_pages, page_size // block_rows]`` (one per block of
tokens), int32 page tables ``[requests, max_pages]``, lengths ``[requests]``
and, for the page calls, a count per page (0 = free).  The calls are the
``smla_window_*``, ``smla_cache_*`` and ``smla_pages_*`` entry points of
``include/smla.h``, which defines them (``smla_prefix_*`` among them); all work on the device, on the current
stream unless ``stream`` is given, and none waits.

    pages_resize(tables, refs, lens, new_lens, ws, page_size=64, moves=moves)   # pages for the new tokens
    pages_copy([rows, scales], moves)                                           # shared pages about to be written
    append(latent, rows, scales, tables, new_lens, cum_seq_lens_q=cum)          # quantise them in
    out, lse = window_attention(q, rows, scales, tables, new_lens, ws2, window=1024, first_tokens=4,
                                cum_seq_lens_q=cum, bmm1_scale=scale)
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
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


class SmlaPrefixArgs(ctypes.Structure):
    _fields_ = [
        ("cache", SmlaCache),
        ("sum_q", _i32), ("num_heads", _i32), ("num_groups", _i32),
        ("group_starts", _c_void_p), ("prefix_lens", _c_void_p),
        ("q", _c_void_p), ("q_stride_token", _i64), ("sinks", _c_void_p),
        ("bmm1_scale", ctypes.c_float), ("bmm2_scale", ctypes.c_float),
        ("bmm1_scale_dev", _c_void_p), ("bmm2_scale_dev", _c_void_p),
        ("out", _c_void_p), ("out_lse", _c_void_p),
        ("workspace", _c_void_p), ("workspace_bytes", _size), ("error_word", _c_void_p),
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


_extension = None
EXTENSION_PATH = os.path.join(os.path.dirname(_b.LIB_PATH), "smla_torch.so")


def extension():
    """The extension module (raises if it has not been built)."""
    global _extension
    if _extension is None:
        if not os.path.exists(EXTENSION_PATH):
            raise ImportError(f"smla_torch.so is not built ({EXTENSION_PATH}); run "
                              "sparse_mla_decode_token_gb300.build.build() first")
        _b.lib()
        spec = importlib.util.spec_from_file_location("smla_torch", EXTENSION_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _extension = module
    return _extension


def _int32(name: str, value) -> int:
    value = int(value)
    if not -(1 << 31) <= value < 1 << 31:
        raise ValueError(f"{name} {value} is not a 32-bit integer")
    return value


def _words(name: str, t: Optional[torch.Tensor], need: int, dtype=torch.int32) -> None:
    """An array that the kernels index: its type, contiguous, long enough."""
    if t is None or (t.dtype is dtype and t.is_contiguous() and t.numel() >= need):
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} has {t.numel()} entries; the call reads {need}")


def _on(index: int, tensors, names) -> None:
    """Every tensor (of those given) is on CUDA device ``index``."""
    for t in tensors:
        if t is not None and t.get_device() != index or index < 0:
            break
    else:
        return
    for name, t in zip(names, tensors):
        if t is not None and (t.device.type != "cuda" or t.get_device() != index):
            raise ValueError(f"{name} is on {t.device}; every tensor must be on one CUDA device"
                             + (f" (cuda:{index})" if index >= 0 else ""))


def _call(function, index: int, stream: Optional[int], *args) -> None:
    """The entry point on the tensors' device and stream."""
    with torch.cuda.device(index):
        _check(function(*args, torch.cuda.current_stream().cuda_stream if stream is None else stream))


def _table(name: str, t: torch.Tensor) -> None:
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if t.dim() != 2 or t.shape[1] < 1 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [requests, max_pages] with a contiguous last dim")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: rows overlap")


def _check_cache(rows: torch.Tensor, scales: torch.Tensor, tables: torch.Tensor) -> None:
    """Raises what is wrong with a cache's layout."""
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
            (scales.shape[0] > 1 and scales.stride(0) < scales.shape[1]):
        raise ValueError("cache pages must not share memory")
    _table("block_tables", tables)
    if tables.shape[0] < 1:
        raise ValueError("block_tables has no rows")


def _cache(rows: torch.Tensor, scales: torch.Tensor, tables: torch.Tensor, seq_lens: torch.Tensor,
           cum: Optional[torch.Tensor]) -> SmlaCache:
    _check_cache(rows, scales, tables)
    rs, ss, ts = rows.shape, scales.shape, tables.shape
    rt, st, tt = rows.stride(), scales.stride(), tables.stride()
    num_pages, page_size = rs[0], rs[1]
    batch, max_pages = ts
    _words("seq_lens", seq_lens, batch)
    if cum is not None:
        _words("cum_seq_lens_q", cum, batch + 1)
    return SmlaCache(rows.data_ptr(), rt[1] if page_size > 1 else HEAD_DIM, rt[0] if num_pages > 1 else 0,
                     scales.data_ptr(), st[0] if num_pages > 1 else ss[1], num_pages, page_size, page_size // ss[1],
                     tables.data_ptr(), tt[0] if batch > 1 else max_pages, max_pages, batch,
                     seq_lens.data_ptr(), None if cum is None else cum.data_ptr())


def _attention_args(a, q, sinks) -> None:
    """The queries of an attention call: what it checks of them, and their fields of its struct."""
    qs, qt = q.shape, q.stride()
    if q.dtype is not torch.bfloat16:
        raise TypeError(f"q must be bfloat16; got {q.dtype}")
    if len(qs) != 3 or qs[2] != HEAD_DIM or (qs[0] > 0 and (qt[2] != 1 or (qs[1] > 1 and qt[1] != HEAD_DIM))):
        raise ValueError(f"q must be [T, H, {HEAD_DIM}] with contiguous heads; got {tuple(qs)}")
    if qs[0] > 1 and qt[0] <= 0:                       # (0 would stand for the packed stride)
        raise ValueError("the tokens of q must not share memory")
    if sinks is not None:
        _words("sinks", sinks, qs[1], torch.float32)
    a.sum_q, a.num_heads, a.bmm1_scale, a.bmm2_scale = qs[0], qs[1], 1.0, 1.0
    a.q, a.q_stride_token, a.sinks = q.data_ptr(), qt[0] if qs[0] > 1 else 0, None if sinks is None else sinks.data_ptr()


def _attention_call(a, function, names, q, tensors, workspace_buffer, bmm1_scale, bmm2_scale, out, out_lse, error_word, stream):
    """The outputs, scales and workspace of an attention call, and the call."""
    T, H = a.sum_q, a.num_heads
    with _b._allocate_for(stream, q.get_device()):
        new_out = torch.empty_like(q, memory_format=torch.contiguous_format) if out is None else None
        new_lse = torch.empty((T, H), dtype=torch.float32, device=q.device) if out_lse is None else None
    if out is None:
        out = new_out
    elif out.dtype != torch.bfloat16 or not out.is_contiguous() or out.numel() != T * H * HEAD_DIM:
        raise ValueError("out must be a contiguous bfloat16 tensor of T*H*512 elements")
    if out_lse is None:
        out_lse = new_lse
    elif out_lse.dtype != torch.float32 or not out_lse.is_contiguous() or out_lse.numel() != T * H:
        raise ValueError("out_lse must be a contiguous float32 tensor of T*H elements")
    _words("error_word", error_word, 1)
    scale1 = scale2 = None
    if isinstance(bmm1_scale, torch.Tensor):
        scale1 = bmm1_scale
        _words("bmm1_scale", scale1, 1, torch.float32)
        a.bmm1_scale_dev = scale1.data_ptr()
    else:
        a.bmm1_scale = float(bmm1_scale)
    if isinstance(bmm2_scale, torch.Tensor):
        scale2 = bmm2_scale
        _words("bmm2_scale", scale2, 1, torch.float32)
        a.bmm2_scale_dev = scale2.data_ptr()
    else:
        a.bmm2_scale = float(bmm2_scale)
    a.out, a.out_lse = out.data_ptr(), out_lse.data_ptr()
    if error_word is not None:
        a.error_word = error_word.data_ptr()
    if workspace_buffer is not None:
        if not workspace_buffer.is_contiguous():
            raise ValueError("workspace must be contiguous")
        a.workspace, a.workspace_bytes = workspace_buffer.data_ptr(), workspace_buffer.nbytes
    index = q.get_device()
    _on(index, (q, *tensors, workspace_buffer, scale1, scale2, out, out_lse, error_word),
        ("q", *names, "workspace", "bmm1_scale", "bmm2_scale", "out", "out_lse", "error_word"))
    _call(function, index, stream, ctypes.byref(a))
    return out, out_lse


def _window_args(q, rows, scales, tables, seq_lens, cum, sinks, window, first_tokens, num_splits) -> SmlaWindowArgs:
    a = SmlaWindowArgs()
    _attention_args(a, q, sinks)
    a.cache = _cache(rows, scales, tables, seq_lens, cum)
    a.window, a.first_tokens, a.num_splits = _int32("window", window), _int32("first_tokens", first_tokens), \
        _int32("num_splits", num_splits)
    return a


def window_workspace_size(q: torch.Tensor, rows: torch.Tensor, scales: torch.Tensor, block_tables: torch.Tensor,
                          seq_lens: torch.Tensor, *, window: int, first_tokens: int = 0,
                          cum_seq_lens_q: Optional[torch.Tensor] = None, num_splits: int = 0,
                          device: Optional[int] = None) -> int:
    """Workspace bytes of ``window_attention`` for these shapes (no device memory is
    read) and for fewer tokens, shorter windows or narrower tables, on ``device``, by
    default q's."""
    a = _window_args(q, rows, scales, block_tables, seq_lens, cum_seq_lens_q, None, window, first_tokens, num_splits)
    n = ctypes.c_size_t(0)
    if device is None:
        device = max(q.get_device(), 0)
    _check(_b.lib().smla_window_workspace_size(ctypes.byref(a), device, ctypes.byref(n)))
    return int(n.value)


_CACHE_TENSORS = ("rows", "scales", "block_tables", "seq_lens", "cum_seq_lens_q", "sinks")


def window_attention(q: torch.Tensor, rows: torch.Tensor, scales: torch.Tensor, block_tables: torch.Tensor,
                     seq_lens: torch.Tensor, workspace_buffer: Optional[torch.Tensor], *, window: int,
                     first_tokens: int = 0, cum_seq_lens_q: Optional[torch.Tensor] = None,
                     sinks: Optional[torch.Tensor] = None, bmm1_scale=1.0, bmm2_scale=1.0,
                     out: Optional[torch.Tensor] = None, out_lse: Optional[torch.Tensor] = None,
                     num_splits: int = 0, error_word: Optional[torch.Tensor] = None,
                     stream: Optional[int] = None):
    """Attention of BF16 queries ``[T, H, 512]`` over the last ``window`` cached
    tokens of their request up to their own position, and its first
    ``first_tokens``; returns ``(out, out_lse)``, allocated when not given (as
    ``stream``'s memory, where that is another than the current one)."""
    done = (_extension or extension()).window_attention(
        q, rows, scales, block_tables, seq_lens, workspace_buffer, cum_seq_lens_q, sinks, window, first_tokens, num_splits,
        bmm1_scale, bmm2_scale, out, out_lse, error_word, stream)
    if done.__class__ is tuple:
        return done
    if done is not None:
        _check(done)
    a = _window_args(q, rows, scales, block_tables, seq_lens, cum_seq_lens_q, sinks, window, first_tokens, num_splits)
    return _attention_call(a, _b.lib().smla_window_attention, _CACHE_TENSORS, q,
                           (rows, scales, block_tables, seq_lens, cum_seq_lens_q, sinks), workspace_buffer, bmm1_scale,
                           bmm2_scale, out, out_lse, error_word, stream)


def _prefix_args(q, rows, scales, tables, seq_lens, cum, sinks, group_starts, prefix_lens) -> SmlaPrefixArgs:
    a = SmlaPrefixArgs()
    _attention_args(a, q, sinks)
    a.cache = _cache(rows, scales, tables, seq_lens, cum)
    _words("group_starts", group_starts, 1)
    a.num_groups, a.group_starts = group_starts.numel() - 1, group_starts.data_ptr()
    if prefix_lens is not None:
        _words("prefix_lens", prefix_lens, a.num_groups)
        a.prefix_lens = prefix_lens.data_ptr()
    return a


def prefix_workspace_size(q: torch.Tensor, rows: torch.Tensor, scales: torch.Tensor, block_tables: torch.Tensor,
                          seq_lens: torch.Tensor, *, group_starts: torch.Tensor,
                          cum_seq_lens_q: Optional[torch.Tensor] = None, device: Optional[int] = None) -> int:
    """Workspace bytes of ``prefix_attention`` for these shapes (no device memory is
    read) and for fewer tokens, groups or table columns, on ``device``, by default q's."""
    a = _prefix_args(q, rows, scales, block_tables, seq_lens, cum_seq_lens_q, None, group_starts, None)
    n = ctypes.c_size_t(0)
    if device is None:
        device = max(q.get_device(), 0)
    _check(_b.lib().smla_prefix_workspace_size(ctypes.byref(a), device, ctypes.byref(n)))
    return int(n.value)


def prefix_attention(q: torch.Tensor, rows: torch.Tensor, scales: torch.Tensor, block_tables: torch.Tensor,
                     seq_lens: torch.Tensor, workspace_buffer: torch.Tensor, *, group_starts: torch.Tensor,
                     prefix_lens: torch.Tensor, cum_seq_lens_q: Optional[torch.Tensor] = None,
                     sinks: Optional[torch.Tensor] = None, bmm1_scale=1.0, bmm2_scale=1.0,
                     out: Optional[torch.Tensor] = None, out_lse: Optional[torch.Tensor] = None,
                     error_word: Optional[torch.Tensor] = None, stream: Optional[int] = None):
    """Causal attention of BF16 queries ``[T, H, 512]`` over the cached tokens of
    their request, of which the requests ``group_starts[g] <= b <
    group_starts[g + 1]`` share the first ``prefix_lens[g]`` (read through the
    table of the first one with new tokens, once for all); returns ``(out, out_lse)``, allocated when
    not given (as ``stream``'s memory, where that is another than the current one)."""
    done = (_extension or extension()).prefix_attention(
        q, rows, scales, block_tables, seq_lens, workspace_buffer, cum_seq_lens_q, sinks, group_starts, prefix_lens,
        bmm1_scale, bmm2_scale, out, out_lse, error_word, stream)
    if done.__class__ is tuple:
        return done
    if done is not None:
        _check(done)
    a = _prefix_args(q, rows, scales, block_tables, seq_lens, cum_seq_lens_q, sinks, group_starts, prefix_lens)
    return _attention_call(a, _b.lib().smla_prefix_attention, _CACHE_TENSORS + ("group_starts", "prefix_lens"), q,
                           (rows, scales, block_tables, seq_lens, cum_seq_lens_q, sinks, group_starts, prefix_lens),
                           workspace_buffer, bmm1_scale, bmm2_scale, out, out_lse, error_word, stream)


_APPEND_TENSORS = ("latent", "rows", "scales", "block_tables", "seq_lens", "cum_seq_lens_q", "error_word")


def append(latent: torch.Tensor, rows: torch.Tensor, scales: torch.Tensor, block_tables: torch.Tensor,
           seq_lens: torch.Tensor, *, cum_seq_lens_q: Optional[torch.Tensor] = None,
           error_word: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> None:
    """Quantises the new latent rows ``[T, 512]`` (BF16) into the cache, at the
    last positions of their requests (``seq_lens`` counts them)."""
    status = (_extension or extension()).append(latent, rows, scales, block_tables, seq_lens, cum_seq_lens_q, error_word,
                                                stream)
    if status is not None:
        return _check(status) if status else None
    ls, lt = latent.shape, latent.stride()
    if latent.dtype is not torch.bfloat16:
        raise TypeError(f"latent must be bfloat16; got {latent.dtype}")
    if len(ls) != 2 or ls[1] != HEAD_DIM or (lt[1] != 1 and ls[0] > 0):
        raise ValueError(f"latent must be [T, {HEAD_DIM}] with contiguous rows; got {tuple(ls)}")
    if ls[0] > 1 and lt[0] <= 0:                       # (0 would stand for the packed stride)
        raise ValueError("the tokens of latent must not share memory")
    _words("error_word", error_word, 1)
    a = SmlaAppendArgs(_cache(rows, scales, block_tables, seq_lens, cum_seq_lens_q), ls[0], latent.data_ptr(),
                       lt[0] if ls[0] > 1 else HEAD_DIM, None if error_word is None else error_word.data_ptr())
    index = latent.get_device()
    _on(index, (latent, rows, scales, block_tables, seq_lens, cum_seq_lens_q, error_word), _APPEND_TENSORS)
    _call(_b.lib().smla_cache_append, index, stream, ctypes.byref(a))


def _pages_args(tables, ref_counts, lens, page_size, error_word, new_lens=None, parents=None, out_lens=None,
                moves=(None, None, None), workspace=None) -> SmlaPagesArgs:
    _table("block_tables", tables)
    rows, max_pages = tables.shape
    _words("ref_counts", ref_counts, 1)
    _words("lens", lens, rows)
    _words("error_word", error_word, 1)
    _words("new_lens", new_lens, rows)
    _words("parents", parents, rows)
    _words("out_lens", out_lens, rows)
    src, dst, count = moves
    capacity = 0
    if src is not None:
        capacity = src.numel()
        _words("moves.src", src, 0)
        _words("moves.dst", dst, capacity)
        _words("moves.count", count, 1)
        if workspace is None or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor")
    return SmlaPagesArgs(tables.data_ptr(), tables.stride(0) if rows > 1 else max_pages, rows, max_pages,
                         _int32("page_size", page_size),
                         ref_counts.data_ptr(), ref_counts.numel(), lens.data_ptr(), _ptr(new_lens), _ptr(parents),
                         _ptr(out_lens), _ptr(src), _ptr(dst), _ptr(count), capacity, _ptr(workspace),
                         0 if workspace is None else workspace.nbytes, _ptr(error_word))


def pages_workspace_size(block_tables: torch.Tensor, ref_counts: torch.Tensor, page_size: int) -> int:
    """Workspace bytes of ``pages_resize`` and ``pages_compact`` (no device memory is read)."""
    a = SmlaPagesArgs()
    a.rows, a.max_pages, a.page_size = block_tables.shape[0], block_tables.shape[1], _int32("page_size", page_size)
    a.num_pages = ref_counts.numel()
    n = ctypes.c_size_t(0)
    _check(_b.lib().smla_pages_workspace_size(ctypes.byref(a), ctypes.byref(n)))
    return int(n.value)


_PAGES_TENSORS = ("block_tables", "ref_counts", "lens", "new_lens", "workspace", "move_src", "move_dst", "move_count",
                  "error_word")


def pages_resize(block_tables: torch.Tensor, ref_counts: torch.Tensor, lens: torch.Tensor, new_lens: torch.Tensor,
                 workspace_buffer: torch.Tensor, *, page_size: int, moves,
                 error_word: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> None:
    """Takes each request from ``lens`` to ``new_lens`` tokens: pages dropped,
    then the lowest free pages handed out; ``moves`` receives the shared pages
    that a growing request got a copy of (``pages_copy`` them).  Where pages run
    out (``DEVERR_OUT_OF_PAGES`` in ``error_word``) a request may be left with a
    page that it still shares, which ``append`` would write into: look at it first."""
    status = (_extension or extension()).pages_resize(block_tables, ref_counts, lens, new_lens, workspace_buffer, page_size,
                                                      moves, error_word, stream)
    if status is not None:
        return _check(status) if status else None
    a = _pages_args(block_tables, ref_counts, lens, page_size, error_word, new_lens=new_lens, moves=moves,
                    workspace=workspace_buffer)
    index = block_tables.get_device()
    _on(index, (block_tables, ref_counts, lens, new_lens, workspace_buffer, *moves, error_word), _PAGES_TENSORS)
    _call(_b.lib().smla_pages_resize, index, stream, ctypes.byref(a))


def pages_fork(block_tables: torch.Tensor, ref_counts: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor,
               out_lens: torch.Tensor, *, page_size: int, error_word: Optional[torch.Tensor] = None,
               stream: Optional[int] = None) -> None:
    """Requests with ``parents[b] >= 0`` (which hold nothing) share their
    parent's pages; ``out_lens`` receives every request's length after it."""
    status = (_extension or extension()).pages_fork(block_tables, ref_counts, lens, parents, out_lens, page_size, error_word,
                                                    stream)
    if status is not None:
        return _check(status) if status else None
    a = _pages_args(block_tables, ref_counts, lens, page_size, error_word, parents=parents, out_lens=out_lens)
    index = block_tables.get_device()
    _on(index, (block_tables, ref_counts, lens, parents, out_lens, error_word),
        ("block_tables", "ref_counts", "lens", "parents", "out_lens", "error_word"))
    _call(_b.lib().smla_pages_fork, index, stream, ctypes.byref(a))


def reorder_workspace_size(block_tables: torch.Tensor) -> int:
    """Workspace bytes of ``pages_reorder`` (no device memory is read)."""
    a = SmlaPagesArgs()
    a.rows, a.max_pages, a.page_size = block_tables.shape[0], block_tables.shape[1], 1
    n = ctypes.c_size_t(0)
    _check(_b.lib().smla_pages_reorder_workspace_size(ctypes.byref(a), ctypes.byref(n)))
    return int(n.value)


def pages_reorder(block_tables: torch.Tensor, ref_counts: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor,
                  out_lens: torch.Tensor, workspace_buffer: torch.Tensor, *, page_size: int,
                  error_word: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> None:
    """Every request at once becomes what ``parents[b]`` was (pages and length,
    to ``out_lens``); ``parents[b] < 0`` ends it.  Pages follow by their counts
    alone; behind it ``pages_resize`` gives those that grow pages of their own."""
    status = (_extension or extension()).pages_reorder(block_tables, ref_counts, lens, parents, out_lens, workspace_buffer,
                                                       page_size, error_word, stream)
    if status is not None:
        return _check(status) if status else None
    if not workspace_buffer.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor")
    a = _pages_args(block_tables, ref_counts, lens, page_size, error_word, parents=parents, out_lens=out_lens,
                    workspace=workspace_buffer)
    index = block_tables.get_device()
    _on(index, (block_tables, ref_counts, lens, parents, out_lens, workspace_buffer, error_word),
        ("block_tables", "ref_counts", "lens", "parents", "out_lens", "workspace", "error_word"))
    _call(_b.lib().smla_pages_reorder, index, stream, ctypes.byref(a))


def pages_shared_prefix(block_tables: torch.Tensor, lens: torch.Tensor, group_starts: torch.Tensor, prefix_lens: torch.Tensor,
                        *, page_size: int, error_word: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> None:
    """``prefix_lens[g]``: tokens of the leading whole pages that all requests of
    group ``g`` with tokens share, ``group_starts[g] <= b < group_starts[g + 1]``."""
    status = (_extension or extension()).pages_shared_prefix(block_tables, lens, group_starts, prefix_lens, page_size,
                                                             error_word, stream)
    if status is not None:
        return _check(status) if status else None
    _table("block_tables", block_tables)
    _words("lens", lens, block_tables.shape[0])
    _words("prefix_lens", prefix_lens, 0)
    _words("group_starts", group_starts, prefix_lens.numel() + 1)
    _words("error_word", error_word, 1)
    a = SmlaPagesArgs()
    a.rows, a.max_pages, a.page_size = block_tables.shape[0], block_tables.shape[1], _int32("page_size", page_size)
    a.block_tables, a.lens, a.error_word = block_tables.data_ptr(), lens.data_ptr(), _ptr(error_word)
    a.block_table_stride = block_tables.stride(0) if a.rows > 1 else a.max_pages
    index = block_tables.get_device()
    _on(index, (block_tables, lens, group_starts, prefix_lens, error_word),
        ("block_tables", "lens", "group_starts", "prefix_lens", "error_word"))
    _call(_b.lib().smla_pages_shared_prefix, index, stream, ctypes.byref(a), group_starts.data_ptr(), prefix_lens.numel(),
          prefix_lens.data_ptr())


def pages_compact(block_tables: torch.Tensor, ref_counts: torch.Tensor, lens: torch.Tensor,
                  workspace_buffer: torch.Tensor, *, page_size: int, moves,
                  error_word: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> None:
    """Renumbers the pages in use to the front of the pool; ``moves`` receives
    the pages to copy (``pages_copy``) before the cache is used again."""
    status = (_extension or extension()).pages_compact(block_tables, ref_counts, lens, workspace_buffer, page_size, moves,
                                                       error_word, stream)
    if status is not None:
        return _check(status) if status else None
    a = _pages_args(block_tables, ref_counts, lens, page_size, error_word, moves=moves, workspace=workspace_buffer)
    index = block_tables.get_device()
    _on(index, (block_tables, ref_counts, lens, None, workspace_buffer, *moves, error_word), _PAGES_TENSORS)
    _call(_b.lib().smla_pages_compact, index, stream, ctypes.byref(a))


def pages_copy(pools: Sequence[torch.Tensor], moves, *, error_word: Optional[torch.Tensor] = None,
               stream: Optional[int] = None) -> None:
    """Copies the pages of ``moves`` within every pool: tensors ``[num_pages,
    ...]`` of any type whose pages are contiguous (rows and scales of all
    layers in one call)."""
    status = (_extension or extension()).pages_copy(pools, moves, error_word, stream)
    if status is not None:
        return _check(status) if status else None
    src, dst, count = moves
    capacity = src.numel()
    _words("moves.src", src, 0)
    _words("moves.dst", dst, capacity)
    _words("moves.count", count, 1)
    _words("error_word", error_word, 1)
    if not pools:
        return
    index = src.get_device()
    num_pages = pools[0].shape[0] if pools[0].dim() else 0
    described = []
    for i, t in enumerate(pools):
        if t.dim() < 1 or t.shape[0] != num_pages:
            raise ValueError(f"pool {i} must be [num_pages, ...] with the first pool's {num_pages} pages")
        if num_pages < 1 or t.numel() == 0 or not (t.is_contiguous() or t[0].is_contiguous()):
            raise ValueError(f"pool {i}: pages must be contiguous and not empty")
        page = t.nbytes // num_pages
        described.append((t.data_ptr(), page, t.stride(0) * t.element_size() if num_pages > 1 else page))
        if t.get_device() != index:
            _on(index, (t,), (f"pool {i}",))
    _on(index, (src, dst, count, error_word), ("move_src", "move_dst", "move_count", "error_word"))
    array = (SmlaPool * len(described))(*described)
    _call(_b.lib().smla_pages_copy, index, stream, ctypes.byref(array), len(described), num_pages, src.data_ptr(),
          dst.data_ptr(), count.data_ptr(), capacity, _ptr(error_word))
