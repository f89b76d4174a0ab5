"""Beam search's choice (argument marshalling only): the best continuations over a
request's beams and the vocabulary.  The call is ``smla_beam_select`` of
``include/smla.h``, which defines it; plain tensors go through the extension
module.  A step of a search on the paged latent cache:

    ws = torch.empty(beam_workspace_size(logits, scores), dtype=torch.uint8, device="cuda")
    best = beam_select(logits, scores, ws)                      # logits [B * beams, V], scores [B, beams]
    cache.pages_reorder(tables, counts, lens, best.parents, out_lens, ws2, page_size=64)
    cache.pages_shared_prefix(tables, out_lens, group_starts, prefix_lens, page_size=64)
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import binding as _b
from . import cache as _cache
from .binding import _c_void_p, _ptr
from .cache import _call, _int32, _on, _words

_i32, _i64, _size = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
LOGITS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class SmlaBeamArgs(ctypes.Structure):
    _fields_ = [
        ("batch", _i32), ("beams", _i32), ("vocab", _i32), ("num_out", _i32), ("dtype", _i32),
        ("logits", _c_void_p), ("logits_stride", _i64), ("scores", _c_void_p), ("finished", _c_void_p), ("end_token", _i32),
        ("out_scores", _c_void_p), ("out_parents", _c_void_p), ("out_tokens", _c_void_p),
        ("workspace", _c_void_p), ("workspace_bytes", _size), ("error_word", _c_void_p),
    ]


class BeamChoice(NamedTuple):
    """The best continuations of each request, in order: scores (float32), rows of
    the logits they continue and tokens (int32), each ``[B, num_out]``."""
    scores: torch.Tensor
    parents: torch.Tensor
    tokens: torch.Tensor


def _beam_args(logits: torch.Tensor, scores: torch.Tensor, num_out: Optional[int]) -> SmlaBeamArgs:
    if logits.dtype not in LOGITS:
        raise TypeError(f"logits must be bfloat16, float16 or float32; got {logits.dtype}")
    if scores.dtype != torch.float32:
        raise TypeError("scores must be float32")
    if scores.dim() != 2 or not scores.is_contiguous():
        raise ValueError(f"scores must be [requests, beams], contiguous; got {tuple(scores.shape)}")
    if logits.dim() != 2 or logits.shape[0] != scores.numel() or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError(f"logits must be [{scores.numel()}, vocab] with contiguous rows; got {tuple(logits.shape)}")
    rows, vocab = logits.shape
    if rows > 1 and logits.stride(0) < vocab:
        raise ValueError("logits: rows overlap")
    batch, beams = scores.shape
    return SmlaBeamArgs(batch, beams, vocab, _int32("num_out", beams if num_out is None else num_out), LOGITS[logits.dtype],
                        logits.data_ptr(), logits.stride(0) if rows > 1 else vocab, scores.data_ptr())


def beam_workspace_size(logits: torch.Tensor, scores: torch.Tensor, *, num_out: Optional[int] = None,
                        device: Optional[int] = None) -> int:
    """Workspace bytes of ``beam_select`` for these shapes (no device memory is
    read) and for fewer requests or beams or a smaller vocabulary, on ``device``, by
    default the logits'."""
    a = _beam_args(logits, scores, num_out)
    n = ctypes.c_size_t(0)
    if device is None:
        device = max(logits.get_device(), 0)
    _b._check(_b.lib().smla_beam_workspace_size(ctypes.byref(a), device, ctypes.byref(n)))
    return int(n.value)


def beam_select(logits: torch.Tensor, scores: torch.Tensor, workspace_buffer: torch.Tensor, *, num_out: Optional[int] = None,
                finished: Optional[torch.Tensor] = None, end_token: int = 0, out: Optional[BeamChoice] = None,
                error_word: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> BeamChoice:
    """The ``num_out`` (by default as many as there are beams) best continuations
    of each request: ``scores[r, i] + log_softmax(logits[r * beams + i])[v]``, a
    ``finished`` beam (bool ``[B, beams]``) with its own score and ``end_token``."""
    done = (_cache._extension or _cache.extension()).beam_select(logits, scores, workspace_buffer, num_out, finished, end_token,
                                                                 out, error_word, stream)
    if done.__class__ is tuple:
        return BeamChoice._make(done)
    if done is not None:
        _b._check(done)
    a = _beam_args(logits, scores, num_out)
    index = logits.get_device()
    if finished is not None:
        if finished.dtype not in (torch.bool, torch.uint8):
            raise TypeError("finished must be bool")
        if not finished.is_contiguous() or finished.numel() != scores.numel():
            raise ValueError(f"finished must be {tuple(scores.shape)}, contiguous")
        a.finished = finished.data_ptr()
    a.end_token = _int32("end_token", end_token)
    shape = (a.batch, max(a.num_out, 0))
    if out is None:
        with _b._allocate_for(stream, index):
            out = BeamChoice(torch.empty(shape, dtype=torch.float32, device=logits.device),
                             torch.empty(shape, dtype=torch.int32, device=logits.device),
                             torch.empty(shape, dtype=torch.int32, device=logits.device))
    need = shape[0] * shape[1]
    _words("out.scores", out.scores, need, torch.float32)
    _words("out.parents", out.parents, need)
    _words("out.tokens", out.tokens, need)
    _words("error_word", error_word, 1)
    a.out_scores, a.out_parents, a.out_tokens = (t.data_ptr() for t in out)
    if workspace_buffer is not None:
        if not workspace_buffer.is_contiguous():
            raise ValueError("workspace must be contiguous")
        a.workspace, a.workspace_bytes = workspace_buffer.data_ptr(), workspace_buffer.nbytes
    a.error_word = _ptr(error_word)
    _on(index, (logits, scores, workspace_buffer, finished, *out, error_word),
        ("logits", "scores", "workspace", "finished", "out.scores", "out.parents", "out.tokens", "error_word"))
    _call(_b.lib().smla_beam_select, index, stream, ctypes.byref(a))
    return out
