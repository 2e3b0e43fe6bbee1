"""Beam search over a vocabulary of items or of the codes that spell them: the step that
selects each user's best continuations. The beams' event histories follow with
``history_reorder``, and attention reads what they share once
(``history_prefix_attention``).

Argument checks and marshalling only, like the rest of the binding: include/dlrm.h
defines the call. With ``stream`` the launches go there, and the tensors that the call
makes belong to that stream.

    scores, rows, tokens = beam_select(logits, scores, starts, width)   # (groups, width) each
    history_reorder(cache, slots, rows.view(-1))     # a slot each, as many as before
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import operator
import struct

import torch

from . import DlrmError, ERR_INVALID_ARG, ERR_UNSUPPORTED, _check, lib
from .history import INT32_MAX, _dtype_code, _int32_vector, _on, _raw_stream

MAX_WIDTH = 256
_RESULTS = (torch.float32, torch.int32, torch.int32)
_NOWHERE = contextlib.nullcontext()

_VP, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class _BeamSelect(ctypes.Structure):
    _fields_ = ([(n, _VP) for n in ("logits", "scores", "allowed", "starts", "out_scores", "out_rows",
                                    "out_tokens", "err", "work")]
                + [(n, _I64) for n in ("work_bytes", "rows", "vocab", "ld", "ld_allowed")]
                + [(n, _I32) for n in ("groups", "width", "dtype")])


# The same fields, packed in one call.
_SELECT = struct.Struct("@9P5q3i0P")
assert _SELECT.size == ctypes.sizeof(_BeamSelect)


def _bind(lib_):
    for name, res in (("beam_select_work_bytes", _I64), ("beam_select", ctypes.c_int)):
        fn = getattr(lib_, name)
        fn.argtypes, fn.restype = [_VP] if res is _I64 else [_VP, _VP], res


_bound_lib = None


def _bound():
    global _bound_lib
    if _bound_lib is None:
        loaded = lib()
        _bind(loaded)
        _bound_lib = loaded
    return _bound_lib


@functools.lru_cache(maxsize=256)
def _work_bytes(sizes) -> int:
    """Of a call of these sizes; they alone decide, so they are remembered."""
    return _bound().beam_select_work_bytes(_SELECT.pack(*(0,) * 10, *sizes))


def beam_select(logits, scores, starts, width: int, *, allowed=None, err_flag=None, stream=None):
    """The ``width`` best continuations of each group of beams: (scores, rows, tokens),
    (groups, width) in float32, int32 and int32, best first.

    ``logits``: (rows, vocab) in float32, bfloat16 or float16, unit stride along the
    vocabulary; ``scores``: (rows,) float32, the beams' own, or None for zeros;
    ``starts``: (groups + 1,) int32: rows [starts[g], starts[g+1]) are group g's. A
    candidate's score is its row's plus the token's log-probability among the allowed
    ones; equal scores go by row, then token. ``allowed``: (rows, vocab) bool, or
    (vocab,) or (1, vocab) for all rows; None: every token. Places past the candidates
    hold -infinity, -1, -1. ``err_flag``: (1,) int32, receives the error bits of bad
    starts and of rows with a NaN or +infinity. ``width`` is at most 256."""
    where = "beam_select"
    if not isinstance(logits, torch.Tensor):
        raise TypeError(f"{where}: logits must be a torch.Tensor")
    if not logits.is_cuda:
        raise ValueError(f"{where}: logits must be a CUDA tensor")
    index = logits.get_device()
    shape = logits.shape
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError(f"{where}: logits: expected (rows, vocab), got {tuple(shape)}")
    rows, vocab = shape
    ld, unit = logits.stride()
    if unit != 1 and vocab > 1 and rows:
        raise ValueError(f"{where}: logits: its last dimension must be contiguous")
    dtype = _dtype_code(logits, "beam_select: logits")
    groups = _int32_vector(starts, "beam_select: starts", None, index) - 1
    if groups < 0:
        raise ValueError(f"{where}: starts: expected at least one entry")
    if scores is not None:
        if not isinstance(scores, torch.Tensor) or scores.dtype is not torch.float32:
            raise TypeError(f"{where}: scores: expected a float32 tensor")
        if scores.shape != shape[:1] or scores.get_device() != index or not scores.is_contiguous():
            raise ValueError(f"{where}: scores: expected contiguous ({rows},) on {logits.device}")
    ld_allowed = 0
    if allowed is not None:
        if not isinstance(allowed, torch.Tensor) or allowed.dtype is not torch.bool:
            raise TypeError(f"{where}: allowed: expected a bool tensor")
        if allowed.shape not in (shape, shape[1:], (1, vocab)) or allowed.get_device() != index:
            raise ValueError(f"{where}: allowed: expected ({rows}, {vocab}) or ({vocab},) on {logits.device}, "
                             f"got {tuple(allowed.shape)} on {allowed.device}")
        strides = allowed.stride()
        if strides[-1] != 1 and vocab > 1 and allowed.numel():
            raise ValueError(f"{where}: allowed: its last dimension must be contiguous")
        if allowed.shape == shape and rows > 1:
            ld_allowed = strides[0]
    if err_flag is not None:
        _int32_vector(err_flag, "beam_select: err_flag", 1, index)
    width = operator.index(width)
    if not 1 <= width <= MAX_WIDTH:
        raise DlrmError(ERR_INVALID_ARG if width < 1 else ERR_UNSUPPORTED, f"{where}: width {width}")
    if max(rows, groups) > INT32_MAX:
        raise DlrmError(ERR_UNSUPPORTED, where)
    queue = _raw_stream(stream, index)
    sizes = (rows, vocab, ld, ld_allowed, groups, width, dtype)
    need = _work_bytes(sizes)
    if need < 0:
        raise DlrmError(ERR_UNSUPPORTED, where)
    with _NOWHERE if stream is None else _on(stream, logits.device):
        best, parents, tokens = (torch.empty((groups, width), dtype=t, device=logits.device) for t in _RESULTS)
        work = torch.empty(need, dtype=torch.uint8, device=logits.device) if need else None
    args = _SELECT.pack(logits.data_ptr(), 0 if scores is None else scores.data_ptr(),
                        0 if allowed is None else allowed.data_ptr(), starts.data_ptr(), best.data_ptr(),
                        parents.data_ptr(), tokens.data_ptr(), 0 if err_flag is None else err_flag.data_ptr(),
                        0 if work is None else work.data_ptr(), need, *sizes)
    _check(_bound().beam_select(args, queue), where)
    return best, parents, tokens
