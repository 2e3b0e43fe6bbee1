"""Event histories: an 8-bit paged cache of keys and values, attention over
it, and windowed attention over plain rows.

Argument checks and marshalling only, like the rest of the binding:
include/dlrm.h defines the pool, the codes and every operator, and says which
faults only the device sees (they set bits in the cache's error word, read by
``HistoryCache.error()``). Nothing here waits for the GPU but ``error()``. With ``stream``
the launches go there, and tensors that a call makes belong to that stream, as under
``torch.cuda.stream``; its order against the inputs' and outputs' other streams is the
caller's.

    cache = HistoryCache(n_pages, n_slots, max_pages, n_heads, head_dim)
    history_append(cache, slots, starts, k, v)            # (rows, n_heads, head_dim)
    out = history_attention(cache, slots, starts, q)      # (rows, query heads, head_dim)
"""
from __future__ import annotations

import contextlib
import ctypes
import operator
import struct
from typing import Optional

import torch

from . import (DlrmError, ERR_INDEX_OOB, ERR_INVALID_ARG, ERR_OOM, ERR_TIMEOUT, ERR_UNSUPPORTED,
               OK, _check, _stream, lib)

DTYPE_FP32, DTYPE_BF16, DTYPE_FP16 = 0, 1, 2
PAGE_TOKENS = (32, 64, 128)
HEAD_DIMS = (32, 64, 128)
INT32_MAX = 2 ** 31 - 1
FP32_MAX = 2.0 ** 128 - 2.0 ** 104

_VP, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class _History(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("n_pages", "page_tokens", "n_heads", "head_dim", "n_slots",
                                     "max_pages")]
                + [(n, _VP) for n in ("k_codes", "v_codes", "k_scales", "v_scales", "table",
                                      "lengths", "refs", "free_pages", "n_free", "err", "work")]
                + [("work_bytes", _I64)])


class _Attention(ctypes.Structure):
    _fields_ = ([(n, _VP) for n in ("q", "k", "v", "out", "lse", "slots", "q_starts", "k_starts")]
                + [(n, _I64) for n in ("q_rows", "k_rows", "ld_q", "ld_q_head", "ld_k", "ld_k_head",
                                       "ld_v", "ld_v_head", "ld_out", "ld_out_head")]
                + [(n, _I32) for n in ("batch", "n_heads", "n_kv_heads", "head_dim", "dtype",
                                       "causal", "window", "sinks")]
                + [("scale", ctypes.c_float), ("err", _VP)])


# The same fields as _Attention, packed in one call: a ctypes structure takes
# as long to fill, attribute by attribute, as the launch takes.
_ATTENTION = struct.Struct("@8P10q8if0PP")
assert _ATTENTION.size == ctypes.sizeof(_Attention)


def _bind(lib_):
    # attention arguments: a _Attention by reference, or its packed bytes
    st, h, a = ctypes.c_int, ctypes.POINTER(_History), _VP
    sig = {
        "history_work_bytes": ([h], _I64),
        "history_reset": ([h, _VP], st),
        "history_append": ([h, _VP, _VP, _I32, _VP, _I64, _I64, _VP, _I64, _I64, _I64, _I32, _VP],
                           st),
        "history_fork": ([h, _VP, _VP, _I32, _VP], st),
        "history_copy": ([h, _VP, _VP, _I32, _VP], st),
        "history_free": ([h, _VP, _I32, _VP], st),
        "history_trim": ([h, _VP, _I32, _I32, _I32, _VP], st),
        "history_compact": ([h, _VP], st),
        "history_attention": ([h, a, _VP], st),
        "window_attention": ([a, _VP], st),
        "attention_test_stall": ([_I64, _I32], st),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib_, name)
        fn.argtypes, fn.restype = args, res


_DTYPES = {torch.float32: DTYPE_FP32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_FP16}


def _dtype_code(t, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected float32, bfloat16 or float16, got {t.dtype}")
    return code


# (absent from a build of torch without CUDA, where nothing gets as far as to ask)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _raw_stream(stream, index: int):
    """The cudaStream_t of ``stream``, or of device ``index``'s current stream (read
    without making a Stream object, which takes microseconds). A launch goes to the
    current device, so that has to be the tensors'."""
    if index != _current_device():
        raise ValueError(f"the tensors are not on the current device ({_current_device()}): make "
                         f"device {index} current (torch.cuda.device)")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return _stream(stream)


def _on(stream, device):
    """A context in which tensors are made on ``stream``: from memory that no work queued on
    another stream still uses, filled in its order."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        # (1, the legacy default stream's handle, is no address, and torch takes none such)
        stream = (torch.cuda.default_stream(device) if int(stream) == 1
                  else torch.cuda.ExternalStream(int(stream), device=device))
    return torch.cuda.stream(stream)


# The checks below run with every call: a tensor that passes costs a few attributes
# (all of a call's about as much as the launch), and messages are made for errors
# only. ``device`` is an index (quick) or a torch.device.

def _elsewhere(t, device) -> bool:
    return t.device != device if isinstance(device, torch.device) else t.get_device() != device


def _int32_vector(t, name: str, n: Optional[int], device) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32:
        raise TypeError(f"{name}: expected an int32 tensor")
    shape = t.shape
    if len(shape) != 1 or (n is not None and shape[0] != n):
        raise ValueError(f"{name}: expected ({'n' if n is None else n},), got {tuple(shape)}")
    if t.get_device() != device and _elsewhere(t, device):
        raise ValueError(f"{name}: on {t.device}, not where the call's other tensors are")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return shape[0]


def _rows(t, name: str, heads: Optional[int], dim: Optional[int], device):
    """Shape and strides of a (rows, heads, dim) tensor with unit stride along dim."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or (
            dim is not None and shape[2] != dim):
        raise ValueError(f"{name}: expected (rows, {heads or 'heads'}, {dim or 'dim'}), "
                         f"got {tuple(shape)}")
    if t.get_device() != device and _elsewhere(t, device):
        raise ValueError(f"{name}: on {t.device}, not where the call's other tensors are")
    strides = t.stride()
    if strides[2] != 1 and shape[2] > 1 and t.numel():
        raise ValueError(f"{name}: its last dimension must be contiguous")
    return shape, strides


class HistoryCache:
    """A pool of pages for event histories and the tables of its slots.

    ``n_pages`` pages of ``page_tokens`` events of ``n_heads`` heads; ``n_slots``
    histories of at most ``max_pages`` pages each. The tensors (``k_codes``,
    ``v_codes``, ``k_scales``, ``v_scales``, ``table``, ``lengths``, ``refs``,
    ``free_pages``, ``n_free``, ``err``) are the caller's to read, e.g. to save
    a pool; calls on one cache go to one stream, the one that made it or one that has
    waited for it. Its device has to be the current one, here and in every call.
    """

    def __init__(self, n_pages: int, n_slots: int, max_pages: int, n_heads: int, head_dim: int,
                 page_tokens: int = 64, device="cuda", stream=None):
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError("HistoryCache: device must be a CUDA device")
        if device.index is not None and device.index != torch.cuda.current_device():
            raise ValueError(f"HistoryCache: {device} is not the current device: make it so (torch.cuda.device)")
        # (ctypes cuts integers off)
        if max(n_pages, page_tokens, n_heads, head_dim, n_slots, max_pages) > INT32_MAX:
            raise DlrmError(ERR_UNSUPPORTED, "HistoryCache")
        c = _History(int(n_pages), int(page_tokens), int(n_heads), int(head_dim), int(n_slots),
                     int(max_pages))
        bound = _bound()
        work = int(bound.history_work_bytes(ctypes.byref(c)))
        if work < 0:
            bad = min(n_pages, n_slots, max_pages, n_heads) < 1
            raise DlrmError(ERR_INVALID_ARG if bad else ERR_UNSUPPORTED, "HistoryCache")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        shape = (n_pages, n_heads, page_tokens, head_dim)
        new = dict(device=device)
        i32 = dict(dtype=torch.int32, device=device)
        with _on(stream, device):
            self.k_codes = torch.zeros(shape, dtype=torch.uint8, **new).view(torch.float8_e4m3fn)
            self.v_codes = torch.zeros(shape, dtype=torch.uint8, **new).view(torch.float8_e4m3fn)
            self.k_scales = torch.zeros(shape[:2], **new)
            self.v_scales = torch.zeros(shape[:2], **new)
            self.table = torch.empty((n_slots, max_pages), **i32)
            self.lengths = torch.empty(n_slots, **i32)
            self.refs = torch.empty(n_pages, **i32)
            self.free_pages = torch.empty(n_pages, **i32)
            self.n_free = torch.empty(1, **i32)
            self.err = torch.empty(1, **i32)
            self._work = torch.empty(work, dtype=torch.uint8, **new)
        for name in ("k_codes", "v_codes", "k_scales", "v_scales", "table", "lengths", "refs",
                     "free_pages", "n_free", "err"):
            setattr(c, name, getattr(self, name).data_ptr())
        c.work, c.work_bytes = self._work.data_ptr(), work
        self.device, self.n_slots, self.max_pages = device, int(n_slots), int(max_pages)
        self.n_heads, self.head_dim, self.page_tokens = int(n_heads), int(head_dim), int(page_tokens)
        self._c, self._ref, self._index = c, ctypes.byref(c), device.index
        self.reset(stream)

    def reset(self, stream=None) -> None:
        """Every page free, every slot empty, the error word cleared."""
        _check(_bound().history_reset(self._ref, _raw_stream(stream, self._index)), "history_reset")

    def error(self, stream=None) -> int:
        """Waits for ``stream``, returns the first error that the device recorded
        since the last call (INDEX_OOB before UNSUPPORTED, OOM, INVALID_ARG and
        TIMEOUT; OK if none) and clears it."""
        with _on(torch.cuda.current_stream(self.device) if stream is None else stream, self.device):
            bits = int(self.err.item())
            if bits:
                self.err.zero_()
        for code in (ERR_INDEX_OOB, ERR_UNSUPPORTED, ERR_OOM, ERR_INVALID_ARG, ERR_TIMEOUT):
            if bits & (1 << code):
                return code
        return OK


_bound_lib = None


def _bound():
    global _bound_lib
    if _bound_lib is None:
        loaded = lib()
        _bind(loaded)
        _bound_lib = loaded
    return _bound_lib


def _cache_of(cache, where: str):
    if not isinstance(cache, HistoryCache):
        raise TypeError(f"{where}: cache must be a HistoryCache")
    return cache


def history_append(cache: HistoryCache, slots, starts, k, v, stream=None) -> None:
    """Appends rows [starts[b], starts[b+1]) of ``k`` and ``v``, (rows, n_heads,
    head_dim) in float32, bfloat16 or float16, to history ``slots[b]``. ``slots``
    (B,) and ``starts`` (B+1,) are int32; a slot occurs once."""
    where = "history_append"
    c = _cache_of(cache, where)
    index = c._index
    b = _int32_vector(slots, "history_append: slots", None, index)
    _int32_vector(starts, "history_append: starts", b + 1, index)
    (rows, _, _), ks = _rows(k, "history_append: k", c.n_heads, c.head_dim, index)
    (v_rows, _, _), vs = _rows(v, "history_append: v", c.n_heads, c.head_dim, index)
    dt = _dtype_code(k, "history_append: k")
    if v.dtype is not k.dtype:
        raise TypeError(f"{where}: v: expected {k.dtype}, got {v.dtype}")
    if v_rows != rows:
        raise ValueError(f"{where}: k and v must have as many rows")
    if b > c.n_slots:
        raise ValueError(f"{where}: {b} requests for {c.n_slots} slots")
    _check(_bound().history_append(c._ref, slots.data_ptr(), starts.data_ptr(), b, k.data_ptr(),
                                   ks[0], ks[1], v.data_ptr(), vs[0], vs[1], rows, dt,
                                   _raw_stream(stream, index)), where)


def _slots_call(name: str, cache, vectors, stream, *more) -> None:
    c = _cache_of(cache, name)
    index = c._index
    b, pointers = None, []
    for label, t in vectors:
        b = _int32_vector(t, label, b, index)
        pointers.append(t.data_ptr())
    if b > c.n_slots:
        raise ValueError(f"{name}: {b} requests for {c.n_slots} slots")
    _check(getattr(_bound(), name)(c._ref, *pointers, b, *more, _raw_stream(stream, index)), name)


def history_fork(cache: HistoryCache, src, dst, stream=None) -> None:
    """The empty slot ``dst[b]`` becomes a history like ``src[b]``'s: full pages are
    shared, a last page that is not full is copied."""
    _slots_call("history_fork", cache, (("history_fork: src", src), ("history_fork: dst", dst)),
                stream)


def history_copy(cache: HistoryCache, src, dst, stream=None) -> None:
    """As history_fork, with every page copied."""
    _slots_call("history_copy", cache, (("history_copy: src", src), ("history_copy: dst", dst)),
                stream)


def history_free(cache: HistoryCache, slots, stream=None) -> None:
    """Empties slots; pages that no slot holds any more become free."""
    _slots_call("history_free", cache, (("history_free: slots", slots),), stream)


def history_trim(cache: HistoryCache, slots, window: int, sinks: int = 0, stream=None) -> None:
    """Gives up the pages that attention with this window and these sinks no
    longer reads, in queries at the histories' ends or later."""
    if not 1 <= window <= INT32_MAX or not 0 <= sinks <= INT32_MAX:
        raise ValueError("history_trim: window must be at least 1, sinks at least 0, both below 2^31")
    _slots_call("history_trim", cache, (("history_trim: slots", slots),), stream,
                operator.index(window), operator.index(sinks))


def history_compact(cache: HistoryCache, stream=None) -> None:
    """Moves pages in use to the front of the pool and rebuilds the free stack."""
    c = _cache_of(cache, "history_compact")
    _check(_bound().history_compact(c._ref, _raw_stream(stream, c._index)), "history_compact")


def _check_outputs(where, q, shape, out, lse, window, sinks, index, stream):
    """out, made (on ``stream``) if there is none, and its strides."""
    if out is None:
        if stream is None:
            out = torch.empty(shape, dtype=q.dtype, device=q.device)
        else:
            with _on(stream, q.device):
                out = torch.empty(shape, dtype=q.dtype, device=q.device)
        strides = out.stride()
    else:
        if not isinstance(out, torch.Tensor) or out.dtype is not q.dtype:
            raise TypeError(f"{where}: out: expected a {q.dtype} tensor")
        got, strides = _rows(out, "out", shape[1], shape[2], index)
        if got[0] != shape[0]:
            raise ValueError(f"{where}: out: expected {shape[0]} rows, got {got[0]}")
    if lse is not None:
        if not isinstance(lse, torch.Tensor) or lse.dtype is not torch.float32:
            raise TypeError(f"{where}: lse: expected a float32 tensor")
        if lse.shape != shape[:2] or lse.get_device() != index or not lse.is_contiguous():
            raise ValueError(f"{where}: lse: expected contiguous {tuple(shape[:2])} on {q.device}")
    if window < 0 or sinks < 0:
        raise ValueError(f"{where}: window and sinks must not be negative")
    return out, strides


def _unpackable(where, e):
    return ValueError(f"{where}: window and sinks must be integers below 2^31 ({e})")


def _scale(where, scale):
    if not -FP32_MAX <= scale <= FP32_MAX:
        raise ValueError(f"{where}: scale must be a finite float32")
    return scale


def history_attention(cache: HistoryCache, slots, starts, q, out=None, *, scale=None,
                      causal: bool = False, window: int = 0, sinks: int = 0, lse=None,
                      stream=None):
    """Attention of the query rows [starts[b], starts[b+1]) of ``q``, (rows, query
    heads, head_dim), over history ``slots[b]``; returns ``out``.

    Query heads are a multiple of the cache's heads; consecutive ones share a
    head. With ``causal`` the rows are the history's last events; otherwise each
    sees all of it (candidates to rank). ``window`` > 0 leaves a row the last
    ``window`` events and the first ``sinks``. ``scale`` defaults to head_dim
    ** -0.5. ``lse``, (rows, query heads) float32, receives the log of the sum of
    exponentials."""
    where = "history_attention"
    c = _cache_of(cache, where)
    index = c._index
    b = _int32_vector(slots, "history_attention: slots", None, index)
    _int32_vector(starts, "history_attention: starts", b + 1, index)
    shape, qs = _rows(q, "history_attention: q", None, c.head_dim, index)
    rows, heads, dim = shape
    if heads < 1 or heads % c.n_heads:
        raise ValueError(f"{where}: q: {heads} heads are no multiple of the cache's {c.n_heads}")
    dtype = _dtype_code(q, "history_attention: q")
    out, os = _check_outputs(where, q, shape, out, lse, window, sinks, index, stream)
    try:
        args = _ATTENTION.pack(
            q.data_ptr(), 0, 0, out.data_ptr(), 0 if lse is None else lse.data_ptr(), slots.data_ptr(),
            starts.data_ptr(), 0, rows, 0, qs[0], qs[1], 0, 0, 0, 0, os[0], os[1], b, heads, c.n_heads,
            dim, dtype, causal, window, sinks, dim ** -0.5 if scale is None else _scale(where, scale), 0)
    except struct.error as e:
        raise _unpackable(where, e) from None
    _check(_bound().history_attention(c._ref, args, _raw_stream(stream, index)), where)
    return out


def window_attention(q, k, v, starts, out=None, *, k_starts=None, scale=None, window: int = 0,
                     sinks: int = 0, lse=None, err_flag=None, stream=None):
    """Causal attention of ragged rows over plain keys and values; returns ``out``.

    Sequence b has the query rows [starts[b], starts[b+1]) of ``q`` (rows, heads,
    head_dim) and the rows [k_starts[b], k_starts[b+1]) of ``k`` and ``v`` (rows,
    kv heads, head_dim); ``k_starts`` defaults to ``starts``. Its queries stand at
    the last positions of its keys. ``window``, ``sinks``, ``scale`` and ``lse`` as in
    history_attention. ``err_flag``: (1,) int32, receives the error bits of bad starts and
    of a wait that ran out."""
    where = "window_attention"
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{where}: {name} must be a torch.Tensor")
        if t.dtype is not q.dtype:
            raise TypeError(f"{where}: {name}: expected {q.dtype}, got {t.dtype}")
    if not q.is_cuda:
        raise ValueError(f"{where}: q must be a CUDA tensor")
    index = q.get_device()
    shape, qs = _rows(q, "window_attention: q", None, None, index)
    rows, heads, dim = shape
    (k_rows, kv_heads, _), ks = _rows(k, "window_attention: k", None, dim, index)
    (v_rows, _, _), vs = _rows(v, "window_attention: v", kv_heads, dim, index)
    if k_rows != v_rows:
        raise ValueError(f"{where}: k and v must have as many rows")
    if kv_heads < 1 or heads < 1 or heads % kv_heads:
        raise ValueError(f"{where}: {heads} query heads are no multiple of {kv_heads} kv heads")
    b = _int32_vector(starts, "window_attention: starts", None, index) - 1
    if b < 0:
        raise ValueError(f"{where}: starts: expected at least one entry")
    if k_starts is None:
        k_starts = starts
    else:
        _int32_vector(k_starts, "window_attention: k_starts", b + 1, index)
    dtype = _dtype_code(q, "window_attention: q")
    out, os = _check_outputs(where, q, shape, out, lse, window, sinks, index, stream)
    if err_flag is not None:
        _int32_vector(err_flag, "window_attention: err_flag", 1, index)
    try:
        args = _ATTENTION.pack(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
            0 if lse is None else lse.data_ptr(), 0, starts.data_ptr(), k_starts.data_ptr(), rows,
            k_rows, qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], os[0], os[1], b, heads, kv_heads,
            dim, dtype, 1, window, sinks, dim ** -0.5 if scale is None else _scale(where, scale),
            0 if err_flag is None else err_flag.data_ptr())
    except struct.error as e:
        raise _unpackable(where, e) from None
    _check(_bound().window_attention(args, _raw_stream(stream, index)), where)
    return out


def attention_test_stall(wait_limit_ns: int = 0, withhold: bool = False) -> None:
    """Failure-detection test hook: the limit of the bounded device waits of later
    attention calls (0: the default) and, with ``withhold``, a piece of work is kept back, so
    that the wait on it runs out (TIMEOUT in the cache's error word, or in ``err_flag``).
    ``attention_test_stall()`` restores normal operation."""
    _check(_bound().attention_test_stall(int(wait_limit_ns), 1 if withhold else 0), "attention_test_stall")
