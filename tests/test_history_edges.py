"""Event-history calls at the edges, on the host: what they refuse before anything is
launched or allocated (no GPU needed)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402
from dlrm_embedding_interaction_gb300 import history  # noqa: E402


class OnDevice(torch.Tensor):
    """A host tensor that says it is on a CUDA device (of index -1, as host tensors do)."""
    is_cuda = True


class Library:
    """Stands in for the library: every call of it is written down, and is OK."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append(name) or dl.OK


@pytest.fixture
def fake(monkeypatch):
    """A cache whose tensors and stream are the host's, and the library that its calls reach."""
    lib = Library()
    monkeypatch.setattr(history, "_bound", lambda: lib)
    monkeypatch.setattr(history, "_current_device", lambda: -1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    cache = object.__new__(history.HistoryCache)
    cache._index, cache._ref, cache.n_slots, cache.n_heads, cache.head_dim = -1, None, 8, 2, 64
    cache.device = torch.device("cpu")
    return cache, lib


def calls(cache):
    """Every operator once, with good arguments."""
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)   # noqa: E731
    q, kv = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    plain = [t.as_subclass(OnDevice) for t in (q, kv, kv)]
    return {
        "history_reset": lambda: cache.reset(),
        "history_append": lambda: dl.history_append(cache, i32(0), i32(0, 3), kv, kv),
        "history_fork": lambda: dl.history_fork(cache, i32(0), i32(1)),
        "history_copy": lambda: dl.history_copy(cache, i32(0), i32(1)),
        "history_free": lambda: dl.history_free(cache, i32(0)),
        "history_trim": lambda: dl.history_trim(cache, i32(0), 5),
        "history_compact": lambda: dl.history_compact(cache),
        "history_attention": lambda: dl.history_attention(cache, i32(0), i32(0, 3), q),
        "window_attention": lambda: dl.window_attention(*plain, i32(0, 3)),
    }


# ------------------------------------------------------------------ devices

def test_good_calls_reach_the_library(fake):
    cache, lib = fake
    for name, call in calls(cache).items():
        call()
        assert lib.calls.pop() == name


def test_calls_refuse_tensors_that_are_not_on_the_current_device(fake, monkeypatch):
    """A launch goes to the current device, with the other one's pointers."""
    cache, lib = fake
    monkeypatch.setattr(history, "_current_device", lambda: 1)
    for name, call in calls(cache).items():
        with pytest.raises(ValueError, match="current device"):
            call()
    assert not lib.calls


def test_a_cache_is_made_on_the_current_device_only(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: pytest.fail("allocated"))
    with pytest.raises(ValueError, match="current device"):
        dl.HistoryCache(4, 4, 4, 1, 64, device="cuda:1")


# ------------------------------------------------------------------ numbers

@pytest.mark.parametrize("number", [2 ** 31, 2 ** 32 + 1, 2 ** 64 + 1, -1, -2 ** 32 + 1, 2.5])
def test_numbers_past_32_bits_are_refused(fake, number):
    """Not cut off: a window of 2^32 + 1 is not one of 1, which gives nearly all up."""
    cache, lib = fake
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)   # noqa: E731
    q = torch.zeros(3, 4, 64)
    plain = [q.as_subclass(OnDevice)] * 3
    for name in ("window", "sinks"):
        for call in (lambda **n: dl.history_trim(cache, i32(0), **dict(dict(window=5), **n)),
                     lambda **n: dl.history_attention(cache, i32(0), i32(0, 3), q, **n),
                     lambda **n: dl.window_attention(*plain, i32(0, 3), **n)):
            with pytest.raises((ValueError, TypeError)):
                call(**{name: number})
    with pytest.raises(ValueError):
        dl.history_attention(cache, i32(0), i32(0, 3), q, scale=1e39)
    assert not lib.calls


def test_a_cache_of_sizes_past_32_bits_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: pytest.fail("allocated"))
    good = dict(n_pages=4, n_slots=4, max_pages=4, n_heads=1, head_dim=64, page_tokens=64)
    for name, value in good.items():
        with pytest.raises(dl.DlrmError) as e:
            dl.HistoryCache(**dict(good, **{name: value + 2 ** 32}))
        assert e.value.status == dl.ERR_UNSUPPORTED


# ------------------------------------------------------------------ streams

@pytest.fixture
def streams(monkeypatch):
    """Which stream is current where tensors are made: "current", or what was asked for."""
    import contextlib
    seen, current = [], ["current"]

    @contextlib.contextmanager
    def stream(s):
        current.append(s.number)
        yield
        current.pop()

    class External:
        def __init__(self, number, device=None):
            self.number = number

    def made(real):
        def make(*shape, dtype=None, device=None):
            seen.append(current[-1])
            return real(*shape, dtype=dtype)
        return make

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch, "zeros", made(torch.zeros))
    monkeypatch.setattr(torch, "empty", made(torch.empty))
    return seen


def test_tensors_are_made_on_the_stream_of_the_call(fake, streams, monkeypatch):
    """Otherwise they are filled, or their memory is still used, out of that stream's order."""
    cache, lib = fake
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)   # noqa: E731
    q = torch.ones(3, 4, 64)
    plain = [q.as_subclass(OnDevice)] * 3
    for stream in (None, 77):
        want = "current" if stream is None else stream
        dl.history_attention(cache, i32(0), i32(0, 3), q, stream=stream)
        dl.window_attention(*plain, i32(0, 3), stream=stream)
        assert streams == [want] * 2
        streams.clear()
    monkeypatch.setattr(history, "_current_device", lambda: 0)
    for stream in (None, 77):
        history.HistoryCache(4, 4, 4, 1, 64, stream=stream)
        assert len(streams) == 11 and set(streams) == {"current" if stream is None else stream}
        streams.clear()
