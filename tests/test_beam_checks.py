"""The beam search's calls on the host (no GPU needed): what they refuse before anything is
launched, their launch code over a stand-in for the CUDA runtime, and the restatement that
the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import beam_ref

torch = pytest.importorskip("torch")
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402
from dlrm_embedding_interaction_gb300 import beams, history  # noqa: E402
from test_history_checks import BAD_POOLS, FAKE, attention, pool  # noqa: E402
from test_history_edges import OnDevice, fake, streams  # noqa: E402, F401
from test_history_launch import lib as fake_lib  # noqa: E402, F401


@pytest.fixture(scope="module")
def lib():
    from dlrm_embedding_interaction_gb300 import build
    build.build()
    beams._bound()
    return history._bound()


def select(**change):
    a = beams._BeamSelect()
    for name in ("logits", "scores", "allowed", "starts", "out_scores", "out_rows", "out_tokens", "err", "work"):
        setattr(a, name, FAKE)
    a.rows, a.vocab, a.ld, a.ld_allowed, a.groups, a.width, a.dtype = 5, 100, 100, 100, 2, 4, 0
    a.work_bytes = 1 << 40
    for name, value in change.items():
        setattr(a, name, value)
    return a


# ------------------------------------------------------------------ the C boundary

@pytest.mark.parametrize("change,status", BAD_POOLS)
def test_the_new_calls_refuse_a_bad_pool(lib, change, status):
    h = ctypes.byref(pool(**change))
    assert lib.history_reorder(h, FAKE, FAKE, 1, None) == status
    assert lib.history_prefix_attention(h, ctypes.byref(attention()), FAKE, 1, None) == status


def test_reorder_checks_its_arguments(lib):
    h = ctypes.byref(pool())
    bad = dl.ERR_INVALID_ARG
    assert lib.history_reorder(h, FAKE, FAKE, 5, None) == bad     # > slots
    assert lib.history_reorder(h, FAKE, FAKE, -1, None) == bad
    assert lib.history_reorder(h, None, FAKE, 1, None) == bad
    assert lib.history_reorder(h, FAKE, FAKE + 2, 1, None) == bad
    assert lib.history_reorder(h, None, None, 0, None) == dl.OK


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), dl.ERR_INVALID_ARG), (dict(q_rows=-1), dl.ERR_INVALID_ARG), (dict(batch=5), dl.ERR_INVALID_ARG),
    (dict(n_heads=3), dl.ERR_INVALID_ARG), (dict(dtype=3), dl.ERR_INVALID_ARG), (dict(window=-1), dl.ERR_INVALID_ARG),
    (dict(scale=float("nan")), dl.ERR_INVALID_ARG), (dict(q=0), dl.ERR_INVALID_ARG), (dict(slots=0), dl.ERR_INVALID_ARG),
    (dict(out=FAKE + 2), dl.ERR_INVALID_ARG), (dict(q_starts=0), dl.ERR_INVALID_ARG), (dict(ld_out=60), dl.ERR_INVALID_ARG),
    (dict(q_rows=1 << 31), dl.ERR_UNSUPPORTED), (dict(q_rows=1 << 18, ld_out=256, ld_out_head=64), dl.ERR_UNSUPPORTED)])
def test_prefix_attention_checks_its_arguments(lib, change, status):
    a = ctypes.byref(attention(**change))
    assert lib.history_prefix_attention(ctypes.byref(pool()), a, FAKE, 1, None) == status


def test_prefix_attention_checks_its_groups(lib):
    h, a = ctypes.byref(pool()), ctypes.byref(attention(ld_out=256, ld_out_head=64))
    assert lib.history_prefix_attention(h, a, FAKE, -1, None) == dl.ERR_INVALID_ARG
    assert lib.history_prefix_attention(h, a, FAKE, 5, None) == dl.ERR_INVALID_ARG      # > slots
    assert lib.history_prefix_attention(h, a, None, 1, None) == dl.ERR_INVALID_ARG
    assert lib.history_prefix_attention(h, a, FAKE + 1, 1, None) == dl.ERR_INVALID_ARG
    assert lib.history_prefix_attention(h, None, FAKE, 1, None) == dl.ERR_INVALID_ARG
    assert lib.history_prefix_attention(h, a, FAKE, 0, None) == dl.OK
    assert lib.history_prefix_attention(h, ctypes.byref(attention(batch=0)), FAKE, 1, None) == dl.OK


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), dl.ERR_INVALID_ARG), (dict(vocab=0), dl.ERR_INVALID_ARG), (dict(ld=-1), dl.ERR_INVALID_ARG),
    (dict(ld_allowed=-1), dl.ERR_INVALID_ARG), (dict(groups=-1), dl.ERR_INVALID_ARG), (dict(width=0), dl.ERR_INVALID_ARG),
    (dict(dtype=3), dl.ERR_INVALID_ARG), (dict(logits=0), dl.ERR_INVALID_ARG), (dict(logits=FAKE + 2), dl.ERR_INVALID_ARG),
    (dict(scores=FAKE + 2), dl.ERR_INVALID_ARG), (dict(starts=0), dl.ERR_INVALID_ARG),
    (dict(out_scores=0), dl.ERR_INVALID_ARG), (dict(out_rows=FAKE + 1), dl.ERR_INVALID_ARG),
    (dict(out_tokens=0), dl.ERR_INVALID_ARG), (dict(err=FAKE + 1), dl.ERR_INVALID_ARG),
    (dict(vocab=1 << 20, ld=1 << 20, work=0), dl.ERR_INVALID_ARG), (dict(vocab=1 << 20, work=FAKE + 8), dl.ERR_INVALID_ARG),
    (dict(vocab=1 << 20, work_bytes=100), dl.ERR_INVALID_ARG), (dict(width=257), dl.ERR_UNSUPPORTED),
    (dict(vocab=1 << 31), dl.ERR_UNSUPPORTED), (dict(rows=1 << 31), dl.ERR_UNSUPPORTED),
    (dict(rows=1 << 24, vocab=1 << 30), dl.ERR_UNSUPPORTED)])
def test_select_checks_its_arguments(lib, change, status):
    a = select(**change)
    assert lib.beam_select(ctypes.byref(a), None) == status
    assert lib.beam_select(None, None) == dl.ERR_INVALID_ARG


def test_select_tells_its_scratch(lib):
    need = lambda **c: lib.beam_select_work_bytes(ctypes.byref(select(**c)))   # noqa: E731
    assert need() == 0                              # one launch, few rows
    assert need(rows=1000, groups=500) > 0
    assert need(vocab=1 << 20) > need(vocab=1 << 16) > 0
    assert need(width=0) == need(width=300) == lib.beam_select_work_bytes(None) == -1
    assert lib.beam_select(ctypes.byref(select(groups=0)), None) == dl.OK


# ------------------------------------------------------------------ launches, over the stand-in

@pytest.mark.parametrize("head_dim", [32, 64, 128])
@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("rows", [4, 5000])
def test_launches_on_every_device_of_a_process(fake_lib, head_dim, dtype, rows):  # noqa: F811
    """A call that shares is two launches, one that is too small for it one."""
    ld = 4 * head_dim
    more = dict(head_dim=head_dim, dtype=dtype, q_rows=rows, ld_q=ld, ld_q_head=head_dim, ld_out=ld, ld_out_head=head_dim)
    a = ctypes.byref(attention(**more))
    for max_pages, launches in ((3, 1 if rows == 4 else 2), (100000, 2)):
        h = ctypes.byref(pool(head_dim=head_dim, max_pages=max_pages, n_slots=8))
        if max_pages == 3 and rows > 4:
            continue
        for device in (0, 1, 63, 64, 65):
            fake_lib.fake_set_device(device)
            before = fake_lib.fake_launches()
            assert fake_lib.history_prefix_attention(h, a, FAKE, 1, None) == dl.OK, device
            assert fake_lib.fake_launches() == before + launches
    fake_lib.fake_set_device(0)


@pytest.mark.parametrize("n_heads,batch", [(1, 1), (1, 3000), (131071, 4)])
def test_reorder_launches(fake_lib, n_heads, batch):  # noqa: F811
    h = ctypes.byref(pool(n_heads=n_heads, page_tokens=128, head_dim=128, n_slots=3000))
    before = fake_lib.fake_launches()
    assert fake_lib.history_reorder(h, 0x10000, 0x10000, batch, None) == dl.OK
    assert fake_lib.fake_launches() == before + 3


@pytest.mark.parametrize("vocab,rows,launches", [(100, 5, 1), (100, 0, 1), (5000, 5, 2), (1 << 20, 5, 2), (5000, 0, 1)])
@pytest.mark.parametrize("change", [{}, dict(allowed=0), dict(logits=FAKE + 4), dict(dtype=1), dict(dtype=2, width=256)])
def test_select_launches(fake_lib, vocab, rows, launches, change):  # noqa: F811
    beams._bind(fake_lib)
    before = fake_lib.fake_launches()
    a = select(vocab=vocab, ld=vocab, ld_allowed=vocab, rows=rows, **change)
    assert fake_lib.beam_select(ctypes.byref(a), None) == dl.OK
    assert fake_lib.fake_launches() == before + launches


# ------------------------------------------------------------------ the binding

def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.fixture
def library(fake, monkeypatch):  # noqa: F811
    cache, lib = fake
    monkeypatch.setattr(beams, "_bound", lambda: lib)
    monkeypatch.setattr(beams, "_work_bytes", lambda sizes: 64)
    return cache, lib


def calls(cache):
    logits = torch.zeros(4, 9).as_subclass(OnDevice)
    return {
        "history_reorder": lambda: dl.history_reorder(cache, i32(0, 1), i32(1, 1)),
        "history_prefix_attention": lambda: dl.history_prefix_attention(cache, i32(0), i32(0, 3), i32(0, 1),
                                                                        torch.zeros(3, 4, 64)),
        "beam_select": lambda: dl.beam_select(logits, torch.zeros(4), i32(0, 4), 2),
    }


def test_good_calls_reach_the_library(library):
    cache, lib = library
    for name, call in calls(cache).items():
        call()
        assert lib.calls.pop() == name


def test_calls_refuse_tensors_that_are_not_on_the_current_device(library, monkeypatch):
    cache, lib = library
    monkeypatch.setattr(history, "_current_device", lambda: 1)
    for call in calls(cache).values():
        with pytest.raises(ValueError, match="current device"):
            call()
    assert not lib.calls


def test_tensors_are_made_on_the_stream_of_the_call(library, streams):  # noqa: F811
    cache, lib = library
    logits = torch.ones(4, 9).as_subclass(OnDevice)
    q = torch.ones(3, 4, 64)
    for stream in (None, 77):
        dl.history_prefix_attention(cache, i32(0), i32(0, 3), i32(0, 1), q, stream=stream)
        dl.beam_select(logits, None, i32(0, 4), 2, stream=stream)
        assert len(streams) == 5 and set(streams) == {"current" if stream is None else stream}
        streams.clear()


def test_the_binding_refuses_wrong_tensors(library):
    cache, lib = library
    logits = torch.zeros(4, 9).as_subclass(OnDevice)
    scores, starts = torch.zeros(4), i32(0, 4)
    q = torch.zeros(3, 4, 64)
    good = dict(logits=logits, scores=scores, starts=starts, width=2)
    for change, error in ((dict(logits=torch.zeros(4, 9)), ValueError), (dict(logits=logits.double()), TypeError),
                          (dict(logits=logits[0]), ValueError), (dict(logits=logits.t()), ValueError),
                          (dict(logits="x"), TypeError), (dict(logits=logits[:, :0]), ValueError),
                          (dict(scores=scores.half()), TypeError), (dict(scores=scores[:3]), ValueError),
                          (dict(scores=torch.zeros(8)[::2]), ValueError), (dict(starts=starts.long()), TypeError),
                          (dict(starts=i32()), ValueError), (dict(width=0), dl.DlrmError), (dict(width=257), dl.DlrmError),
                          (dict(width=2.5), TypeError), (dict(allowed=torch.ones(4, 9)), TypeError),
                          (dict(allowed=torch.ones(3, 9, dtype=torch.bool)), ValueError),
                          (dict(allowed=torch.ones(9, 4, dtype=torch.bool).t()), ValueError),
                          (dict(err_flag=i32(0, 0)), ValueError)):
        with pytest.raises(error):
            dl.beam_select(**dict(good, **change))
    with pytest.raises(ValueError, match="slots"):
        dl.history_reorder(cache, i32(*range(9)), i32(*range(9)))
    with pytest.raises(ValueError):
        dl.history_reorder(cache, i32(0, 1), i32(0))
    with pytest.raises(ValueError, match="groups"):
        dl.history_prefix_attention(cache, i32(0), i32(0, 3), i32(), q)
    with pytest.raises(ValueError, match="slots"):
        dl.history_prefix_attention(cache, i32(0), i32(0, 3), i32(*range(12)), q)
    with pytest.raises(TypeError):
        dl.history_prefix_attention(cache, i32(0), i32(0, 3), starts.long(), q)
    with pytest.raises(TypeError):
        dl.history_prefix_attention("cache", i32(0), i32(0, 3), starts, q)
    assert not lib.calls


# ------------------------------------------------------------------ the restatement

def test_pool_restatement_keeps_its_books():
    rng = np.random.default_rng(0)
    p = beam_ref.Pool(40, 8, 4, 1, 32, 32)
    for step in range(300):
        x = rng.standard_normal((40, 1, 32))
        slots = rng.permutation(8)[:int(rng.integers(1, 8))].tolist()
        before = (p.table.copy(), p.lengths.copy(), [c.copy() for c in p.codes], [s.copy() for s in p.scales])
        if step % 3 == 0:
            p.append(slots[:1], [0, int(rng.integers(0, 40))], (x, x))
        elif step % 3 == 1:
            parents = rng.integers(-1, len(slots), len(slots)).tolist()
            done = p.reorder(slots, parents)
            for s, parent in zip(slots, parents):   # each slot holds what its parent held
                want = s if not done else -1 if parent == -1 else slots[parent]
                assert p.lengths[s] == (0 if want == -1 else before[1][want])
                for j in range(p.pages(p.lengths[s])):
                    a, b = p.table[s, j], before[0][want, j]
                    e = min(32, int(p.lengths[s]) - 32 * j)
                    for now, was in zip(p.codes, before[2]):
                        np.testing.assert_array_equal(now[a, :, :e], was[b, :, :e])
                    for now, was in zip(p.scales, before[3]):
                        np.testing.assert_array_equal(now[a], was[b])
        elif step % 9 == 2:
            p.release(slots[:2])
        held = p.table[p.table >= 0]
        assert (np.bincount(held, minlength=40) == p.refs).all()
        assert sorted(p.free + np.flatnonzero(p.refs).tolist()) == list(range(40))
        last = [p.table[s, int(n) // 32] for s, n in enumerate(p.lengths) if n % 32]
        assert len(set(last)) == len(last)          # a last page that is not full has one holder


def test_selection_restatement_against_torch():
    rng = np.random.default_rng(1)
    x, s = rng.standard_normal((5, 30)), rng.standard_normal(5)
    allowed = rng.random((5, 30)) < 0.5
    allowed[4] = False
    best, rows, tokens, _ = beam_ref.select(x, s, [0, 3, 5], 6, allowed)
    t = torch.from_numpy(x).masked_fill(~torch.from_numpy(allowed), -np.inf).log_softmax(1) + torch.from_numpy(s)[:, None]
    for g, (a, b) in enumerate(((0, 3), (3, 5))):
        want = t[a:b].nan_to_num(-np.inf).reshape(-1).topk(6)
        np.testing.assert_allclose(best[g], want.values.numpy(), atol=1e-12)
        np.testing.assert_array_equal(30 * (rows[g] - a) + tokens[g], want.indices.numpy())
