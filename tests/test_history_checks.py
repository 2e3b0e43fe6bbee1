"""The event-history calls refuse bad arguments on the host, before anything is
launched (no GPU needed), and the restatement that the GPU tests compare with
holds on its own."""
import ctypes

import numpy as np
import pytest

import history_ref as ref

torch = pytest.importorskip("torch")
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402
from dlrm_embedding_interaction_gb300 import history  # noqa: E402

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from dlrm_embedding_interaction_gb300 import build
    build.build()
    return history._bound()


def pool(**change):
    c = history._History(8, 64, 2, 64, 4, 3)
    for name in ("k_codes", "v_codes", "k_scales", "v_scales", "table", "lengths", "refs",
                 "free_pages", "n_free", "err", "work"):
        setattr(c, name, FAKE)
    c.work_bytes = 1 << 40
    for name, value in change.items():
        setattr(c, name, value)
    return c


def attention(**change):
    a = history._Attention()
    for name in ("q", "k", "v", "out", "slots", "q_starts", "k_starts"):
        setattr(a, name, FAKE)
    a.q_rows = a.k_rows = 5
    a.batch, a.n_heads, a.n_kv_heads, a.head_dim, a.scale = 1, 4, 2, 64, 0.125
    for name, value in change.items():
        setattr(a, name, value)
    return a


BAD_POOLS = [(dict(n_pages=0), dl.ERR_INVALID_ARG), (dict(n_heads=0), dl.ERR_INVALID_ARG),
             (dict(n_slots=0), dl.ERR_INVALID_ARG), (dict(max_pages=-1), dl.ERR_INVALID_ARG),
             (dict(page_tokens=48), dl.ERR_UNSUPPORTED), (dict(head_dim=80), dl.ERR_UNSUPPORTED),
             (dict(n_slots=1 << 20, max_pages=1 << 12), dl.ERR_UNSUPPORTED),
             (dict(max_pages=1 << 25), dl.ERR_UNSUPPORTED),
             (dict(k_codes=0), dl.ERR_INVALID_ARG), (dict(v_codes=FAKE + 8), dl.ERR_INVALID_ARG),
             (dict(k_scales=FAKE + 2), dl.ERR_INVALID_ARG), (dict(table=0), dl.ERR_INVALID_ARG),
             (dict(lengths=FAKE + 1), dl.ERR_INVALID_ARG), (dict(refs=0), dl.ERR_INVALID_ARG),
             (dict(free_pages=0), dl.ERR_INVALID_ARG), (dict(n_free=FAKE + 2), dl.ERR_INVALID_ARG),
             (dict(err=0), dl.ERR_INVALID_ARG), (dict(work=FAKE + 4), dl.ERR_INVALID_ARG),
             (dict(work_bytes=100), dl.ERR_INVALID_ARG)]


@pytest.mark.parametrize("change,status", BAD_POOLS)
def test_every_call_refuses_a_bad_pool(lib, change, status):
    h = ctypes.byref(pool(**change))
    a = ctypes.byref(attention())
    assert lib.history_reset(h, None) == status
    assert lib.history_append(h, FAKE, FAKE, 1, FAKE, 1, 1, FAKE, 1, 1, 1, 0, None) == status
    assert lib.history_fork(h, FAKE, FAKE, 1, None) == status
    assert lib.history_copy(h, FAKE, FAKE, 1, None) == status
    assert lib.history_free(h, FAKE, 1, None) == status
    assert lib.history_trim(h, FAKE, 1, 1, 0, None) == status
    assert lib.history_compact(h, None) == status
    assert lib.history_attention(h, a, None) == status


def test_null_pools_and_empty_calls(lib):
    h = ctypes.byref(pool())
    assert lib.history_reset(None, None) == dl.ERR_INVALID_ARG
    assert lib.history_work_bytes(None) == -1
    assert lib.history_work_bytes(ctypes.byref(pool(head_dim=48))) == -1
    assert lib.history_work_bytes(h) > 0
    # nothing to do: OK without a launch
    assert lib.history_append(h, None, None, 0, None, 1, 1, None, 1, 1, 0, 0, None) == dl.OK
    assert lib.history_append(h, FAKE, FAKE, 1, None, 1, 1, None, 1, 1, 0, 0, None) == dl.OK
    assert lib.history_fork(h, None, None, 0, None) == dl.OK
    assert lib.history_free(h, None, 0, None) == dl.OK
    assert lib.history_attention(h, ctypes.byref(attention(batch=0)), None) == dl.OK
    assert lib.window_attention(ctypes.byref(attention(q_rows=0)), None) == dl.OK


def test_page_calls_check_their_arguments(lib):
    h = ctypes.byref(pool())
    bad = dl.ERR_INVALID_ARG
    assert lib.history_append(h, FAKE, FAKE, 5, FAKE, 1, 1, FAKE, 1, 1, 1, 0, None) == bad  # > slots
    assert lib.history_append(h, FAKE, FAKE, -1, FAKE, 1, 1, FAKE, 1, 1, 1, 0, None) == bad
    assert lib.history_append(h, None, FAKE, 1, FAKE, 1, 1, FAKE, 1, 1, 1, 0, None) == bad
    assert lib.history_append(h, FAKE, None, 1, FAKE, 1, 1, FAKE, 1, 1, 1, 0, None) == bad
    assert lib.history_append(h, FAKE, FAKE, 1, FAKE + 2, 1, 1, FAKE, 1, 1, 1, 0, None) == bad
    assert lib.history_append(h, FAKE, FAKE, 1, FAKE, -1, 1, FAKE, 1, 1, 1, 0, None) == bad
    assert lib.history_append(h, FAKE, FAKE, 1, FAKE, 1, 1, FAKE, 1, 1, 1, 3, None) == bad
    assert lib.history_append(h, FAKE, FAKE, 1, FAKE, 1, 1, FAKE, 1, 1, -1, 0, None) == bad
    assert lib.history_fork(h, FAKE, FAKE + 2, 1, None) == bad
    assert lib.history_copy(h, None, FAKE, 1, None) == bad
    assert lib.history_free(h, FAKE, 5, None) == bad
    assert lib.history_trim(h, FAKE, 1, 0, 0, None) == bad
    assert lib.history_trim(h, FAKE, 1, 5, -1, None) == bad


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), dl.ERR_INVALID_ARG), (dict(q_rows=-1), dl.ERR_INVALID_ARG),
    (dict(n_heads=3), dl.ERR_INVALID_ARG), (dict(n_heads=0), dl.ERR_INVALID_ARG),
    (dict(dtype=3), dl.ERR_INVALID_ARG), (dict(window=-1), dl.ERR_INVALID_ARG),
    (dict(sinks=-1), dl.ERR_INVALID_ARG), (dict(scale=float("nan")), dl.ERR_INVALID_ARG),
    (dict(q=0), dl.ERR_INVALID_ARG), (dict(out=FAKE + 2), dl.ERR_INVALID_ARG),
    (dict(lse=FAKE + 2), dl.ERR_INVALID_ARG), (dict(q_starts=0), dl.ERR_INVALID_ARG),
    (dict(ld_q=-4), dl.ERR_INVALID_ARG), (dict(q_rows=1 << 31), dl.ERR_UNSUPPORTED)])
def test_attention_calls_check_their_arguments(lib, change, status):
    a = ctypes.byref(attention(**change))
    assert lib.history_attention(ctypes.byref(pool()), a, None) == status
    assert lib.window_attention(a, None) == status


def test_window_attention_checks_its_keys(lib):
    for change, status in ((dict(k=0), dl.ERR_INVALID_ARG), (dict(v=FAKE + 2), dl.ERR_INVALID_ARG),
                           (dict(k_starts=0), dl.ERR_INVALID_ARG), (dict(k_rows=-1), dl.ERR_INVALID_ARG),
                           (dict(head_dim=80), dl.ERR_UNSUPPORTED), (dict(n_kv_heads=0), dl.ERR_INVALID_ARG),
                           (dict(k_rows=1 << 31), dl.ERR_UNSUPPORTED)):
        assert lib.window_attention(ctypes.byref(attention(**change)), None) == status
    assert lib.window_attention(None, None) == dl.ERR_INVALID_ARG
    assert lib.history_attention(ctypes.byref(pool()), ctypes.byref(attention(slots=0)),
                                 None) == dl.ERR_INVALID_ARG


def test_the_binding_refuses_wrong_tensors():
    q = torch.zeros(4, 2, 64)
    with pytest.raises(TypeError):
        dl.history_attention("cache", None, None, q)
    with pytest.raises(ValueError):
        dl.HistoryCache(4, 4, 4, 1, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        dl.window_attention(q, q, q, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        dl.window_attention(q, q.half(), q, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        history._dtype_code(q.double(), "q")
    with pytest.raises(TypeError):
        history._int32_vector(torch.zeros(3), "slots", None, q.device)
    with pytest.raises(ValueError):
        history._int32_vector(torch.zeros(3, dtype=torch.int32), "starts", 4, q.device)
    with pytest.raises(ValueError):
        history._int32_vector(torch.zeros(6, dtype=torch.int32)[::2], "starts", 3, q.device)
    with pytest.raises(ValueError, match="last dimension"):
        history._rows(q.transpose(1, 2), "q", None, None, q.device)
    with pytest.raises(ValueError):
        history._rows(q, "q", 3, None, q.device)


# ------------------------------------------------------------------ the restatement

def test_e4m3_restatement_against_torch():
    codes = np.arange(256, dtype=np.uint8)
    got = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(got, ref.VALUES)
    x = np.concatenate([np.linspace(-460, 460, 20001), ref.VALUES[:127],
                        (ref.VALUES[:126] + ref.VALUES[1:127]) / 2]).astype(np.float32)
    want = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    have = ref.to_e4m3(x)
    np.testing.assert_array_equal(ref.VALUES[have], ref.VALUES[want])
    assert ref.to_e4m3([np.nan])[0] == 0x7f and ref.to_e4m3([np.inf])[0] == 126


def test_scale_restatement():
    assert ref.scale_of([448.0]) == 1.0 and ref.scale_of([448.1]) == 2.0 and ref.scale_of([224.0]) == 0.5
    assert ref.scale_of([0.0]) == 2.0 ** -60 and ref.scale_of([np.inf, 1e38]) == 2.0 ** 60
    assert ref.scale_of([np.nan, -7.0]) == 2.0 ** -6


def test_attention_restatement_against_torch():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((5, 2, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    out, lse = ref.attention(q, k, v, 0.3, True, 4, 2)
    pos = np.arange(5)[:, None] + 4
    t = np.arange(9)
    mask = (t <= pos) & ((t > pos - 4) | (t < 2))
    x = torch.from_numpy(np.einsum("ihd,thd->hit", q, k) * 0.3).masked_fill(~torch.from_numpy(mask), -np.inf)
    want = torch.einsum("hit,thd->ihd", x.softmax(-1), torch.from_numpy(v)).numpy()
    np.testing.assert_allclose(out, want, atol=1e-14)
    np.testing.assert_allclose(lse, x.logsumexp(-1).numpy().T, atol=1e-14)


def test_pool_restatement_keeps_its_books():
    rng = np.random.default_rng(0)
    p = ref.Pool(20, 6, 4, 1, 32, 32)
    for step in range(200):
        op, a, b = rng.integers(0, 5), int(rng.integers(0, 6)), int(rng.integers(0, 6))
        x = rng.standard_normal((40, 1, 32))
        if op == 0:
            p.append([a], [0, int(rng.integers(0, 40))], (x, x))
        elif op < 3:
            p.fork([a], [b], op == 1)
        elif op == 3:
            p.release([a, b])
        else:
            p.compact()
        held = p.table[p.table >= 0]
        assert (np.bincount(held, minlength=20) == p.refs).all()
        assert sorted(p.free + np.flatnonzero(p.refs).tolist()) == list(range(20))
