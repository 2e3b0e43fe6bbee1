"""The history-ranking example end to end against a float64 restatement: the cache
against the encoder's keys and values within e4m3's rounding, the probabilities
against those that the cache's contents give."""
import importlib.util
import os

import numpy as np
import pytest

import history_ref as ref

torch = pytest.importorskip("torch")
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    from dlrm_embedding_interaction_gb300 import build
    build.build()
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location("history_ranking",
                                                  os.path.join(ROOT, "examples", "history_ranking.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def f64(t):
    return t.detach().double().cpu().numpy()


def encode(r, ids, counts):
    """The encoder in float64: keys and values of each history."""
    x = f64(r.items)[ids.cpu().numpy()]
    heads, hd = r.heads, r.dim // r.heads
    q, k, v = (x @ f64(w).T for w in r.enc)
    out, at = [], 0
    for n in counts:
        h, _ = ref.attention(*(y[at:at + n].reshape(n, heads, hd) for y in (q, k, v)), hd ** -0.5, True,
                             r.window, r.sinks)
        out.append([(h.reshape(n, r.dim) @ f64(w).T).reshape(n, heads, hd) for w in r.kv])
        at += n
    return out


def cached(cache, slot):
    """A history's keys and values as the cache holds them."""
    n, page = int(cache.lengths[slot]), cache.page_tokens
    ids = cache.table[slot, : -(-n // page)].long()
    out = []
    for codes, scales in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        x = codes.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * scales[ids].double()[:, :, None, None]
        s = scales[ids].double()[:, :, None, None].expand_as(x)
        out.append([f64(y.permute(0, 2, 1, 3).reshape(-1, *y.shape[1::2])[:n]) for y in (x, s)])
    return out


def test_example_main_runs(example, capsys):
    example.main()
    assert "64 users" in capsys.readouterr().out


def test_ranking_against_float64(example):
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    items = torch.randn(500, 64, generator=g, device="cuda")
    r = example.HistoryRanker(items, heads=2, n_users=4, max_events=300, window=40, sinks=3, page_tokens=32)

    def some(counts):
        return torch.randint(500, (sum(counts),), generator=g, device="cuda"), example.starts_of(counts)

    lens, events, cands = [130, 1, 0, 64], [2, 1, 3, 0], [5, 70, 1, 9]
    users = torch.arange(4, dtype=torch.int32, device="cuda")
    ids, at = some(lens)
    r.load(users, ids, at)
    for u, want in enumerate(encode(r, ids, lens)):
        for (x, scale), y in zip(cached(r.cache, u), want):
            # half an ulp of e4m3: 2^-4 of the value, 2^-10 scales below its normal range
            assert (np.abs(x - y) <= 2.0 ** -4 * np.abs(y) + 2.0 ** -10 * scale + 1e-4).all()
    session, candidates = some(events), some(cands)
    state = r.cache.table.clone(), r.cache.n_free.clone()
    p = f64(r.rank(users, *session, *candidates))
    assert r.cache.error() == dl.OK
    assert torch.equal(r.cache.table, state[0]) and torch.equal(r.cache.n_free, state[1])
    # the forks as rank() made them, kept this time
    forks = users + 4
    dl.history_fork(r.cache, users, forks)
    dl.history_append(r.cache, forks, session[1], *r.encode(*session))
    at, where = 0, candidates[0].cpu().numpy()
    for u, n in enumerate(cands):
        x = f64(items)[where[at:at + n]]
        (k, _), (v, _) = cached(r.cache, u + 4)
        q = (x @ f64(r.query).T).reshape(n, 2, 32)
        found, _ = ref.attention(q, k, v, 32 ** -0.5, False, 0, 0)
        y = np.concatenate([x, (x * found.reshape(n, 64)).sum(1, keepdims=True)], 1)
        (w0, b0, _), (w1, b1, _) = r.top
        y = np.maximum(y @ f64(w0).T + f64(b0), 0) @ f64(w1).T + f64(b1)
        np.testing.assert_allclose(p[at:at + n], 1 / (1 + np.exp(-y[:, 0])), atol=1e-4)
        at += n
