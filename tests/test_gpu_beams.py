"""The beam search's operators on the GPU against a float64 restatement of their definitions
(beam_ref.py): pages bit for bit, attention and selection within bounds that follow from
the arithmetic.

Attention with a shared prefix has history_attention's arithmetic and bounds (outputs are
averages of values of magnitude <= V): queries and weights of 22 bits in fp32, errors below
2^-16 V; weights of 11 bits in fp16 and bf16, below 2^-11 V with the scores' part, and half an
ulp of the output type, finfo.eps / 2 of it. lse: 2^-17 (1 + |lse|).

Selection: a term of a row's sum of exponentials errs by 2^-22 of itself (the instruction) and
by the rounding of its argument, at most 2^-24 log2(e) |logit - largest| of itself; weighed by
the terms that is at most 2^-24 log2(e) (1 + ln vocab) on average, below 2^-20 in all for a
vocabulary of 2^20. The score is then rounded to fp32: half an ulp, 2^-24 of it.
"""
import numpy as np
import pytest

import beam_ref
import history_ref as ref

torch = pytest.importorskip("torch")
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402
from test_gpu_history import TYPES, f64, half_ulp, i32, rows, same_state, starts_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    from dlrm_embedding_interaction_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def make(n_pages, n_slots, max_pages, heads, dim, page):
    return (dl.HistoryCache(n_pages, n_slots, max_pages, heads, dim, page_tokens=page),
            beam_ref.Pool(n_pages, n_slots, max_pages, heads, dim, page))


def append(cache, pool, rng, slots, counts, spread=0.5):
    at = starts_of(counts)
    heads, dim = pool.codes[0].shape[1], pool.codes[0].shape[3]
    k, v = (rows(rng, at[-1], heads, dim, "fp32", spread) for _ in range(2))
    dl.history_append(cache, i32(slots), i32(at), k, v)
    pool.append(slots, at, (f64(k), f64(v)))


SHARED = 1 << 27                                  # bytes a side that make every call large enough to share


def beams(rng, lens, counts, new, kv, dim, page, spread=0.5, spare=0, shared=True, idle=0):
    """Users' histories in the first slots, and their beams, forks with events of their
    own, in the following ones, user by user: cache, restatement, the beams' slots, groups.
    shared: tables with room for so many events that no call passes as a small one."""
    users, n = len(lens), sum(counts)
    src = [u for u, c in enumerate(counts) for _ in range(c)]
    slots = list(range(users, users + n))
    most = max(-(-(x + max(new, default=0)) // page) for x in lens) + 1
    if shared:
        most = max(most, SHARED // (n * kv * dim * page) + 1)
    total = sum(-(-x // page) for x in lens) + sum(2 + x // page for x in new) + spare
    cache, pool = make(total + 1, users + n + 1 + idle, most, kv, dim, page)
    append(cache, pool, rng, list(range(users)), lens, spread)
    dl.history_fork(cache, i32(src), i32(slots))
    pool.fork(src, slots, True)
    append(cache, pool, rng, slots, new, spread)
    return cache, pool, slots, starts_of(counts)


def check_rows(pool, slots, at, q, out, lse, dtype, *, scale=None, causal=False, window=0, sinks=0):
    """Rows of each request against the definition."""
    q, out, lse = f64(q), f64(out), None if lse is None else f64(lse)
    scale = q.shape[2] ** -0.5 if scale is None else scale
    for b, s in enumerate(slots):
        a, e = at[b], at[b + 1]
        if a == e:
            continue
        k, v = pool.events(s) if 0 <= s < len(pool.lengths) else (np.zeros((0, 1, q.shape[2])),) * 2
        want, want_lse = ref.attention(q[a:e], k, v, scale, causal, window, sinks)
        big = np.abs(v[np.isfinite(v)]).max(initial=0.0)   # of the events that any row can see
        tol = 2.0 ** (-16 if dtype == "fp32" else -11) * big + half_ulp(dtype) * np.abs(want)
        assert (np.abs(out[a:e] - want) <= tol + 1e-30).all(), (b, np.abs(out[a:e] - want).max(), big)
        if lse is not None:
            seen = np.isfinite(want_lse)
            np.testing.assert_array_equal(seen, np.isfinite(lse[a:e]))
            err = np.abs(lse[a:e][seen] - want_lse[seen])
            assert (err <= 2.0 ** -17 * (1 + np.abs(want_lse[seen]))).all()


# ------------------------------------------------------------------ attention with a shared prefix

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim,page,kv,group", [(32, 32, 3, 1), (64, 64, 2, 4), (128, 128, 1, 2), (64, 32, 1, 5),
                                               (128, 32, 2, 1), (32, 128, 1, 8)])
@pytest.mark.parametrize("causal,window,sinks", [(False, 0, 0), (True, 0, 0), (True, 70, 3), (False, 33, 40)])
@pytest.mark.parametrize("shared", [True, False])
def test_beams_of_ragged_histories(dtype, dim, page, kv, group, causal, window, sinks, shared):
    rng = np.random.default_rng(dim + page + kv + group + window)
    lens = [1, 0, page, 3 * page + 5, 700, 2 * page - 1]
    counts = [3, 2, 1, 9, 20, 4]
    n = sum(counts)
    new = [int(x) for x in rng.integers(0, 2 * page, n)]
    new[0] = new[4] = 0
    # (a window bounds what a call reads: there, requests without rows make it a large one)
    more = 3000 // kv if shared and window else 0
    cache, pool, slots, groups = beams(rng, lens, counts, new, kv, dim, page, shared=shared, idle=more)
    queries = [int(x) for x in rng.integers(0, 4, n)] + [0] * more
    slots, groups = slots + [0] * more, groups + [n + more]
    at = starts_of(queries)
    q = rows(rng, at[-1], kv * group, dim, dtype, 0.3)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = dl.history_prefix_attention(cache, i32(slots), i32(at), i32(groups), q, causal=causal, window=window,
                                      sinks=sinks, lse=lse)
    check_rows(pool, slots, at, q, out, lse, dtype, causal=causal, window=window, sinks=sinks)
    assert cache.error() == dl.OK


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("cut", ["each", "one", "users", "odd"])
def test_the_result_is_the_same_whatever_the_groups(dtype, dim, cut):
    rng = np.random.default_rng(5)
    counts = [4, 7, 1, 12]
    cache, pool, slots, groups = beams(rng, [300, 1000, 64, 129], counts, [3] * 24, 2, dim, 64)
    order = rng.permutation(24) if cut == "odd" else np.arange(24)
    slots = [slots[i] for i in order]
    groups = {"each": list(range(25)), "one": [0, 24], "users": groups, "odd": [0, 0, 5, 6, 6, 20, 24, 24]}[cut]
    at = list(range(25))
    q = rows(rng, 24, 4, dim, dtype, 0.3)
    out = dl.history_prefix_attention(cache, i32(slots), i32(at), i32(groups), q)
    check_rows(pool, slots, at, q, out, None, dtype)
    again = dl.history_prefix_attention(cache, i32(slots), i32(at), i32(groups), q)
    assert torch.equal(out, again)
    assert cache.error() == dl.OK


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("counts,queries", [([1], 1), ([2], 40), ([64], 1), ([130], 1), ([3, 1, 100], 2)])
def test_long_histories_are_cut_and_joined(dtype, counts, queries):
    rng = np.random.default_rng(6)
    n = sum(counts)
    lens = [9000, 40, 5000][:len(counts)]
    cache, pool, slots, groups = beams(rng, lens, counts, [1] * n, 1, 64, 64)
    at = starts_of([queries] * n)
    q = rows(rng, at[-1], 3, 64, dtype, 0.3)
    lse = torch.empty(q.shape[:2], device="cuda")
    out = dl.history_prefix_attention(cache, i32(slots), i32(at), i32(groups), q, lse=lse)
    few = range(0, n, max(1, n // 8))
    for b in few:
        check_rows(pool, [slots[b]], [0, queries], q[at[b]:at[b + 1]], out[at[b]:at[b + 1]], lse[at[b]:at[b + 1]], dtype)
    assert cache.error() == dl.OK


# ------------------------------------------------------------------ reordering

@pytest.mark.parametrize("page,dim,kv", [(32, 32, 1), (64, 64, 3), (128, 128, 2)])
def test_slots_take_over_their_parents_histories(page, dim, kv):
    rng = np.random.default_rng(8)
    counts = [5, 1, 8, 3]
    n = sum(counts)
    new = [int(x) for x in rng.integers(0, 3 * page, n)]
    cache, pool, slots, groups = beams(rng, [100, 7, 5 * page, 2 * page + 1], counts, new, kv, dim, page, spare=40)
    for step in range(6):
        parents = [int(groups[g] + rng.integers(0, counts[g])) for g in range(4) for _ in range(counts[g])]
        if step == 2:
            parents[3], parents[7] = -1, -1
        if step == 4:
            parents = list(range(n))
        dl.history_reorder(cache, i32(slots), i32(parents))
        assert pool.reorder(slots, parents)
        same_state(cache, pool)
        append(cache, pool, rng, slots, [int(x) for x in rng.integers(0, 3, n)])
        same_state(cache, pool)
    assert cache.error() == dl.OK
    dl.history_free(cache, i32(slots))
    pool.release(slots)
    same_state(cache, pool)


# ------------------------------------------------------------------ selection

def check_select(logits, scores, starts, width, allowed, got):
    best, parents, tokens = (x.cpu().numpy() for x in got)
    x = f64(logits)
    s = np.zeros(len(x)) if scores is None else f64(scores)
    want, want_rows, want_tokens, every = beam_ref.select(x, s, starts, width,
                                                          None if allowed is None else allowed.cpu().numpy())
    there = want > -np.inf
    np.testing.assert_array_equal(best > -np.inf, there)
    np.testing.assert_array_equal(parents[~there], -1)
    np.testing.assert_array_equal(tokens[~there], -1)
    tol = 2.0 ** -20 + 2.0 ** -24 * np.abs(want[there])
    assert (np.abs(best[there] - want[there]) <= tol).all()
    # each candidate once, of its group, in its place but for scores that lie together
    for g in range(len(starts) - 1):
        m = int(there[g].sum())
        pairs = list(zip(parents[g, :m].tolist(), tokens[g, :m].tolist()))
        assert len(set(pairs)) == m
        for i, (r, t) in enumerate(pairs):
            assert starts[g] <= r < starts[g + 1] and 0 <= t < x.shape[1]
            assert abs(every[r, t] - want[g, i]) <= 2.0 ** -19, (g, i)
            if (r, t) != (want_rows[g, i], want_tokens[g, i]):
                assert r != want_rows[g, i]                   # within a row the order is exact
    return parents, tokens


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab,width", [(1, 1), (2, 3), (37, 5), (256, 32), (1000, 256), (4096, 7), (4097, 64),
                                         (8191, 65), (8192, 1), (8193, 256), (50021, 100)])
@pytest.mark.parametrize("keep", [0, 3, 50])
def test_the_best_continuations(dtype, vocab, width, keep):
    rng = np.random.default_rng(vocab + width)
    starts = [0, 3, 3, 4, 11]
    logits = torch.from_numpy(2.0 * rng.standard_normal((11, vocab))).to(TYPES[dtype]).cuda()
    scores = torch.from_numpy(-5.0 * rng.random(11)).float().cuda()
    scores[1] = -float("inf")
    allowed = None
    if keep:
        allowed = torch.from_numpy(rng.random((11, vocab)) < 1.0 / keep).cuda()
        allowed[5] = False
        logits[~allowed] = torch.tensor([float("nan"), float("inf"), 99.0], device="cuda").to(TYPES[dtype])[
            torch.randint(3, (int((~allowed).sum()),), device="cuda")]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = dl.beam_select(logits, scores, i32(starts), width, allowed=allowed, err_flag=err)
    check_select(logits, scores, starts, width, allowed, got)
    assert int(err) == 0
    again = dl.beam_select(logits, scores, i32(starts), width, allowed=allowed)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [200, 4999, 40000])
@pytest.mark.parametrize("kind", ["equal", "two values", "rising", "falling", "few peaks"])
def test_ties_and_adverse_orders(dtype, vocab, kind):
    """Ties go by row, then token; orders in which every logit passes the bound so far."""
    x = torch.arange(vocab, dtype=torch.float64)
    x = {"equal": 0 * x + 1.5, "two values": (x % 2), "rising": x / vocab, "falling": -x / vocab,
         "few peaks": 50.0 * (x % 997 == 3)}[kind]
    logits = x.to(TYPES[dtype]).cuda().repeat(5, 1)
    starts, width = [0, 2, 5], 100
    got = dl.beam_select(logits, None, i32(starts), width)
    best, parents, tokens, _ = beam_ref.select(f64(logits), np.zeros(5), starts, width)
    # rows are alike bit for bit, so equal scores are equal
    np.testing.assert_array_equal(got[1].cpu().numpy(), parents)
    np.testing.assert_array_equal(got[2].cpu().numpy(), tokens)
    check_select(logits, None, starts, width, None, got)
