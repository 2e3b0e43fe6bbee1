"""Event-history operators on the GPU against a float64 restatement of their
definitions (history_ref.py): page operators and codes bit for bit, attention
within bounds that follow from the arithmetic.

Attention bounds, for outputs that are averages of values of magnitude <= V with
scores of magnitude <= S (in units of the softmax's exponent):
  fp32: queries and weights carry 22 bits, sums fp32: a score errs by at most a
    few 2^-22 S, a weight relatively as much plus 2^-21; S <= 32 here, so the
    output errs by less than 2^-16 V. lse: 2^-17 (1 + |lse|).
  fp16 / bf16 over a cache: weights carry 11 bits, relative error 2^-12 each,
    so at most 2^-11 V in all with the scores' part, and half an ulp of the
    output type, which is finfo.eps / 2 of it.
  bf16 over plain rows, and over a cache on the tensor-core kernel (64 rows a
    request and 4096 in all): weights carry 8 bits, relative error 2^-9 each: with
    the scores' part at most 2^-8 V.
"""
import numpy as np
import pytest

import history_ref as ref

torch = pytest.importorskip("torch")
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    from dlrm_embedding_interaction_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


def half_ulp(dtype):
    return torch.finfo(TYPES[dtype]).eps / 2


def starts_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(int).tolist()


def make(n_pages, n_slots, max_pages, heads, dim, page):
    return (dl.HistoryCache(n_pages, n_slots, max_pages, heads, dim, page_tokens=page),
            ref.Pool(n_pages, n_slots, max_pages, heads, dim, page))


def same_state(cache, pool, codes=True):
    n = int(cache.n_free.item())
    assert n == len(pool.free)
    assert cache.free_pages[:n].tolist() == pool.free
    np.testing.assert_array_equal(cache.table.cpu().numpy(), pool.table)
    np.testing.assert_array_equal(cache.lengths.cpu().numpy(), pool.lengths)
    np.testing.assert_array_equal(cache.refs.cpu().numpy(), pool.refs)
    if codes:
        for side, name in ((0, "k"), (1, "v")):
            got = getattr(cache, name + "_codes").view(torch.uint8).cpu().numpy()
            used = pool.refs > 0
            np.testing.assert_array_equal(f64(getattr(cache, name + "_scales"))[used],
                                          pool.scales[side][used])
            # events past a history's end hold whatever was there before
            for s in range(len(pool.lengths)):
                for j in range(pool.pages(pool.lengths[s])):
                    p, e = pool.table[s, j], min(pool.G, pool.lengths[s] - j * pool.G)
                    if p >= 0:
                        a, b = got[p, :, :e], pool.codes[side][p, :, :e]
                        nan = (a & 0x7f) == 0x7f
                        np.testing.assert_array_equal(nan, (b & 0x7f) == 0x7f)
                        np.testing.assert_array_equal(a[~nan], b[~nan])


def rows(rng, n, heads, dim, dtype, spread=1.0):
    x = rng.standard_normal((n, heads, dim)) * np.exp(spread * rng.standard_normal((n, heads, 1)))
    return torch.from_numpy(x).to(TYPES[dtype]).cuda()


def fill(cache, pool, rng, slots, lens, spread=1.0):
    at = starts_of(lens)
    k, v = (rows(rng, at[-1], pool.codes[0].shape[1], pool.codes[0].shape[3], "fp32", spread)
            for _ in range(2))
    dl.history_append(cache, i32(slots), i32(at), k, v)
    pool.append(slots, at, (f64(k), f64(v)))


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim,page,heads", [(32, 32, 3), (64, 64, 1), (128, 128, 2), (64, 32, 5)])
def test_append_writes_the_defined_codes(dtype, dim, page, heads):
    rng = np.random.default_rng(1)
    cache, pool = make(64, 6, 12, heads, dim, page)
    for counts in ([1, 0, page, 5, 2 * page + 1, 33], [1, 1, 1, 1, 1, 1], [page - 1, 3, 0, page, 1, 40]):
        at = starts_of(counts)
        # values whose size drifts, so that scales grow while a page fills
        k, v = (rows(rng, at[-1], heads, dim, dtype, 2.0) for _ in range(2))
        slots = rng.permutation(6).tolist()
        dl.history_append(cache, i32(slots), i32(at), k, v)
        pool.append(slots, at, (f64(k), f64(v)))
    same_state(cache, pool)
    assert cache.error() == dl.OK


def test_append_one_event_at_a_time_grows_the_scale():
    rng = np.random.default_rng(2)
    cache, pool = make(8, 2, 4, 2, 32, 32)
    for i in range(70):
        x = [rows(rng, 2, 2, 32, "fp32") * 2.0 ** (i % 40 - 20) for _ in range(2)]
        dl.history_append(cache, i32([1, 0]), i32([0, 1, 2]), *x)
        pool.append([1, 0], [0, 1, 2], [f64(t) for t in x])
    same_state(cache, pool)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_append_of_zeros_infinities_nan_and_extremes(dtype):
    cache, pool = make(8, 6, 2, 1, 32, 32)
    big = {"fp32": 3e38, "bf16": 3e38, "fp16": 65504.0}[dtype]
    x = torch.zeros(6, 1, 32, dtype=TYPES[dtype], device="cuda")
    x[1, 0, 0] = float("inf")
    x[1, 0, 1] = -float("inf")
    x[1, 0, 2] = 1.0
    x[2, 0, 3] = float("nan")
    x[2, 0, 4] = 448.0
    x[3, 0, 5] = big
    x[4] = 1e-7 if dtype == "fp16" else 1e-38
    x[5, 0, :4] = torch.tensor([448.0, 0.5, 2.0 ** -10, 464.0], dtype=TYPES[dtype])
    dl.history_append(cache, i32(range(6)), i32(range(7)), x, -x)
    pool.append(list(range(6)), list(range(7)), (f64(x), f64(-x)))
    same_state(cache, pool)


def test_append_reads_strided_and_unaligned_rows():
    rng = np.random.default_rng(3)
    cache, pool = make(16, 2, 4, 3, 64, 64)
    wide = torch.from_numpy(rng.standard_normal((100, 5, 3, 64 + 7)).astype(np.float32)).cuda()
    k = wide[:, 1, :, 3:67]
    v = torch.from_numpy(rng.standard_normal((3, 100, 64))).to(torch.float32).cuda().transpose(0, 1)
    dl.history_append(cache, i32([1, 0]), i32([0, 37, 100]), k, v)
    pool.append([1, 0], [0, 37, 100], (f64(k), f64(v)))
    same_state(cache, pool)
    one = torch.from_numpy(rng.standard_normal((1, 1, 64))).to(torch.float16).cuda().expand(3, 3, 64)
    dl.history_append(cache, i32([0]), i32([0, 3]), one, one)   # stride 0
    pool.append([0], [0, 3], (f64(one), f64(one)))
    same_state(cache, pool)


def test_append_refuses_on_the_device_what_it_cannot_do():
    rng = np.random.default_rng(4)
    cache, pool = make(4, 4, 2, 1, 32, 32)
    k = rows(rng, 80, 1, 32, "fp32")

    def both(slots, at):
        dl.history_append(cache, i32(slots), i32(at), k, k)
        pool.append(slots, at, (f64(k), f64(k)))
        same_state(cache, pool)

    both([0, 9, -1], [0, 5, 10, 15])
    assert cache.error() == dl.ERR_INDEX_OOB
    assert cache.error() == dl.OK
    both([0, 0], [0, 5, 10])
    assert cache.error() == dl.ERR_INVALID_ARG
    both([0, 1, 2], [0, 20, 10, 90])                # decreases; passes the rows
    assert cache.error() == dl.ERR_UNSUPPORTED
    both([1], [0, 65])                              # past max_pages
    assert cache.error() == dl.ERR_INVALID_ARG
    # pool of 4: slot 0 has one page; 1 takes two, 2 would take two, 3 one more
    both([1, 2, 3, 0], [0, 40, 80, 80, 80])
    assert cache.error() == dl.ERR_OOM
    both([3, 0], [0, 0, 3])
    assert cache.error() == dl.OK


# ------------------------------------------------------------------ pages

@pytest.mark.parametrize("seed", range(4))
def test_page_operators_in_any_order(seed):
    """Random calls, errors among them, on a small pool: the state stays that of
    the plain restatement, bit for bit."""
    rng = np.random.default_rng(seed)
    slots = 12
    cache, pool = make(60, slots, 7, 2, 32, 32)
    for step in range(60):
        op = rng.integers(0, 7)
        n = int(rng.integers(1, 6))
        some = rng.integers(0, slots + (step % 9 == 0), n).tolist()
        if op <= 1:
            fill(cache, pool, rng, some, rng.integers(0, 70, n).tolist())
        elif op == 2 or op == 3:
            src = rng.integers(0, slots, n).tolist()
            (dl.history_fork if op == 2 else dl.history_copy)(cache, i32(src), i32(some))
            pool.fork(src, some, op == 2)
        elif op == 4:
            dl.history_free(cache, i32(some))
            pool.release(some)
        elif op == 5:
            w, s = int(rng.integers(1, 90)), int(rng.integers(0, 40))
            dl.history_trim(cache, i32(some), w, s)
            pool.release(some, w, s)
        else:
            dl.history_compact(cache)
            pool.compact()
        same_state(cache, pool, codes=step % 10 == 9)
    same_state(cache, pool)


def test_fork_shares_full_pages_and_copies_the_last():
    rng = np.random.default_rng(7)
    cache, pool = make(40, 10, 4, 2, 64, 64)
    fill(cache, pool, rng, [0, 1, 2], [100, 128, 0])
    dl.history_fork(cache, i32([0, 0, 1, 2, 0]), i32([3, 4, 5, 6, 7]))
    pool.fork([0, 0, 1, 2, 0], [3, 4, 5, 6, 7], True)
    same_state(cache, pool)
    assert cache.refs[cache.table[0, 0]].item() == 4
    fill(cache, pool, rng, [4, 0, 5], [60, 1, 1])   # each side appends on its own
    same_state(cache, pool)
    dl.history_free(cache, i32([0, 3, 7]))
    pool.release([0, 3, 7])
    same_state(cache, pool)
    assert cache.error() == dl.OK
    dl.history_fork(cache, i32([4, 4]), i32([5, 8]))  # 5 is not empty
    pool.fork([4, 4], [5, 8], True)
    assert cache.error() == dl.ERR_INVALID_ARG
    same_state(cache, pool)


@pytest.mark.parametrize("n_pages,users", [(3000, 300), (1024, 64), (1025, 64)])
def test_compact_packs_a_large_pool(n_pages, users):
    rng = np.random.default_rng(8)
    cache, pool = make(n_pages, users, 16, 1, 32, 32)
    lens = rng.integers(1, 32 * min(16, n_pages // users), users).tolist()
    fill(cache, pool, rng, list(range(users)), lens)
    gone = rng.permutation(users)[: users // 2].tolist()
    dl.history_free(cache, i32(gone))
    pool.release(gone)
    for _ in range(2):                              # the second finds nothing to move
        dl.history_compact(cache)
        pool.compact()
        same_state(cache, pool)
    live = int((pool.refs > 0).sum())
    assert pool.refs[:live].all() and not pool.refs[live:].any()


def test_compact_of_an_empty_and_of_a_full_pool():
    rng = np.random.default_rng(9)
    cache, pool = make(6, 3, 2, 1, 32, 32)
    for lens in ([0, 0, 0], [64, 64, 64]):
        fill(cache, pool, rng, [0, 1, 2], lens)
        dl.history_compact(cache)
        pool.compact()
        same_state(cache, pool)


def test_many_requests_in_one_call():
    rng = np.random.default_rng(10)
    n = 2500                                        # more than the plan's threads
    cache, pool = make(6000, 2 * n, 3, 1, 32, 32)
    lens = rng.integers(0, 70, n).tolist()
    order = rng.permutation(n).tolist()
    fill(cache, pool, rng, order, lens)
    dl.history_fork(cache, i32(range(n)), i32(range(n, 2 * n)))
    pool.fork(list(range(n)), list(range(n, 2 * n)), True)
    same_state(cache, pool, codes=False)
    back = rng.permutation(2 * n)[: n].tolist()
    dl.history_free(cache, i32(back))
    pool.release(back)
    same_state(cache, pool, codes=False)


@pytest.mark.parametrize("batch", [1, 31, 64, 127, 128, 129, 200, 1025])
def test_requests_of_any_number_with_refusals_among_them(batch):
    """Forks and appends of a whole batch: slots out of range, slots written twice,
    starts that decrease, occupied destinations and a pool that runs dry part of the way."""
    rng = np.random.default_rng(batch)
    users = 40
    cache, pool = make(users * 4 + batch // 2, users + batch + 5, 4, 2, 32, 32)
    fill(cache, pool, rng, list(range(users)), rng.integers(0, 100, users).tolist())
    src, dst = rng.integers(0, users, batch), users + rng.permutation(batch)
    src[rng.random(batch) < 0.05] = users + batch + 5
    dst[rng.random(batch) < 0.05] = -1
    again = rng.random(batch) < 0.1
    dst[again] = dst[rng.integers(0, batch, batch)][again]
    dst[rng.random(batch) < 0.05] = 3               # not empty, or written twice
    src, dst = src.tolist(), dst.tolist()
    dl.history_fork(cache, i32(src), i32(dst))
    pool.fork(src, dst, True)
    same_state(cache, pool)
    at = starts_of(rng.integers(0, 45, batch))
    at[batch // 2] += 20                            # may pass the next one
    k, v = (rows(rng, max(at[-1], 1), 2, 32, "fp32") for _ in range(2))
    dl.history_append(cache, i32(dst), i32(at), k, v)
    pool.append(dst, at, (f64(k), f64(v)))
    same_state(cache, pool)
    dl.history_free(cache, i32(dst))
    pool.release(dst)
    same_state(cache, pool)


# ------------------------------------------------------------------ attention over a cache

def check_attention(cache, pool, rng, slots, counts, heads, dtype, causal, window, sinks, *,
                    q=None, scale=None, lse=True, out=None):
    """Against the bounds above."""
    at = starts_of(counts)
    dim = pool.codes[0].shape[3]
    if q is None:
        q = rows(rng, at[-1], heads, dim, dtype, 0.3)
    sums = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    got = dl.history_attention(cache, i32(slots), i32(at), q, out, scale=scale, causal=causal,
                               window=window, sinks=sinks, lse=sums)
    scale = dim ** -0.5 if scale is None else scale
    all_rows = at[-1] * (heads // pool.codes[0].shape[1])
    many = all_rows >= 64 * len(slots) and at[-1] * heads >= 4096
    eps = {"fp32": 2.0 ** -16, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8 if many else 2.0 ** -11}[dtype]
    half = half_ulp(dtype)
    for b, s in enumerate(slots):
        k, v = pool.events(s)
        want, sums_want = ref.attention(f64(q[at[b]:at[b + 1]]), k, v, scale, causal, window, sinks)
        have = f64(got[at[b]:at[b + 1]])
        big = np.nanmax(np.abs(v)) if v.size else 0.0
        np.testing.assert_array_equal(np.isnan(have), np.isnan(want))
        ok = ~np.isnan(want) & (np.abs(want) <= torch.finfo(TYPES[dtype]).max)
        bound = eps * big + half * np.abs(want)
        assert (np.abs(have - want)[ok] <= bound[ok]).all(), (b, np.abs(have - want)[ok].max(), big)
        past = np.abs(want) > torch.finfo(TYPES[dtype]).max    # past the output type's range
        assert (np.abs(have[past]) >= torch.finfo(TYPES[dtype]).max).all()
        if lse:
            np.testing.assert_allclose(f64(sums[at[b]:at[b + 1]]), sums_want, rtol=2.0 ** -17,
                                       atol=2.0 ** -17 if dtype == "fp32" else 2.0 ** -15)
    return got


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim,page,kv,group", [(32, 32, 1, 4), (64, 64, 2, 1), (128, 128, 1, 2),
                                               (64, 128, 3, 5), (128, 32, 2, 8)])
@pytest.mark.parametrize("causal,window,sinks", [(False, 0, 0), (True, 0, 0), (True, 40, 3),
                                                 (False, 100, 33), (True, 1, 0)])
def test_attention_over_ragged_histories(dtype, dim, page, kv, group, causal, window, sinks):
    rng = np.random.default_rng(11)
    lens = [0, 1, 31, 32, 33, page, page + 1, 300, 517]
    cache, pool = make(80, len(lens), 17, kv, dim, page)
    fill(cache, pool, rng, list(range(len(lens))), lens)
    slots = rng.permutation(len(lens)).tolist() + [7, 8]
    counts = [1, 3, 0, 2, 1, 7, 1, 5, 1, 40, 1]
    check_attention(cache, pool, rng, slots, counts, kv * group, dtype, causal, window, sinks)
    assert cache.error() == dl.OK


@pytest.mark.parametrize("dtype", list(TYPES))
def test_one_long_history_is_split_and_joined(dtype):
    rng = np.random.default_rng(12)
    cache, pool = make(340, 3, 330, 1, 64, 64)
    fill(cache, pool, rng, [0, 1], [20011, 5])
    for counts in ([1, 1], [2, 0]):
        a = check_attention(cache, pool, rng, [0, 1], counts, 1, dtype, False, 0, 0)
    q = rows(rng, 2, 1, 64, dtype)
    a, b = (dl.history_attention(cache, i32([0, 1]), i32([0, 1, 2]), q) for _ in range(2))
    assert torch.equal(a, b)                        # the order of joining is fixed


def test_candidates_of_several_users():
    rng = np.random.default_rng(13)
    cache, pool = make(64, 4, 16, 2, 64, 64)
    fill(cache, pool, rng, [0, 1, 2, 3], [700, 64, 1, 333])
    for dtype in TYPES:
        check_attention(cache, pool, rng, [2, 0, 3, 1], [9, 130, 77, 200], 4, dtype, False, 0, 0)
        check_attention(cache, pool, rng, [2, 0, 3, 1], [1, 300, 150, 64], 4, dtype, True, 50, 5)


# Enough rows for the tensor-core kernel (bf16, 64 a request and 4096 in all);
# the longest histories are split between CTAs, and 3 heads of a group do not
# divide a tile of 128 rows.
MANY = [(64, 64, 2, 2, [3000, 700, 0, 65], [600, 300, 5, 200]),
        (128, 128, 1, 3, [2500, 40], [900, 500]),
        (32, 32, 1, 4, [1111, 1999, 8], [700, 400, 20])]


@pytest.mark.parametrize("dim,page,kv,group,lens,counts", MANY)
@pytest.mark.parametrize("causal,window,sinks", [(False, 0, 0), (True, 0, 0), (True, 300, 5),
                                                 (False, 100, 33), (True, 1, 0)])
def test_many_candidates(dim, page, kv, group, lens, counts, causal, window, sinks):
    rng = np.random.default_rng(26)
    cache, pool = make(2 + sum(-(-n // page) for n in lens), len(lens), -(-max(lens) // page), kv, dim, page)
    fill(cache, pool, rng, list(range(len(lens))), lens)
    slots = list(range(len(lens)))[::-1]
    a = check_attention(cache, pool, rng, slots, counts[::-1], kv * group, "bf16", causal, window, sinks)
    assert torch.isfinite(a).all() and cache.error() == dl.OK


def test_many_candidates_into_strided_outputs_and_the_same_each_time():
    rng = np.random.default_rng(27)
    cache, pool = make(60, 2, 50, 2, 64, 64)
    fill(cache, pool, rng, [0, 1], [3000, 500])
    out = torch.zeros(8, 700, 70, dtype=torch.bfloat16, device="cuda").transpose(0, 1)[:, :, 3:67]
    q = rows(rng, 700, 8, 64, "bf16", 0.3)
    check_attention(cache, pool, rng, [0, 1], [400, 300], 8, "bf16", False, 0, 0, q=q, out=out)
    # launches one after another, nothing between them
    at = i32([0, 400, 700])
    outs = [dl.history_attention(cache, i32([0, 1]), at, q) for _ in range(100)]
    assert cache.error() == dl.OK
    assert all(torch.equal(x, out) for x in outs)


def test_many_candidates_over_nan_stale_codes_and_trimmed_pages():
    rng = np.random.default_rng(28)
    cache, pool = make(40, 2, 30, 1, 64, 64)
    fill(cache, pool, rng, [0, 1], [1000, 1290])
    for slot, n in ((0, 1000), (1, 1290)):          # codes past the end
        for c in (cache.k_codes, cache.v_codes):
            c.view(torch.uint8)[int(cache.table[slot, n // 64]), :, n % 64:] = 0x7f
    x = rows(rng, 10, 1, 64, "fp32")
    x[4] = float("nan")                             # event 1004 of slot 0
    dl.history_append(cache, i32([0]), i32([0, 10]), x, x)
    pool.append([0], [0, 10], (f64(x), f64(x)))
    q = rows(rng, 1200, 4, 64, "bf16", 0.3)
    got = check_attention(cache, pool, rng, [0, 1], [600, 600], 4, "bf16", True, 0, 0, q=q)
    assert torch.isfinite(got[:594]).all() and torch.isnan(got[594:600]).all() and torch.isfinite(got[600:]).all()
    dl.history_trim(cache, i32([1]), 200, 3)
    assert (cache.table[1] == -1).sum() > 9
    want = dl.history_attention(cache, i32([1]), i32([0, 5]), q[:5], window=200, sinks=3)
    got = dl.history_attention(cache, i32([1]), i32([0, 1200]), q, window=200, sinks=3)
    assert cache.error() == dl.OK
    assert (got[:5].float() - want.float()).abs().max() < 2.0 ** -7 * want.abs().max().item()
    dl.history_attention(cache, i32([1]), i32([0, 1200]), q)   # needs what was trimmed
    assert cache.error() == dl.ERR_INDEX_OOB


def test_scales_that_differ_between_pages_by_millions():
    rng = np.random.default_rng(14)
    cache, pool = make(16, 1, 8, 1, 64, 32)
    for e in (0, 20, -20, 5, -12):
        x = rows(rng, 32, 1, 64, "fp32", 0.2)
        kv = (x * 2.0 ** min(e, 0), x * 2.0 ** e)
        dl.history_append(cache, i32([0]), i32([0, 32]), *kv)
        pool.append([0], [0, 32], [f64(t) for t in kv])
    for dtype in TYPES:
        # the window leaves only the pages of small values
        q = rows(rng, 6, 2, 64, dtype, 0.2)
        got = dl.history_attention(cache, i32([0]), i32([0, 6]), q, window=32)
        k, v = pool.events(0)
        want, _ = ref.attention(f64(q), k, v, 0.125, False, 32, 0)
        assert np.abs(f64(got) - want).max() <= 2.0 ** -9 * np.abs(v[-32:]).max()
        check_attention(cache, pool, rng, [0], [4], 2, dtype, False, 0, 0)


def test_what_masked_events_hold_has_no_influence():
    rng = np.random.default_rng(15)
    cache, pool = make(8, 2, 4, 1, 64, 64)
    fill(cache, pool, rng, [0], [70])
    page = int(cache.table[0, 1])
    for c in (cache.k_codes, cache.v_codes):        # codes past the end: as left by an earlier history
        c.view(torch.uint8)[page, :, 6:] = 0x7f
    for dtype in TYPES:
        check_attention(cache, pool, rng, [0], [3], 2, dtype, True, 0, 0)
    # a NaN event in the middle: rows that see it are NaN, the others are not
    x = rows(rng, 10, 1, 64, "fp32")
    x[4] = float("nan")
    dl.history_append(cache, i32([0]), i32([0, 10]), x, x)
    pool.append([0], [0, 10], (f64(x), f64(x)))
    for dtype in TYPES:
        got = check_attention(cache, pool, rng, [0], [20], 2, dtype, True, 0, 0)
        assert torch.isfinite(got[:14]).all() and torch.isnan(got[14:]).all()
        got = check_attention(cache, pool, rng, [0], [20], 2, dtype, True, 3, 1)
        assert torch.isnan(got[14:17]).all() and torch.isfinite(got[17:]).all()


def test_queries_of_any_size_and_the_scale():
    rng = np.random.default_rng(16)
    cache, pool = make(8, 1, 4, 1, 64, 64)
    fill(cache, pool, rng, [0], [90], spread=0.2)
    for dtype, size in (("fp32", 1e25), ("fp32", 1e-30), ("bf16", 1e25), ("bf16", 1e-30),
                        ("fp16", 1e4), ("fp16", 1e-5)):
        q = rows(rng, 3, 2, 64, dtype, 0.2)
        q = (q.double() * size).to(q.dtype)
        check_attention(cache, pool, rng, [0], [3], 2, dtype, False, 0, 0, q=q, scale=0.1 / size)


def test_strided_queries_and_outputs():
    rng = np.random.default_rng(17)
    cache, pool = make(16, 2, 8, 2, 64, 64)
    fill(cache, pool, rng, [0, 1], [100, 200])
    for dtype in TYPES:
        wide = rows(rng, 9, 4, 64 * 3, dtype)
        q = wide[:, :, 65:129]                      # unaligned
        out = torch.zeros(4, 9, 70, dtype=TYPES[dtype], device="cuda").transpose(0, 1)[:, :, 3:67]
        check_attention(cache, pool, rng, [1, 0], [4, 5], 4, dtype, True, 0, 0, q=q, out=out)
        assert (out[:, :, 0] != 0).all()


def test_attention_reports_bad_requests_and_serves_the_others():
    rng = np.random.default_rng(18)
    cache, pool = make(16, 3, 8, 1, 32, 32)
    fill(cache, pool, rng, [0, 1], [100, 200])
    q = rows(rng, 4, 1, 32, "fp32")
    want = dl.history_attention(cache, i32([0]), i32([0, 1]), q[1:2])
    out = torch.full_like(q, 9.0)
    dl.history_attention(cache, i32([7, 0, 1]), i32([0, 1, 2, 9]), q, out)
    assert cache.error() == dl.ERR_INDEX_OOB
    assert cache.error() == dl.OK
    assert (out[0] == 0).all() and torch.equal(out[1:2], want) and (out[2:] == 9).all()
    dl.history_attention(cache, i32([0, 1]), i32([2, 1, 3]), q, out)
    assert cache.error() == dl.ERR_UNSUPPORTED
    # trimmed pages: the window's queries do not need them, others are told
    dl.history_trim(cache, i32([1]), 40, 4)
    pool.release([1], 40, 4)
    got = dl.history_attention(cache, i32([1]), i32([0, 1]), q[:1], window=40, sinks=4)
    assert cache.error() == dl.OK and torch.isfinite(got).all()
    dl.history_attention(cache, i32([1]), i32([0, 1]), q[:1])
    assert cache.error() == dl.ERR_INDEX_OOB


def test_pages_past_four_gigabytes():
    rng = np.random.default_rng(19)
    heads, dim, page = 8, 128, 128
    n = (1 << 32) // (heads * dim * page) + 40      # the last pages lie past 2^32 bytes
    cache = dl.HistoryCache(n, 2, 4, heads, dim, page_tokens=page)
    pool = ref.Pool(40, 2, 4, heads, dim, page)
    cache.free_pages.copy_(torch.arange(n, dtype=torch.int32, device="cuda"))   # the last page first
    pool.free = list(range(40))
    fill(cache, pool, rng, [0, 1], [300, 129])
    assert cache.table.max().item() == n - 1
    for dtype in TYPES:
        check_attention(cache, pool, rng, [1, 0], [2, 1], 8, dtype, False, 0, 0)
    dl.history_copy(cache, i32([0]), i32([0]))      # into itself: not empty
    assert cache.error() == dl.ERR_INVALID_ARG
    dl.history_free(cache, i32([1]))
    dl.history_copy(cache, i32([0]), i32([1]))
    pool.release([1])
    pool.fork([0], [1], False)
    check_attention(cache, pool, rng, [1], [1], 8, "fp32", False, 0, 0)
    dl.history_compact(cache)
    assert cache.table.max().item() == 5
    check_attention(cache, pool, rng, [0, 1], [1, 1], 8, "fp32", False, 0, 0)


def test_calls_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(20)
    cache, pool = make(64, 6, 8, 2, 64, 64)
    fill(cache, pool, rng, [0, 1, 2], [100, 300, 7])
    k = rows(rng, 3, 2, 64, "bf16")
    q = rows(rng, 3, 4, 64, "bf16")
    src, dst, at = i32([0, 1, 2]), i32([3, 4, 5]), i32([0, 1, 2, 3])
    out = torch.empty_like(q)

    def session(stream=None):
        dl.history_fork(cache, src, dst, stream=stream)
        dl.history_append(cache, dst, at, k, k, stream=stream)
        dl.history_attention(cache, dst, at, q, out, stream=stream)
        dl.history_free(cache, dst, stream=stream)

    session()
    torch.cuda.synchronize()
    want, state = out.clone(), [t.clone() for t in (cache.table, cache.refs, cache.lengths, cache.n_free)]
    side = torch.cuda.Stream()
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    session(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        session()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    for a, b in zip(state, (cache.table, cache.refs, cache.lengths, cache.n_free)):
        assert torch.equal(a, b)
    assert cache.error() == dl.OK


# ------------------------------------------------------------------ attention over plain rows

def check_window(rng, q_counts, k_counts, heads, kv, dim, dtype, window, sinks, *, qkv=None, out=None,
                 scale=None):
    qa, ka = starts_of(q_counts), starts_of(k_counts)
    q, k, v = qkv or (rows(rng, qa[-1], heads, dim, dtype, 0.3), rows(rng, ka[-1], kv, dim, dtype, 0.3),
                      rows(rng, ka[-1], kv, dim, dtype, 0.3))
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = dl.window_attention(q, k, v, i32(qa), out, k_starts=None if qa == ka else i32(ka),
                              window=window, sinks=sinks, lse=lse, err_flag=err, scale=scale)
    assert err.item() == 0
    eps, half = {"fp32": 2.0 ** -16, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype], half_ulp(dtype)
    for b in range(len(q_counts)):
        kb, vb = f64(k[ka[b]:ka[b + 1]]), f64(v[ka[b]:ka[b + 1]])
        want, sums = ref.attention(f64(q[qa[b]:qa[b + 1]]), kb, vb, dim ** -0.5 if scale is None else scale,
                                   True, window, sinks)
        have = f64(got[qa[b]:qa[b + 1]])
        np.testing.assert_array_equal(np.isnan(have), np.isnan(want))
        ok = np.isfinite(want)
        np.testing.assert_array_equal(have[~ok & ~np.isnan(want)], want[~ok & ~np.isnan(want)])
        fin = vb[np.isfinite(vb)]
        big = np.abs(fin).max() if fin.size else 0.0
        bound = eps * big + half * np.abs(want)
        assert (np.abs(have - want)[ok] <= bound[ok]).all(), (b, np.abs(have - want)[ok].max(), big)
        np.testing.assert_allclose(f64(lse[qa[b]:qa[b + 1]]), sums, rtol=2.0 ** -17,
                                   atol=2.0 ** -17 if dtype == "fp32" else 2.0 ** -15)
    return got


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim,kv,group", [(32, 2, 1), (64, 1, 4), (128, 2, 3)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 3), (100, 33), (128, 128), (1000, 7)])
def test_window_attention_of_ragged_histories(dtype, dim, kv, group, window, sinks):
    rng = np.random.default_rng(21)
    counts = [0, 1, 33, 2, 127, 129, 0, 300]
    check_window(rng, counts, counts, kv * group, kv, dim, dtype, window, sinks)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_window_attention_of_the_last_queries(dtype):
    """Fewer queries than keys (a chunk of a history), and more: the first rows see nothing."""
    rng = np.random.default_rng(22)
    for window, sinks in ((0, 0), (50, 4)):
        check_window(rng, [1, 10, 0, 200, 40, 3], [300, 10, 7, 260, 30, 0], 4, 2, 64, dtype, window, sinks)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_window_attention_takes_strides_and_alignments(dtype):
    rng = np.random.default_rng(23)
    n, dim = 150, 64
    wide = rows(rng, n, 8, dim, dtype, 0.3)          # q, k and v in one tensor
    qkv = wide[:, :4], wide[:, 4:6], wide[:, 6:]
    check_window(rng, [n], [n], 4, 2, dim, dtype, 30, 2, qkv=qkv)
    odd = rows(rng, n, 8, dim + 1, dtype, 0.3)[:, :, 1:]
    out = torch.zeros(4, n, dim + 3, dtype=TYPES[dtype], device="cuda").transpose(0, 1)[:, :, 1:dim + 1]
    check_window(rng, [100, 50], [100, 50], 4, 2, dim, dtype, 30, 2,
                 qkv=(odd[:, :4], odd[:, 4:6], odd[:, 6:]), out=out)
    shared = rows(rng, n, 1, dim, dtype, 0.3).expand(n, 2, dim)   # one head for both
    check_window(rng, [n], [n], 4, 2, dim, dtype, 0, 0, qkv=(qkv[0], shared, shared))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_window_attention_keeps_masked_infinities_out(dtype):
    rng = np.random.default_rng(24)
    n = 200
    q, k, v = (rows(rng, n, 2, 64, dtype, 0.3) for _ in range(3))
    v[150, 0, 5] = float("inf")
    v[60, 1, 7] = float("nan")
    k[100, 1] = float("nan")
    got = check_window(rng, [120, 80], [120, 80], 2, 2, 64, dtype, 20, 2, qkv=(q, k, v))
    assert torch.isfinite(got[:60]).all() and torch.isfinite(got[80:100]).all()
    assert torch.isinf(got[150:170, 0, 5]).all() and torch.isfinite(got[170:]).all()


@pytest.mark.parametrize("dim", [32, 64, 128])
def test_window_attention_launches_one_after_another(dim):
    """Many launches with nothing between them, on units of one key tile and of many."""
    rng = np.random.default_rng(29)
    counts = [1, 700, 64, 3, 1500, 65, 128, 0, 260]
    n = sum(counts)
    q, k, v = (rows(rng, n, h, dim, "bf16", 0.3) for h in (4, 2, 2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = i32(starts_of(counts))
    for window in (0, 100):
        want = check_window(rng, counts, counts, 4, 2, dim, "bf16", window, 3, qkv=(q, k, v))
        outs = [dl.window_attention(q, k, v, at, window=window, sinks=3, err_flag=err) for _ in range(100)]
        assert err.item() == 0
        assert all(torch.equal(x, want) for x in outs)


def test_window_attention_flags_bad_starts():
    rng = np.random.default_rng(25)
    q = rows(rng, 10, 1, 32, "fp32")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 9.0)
    dl.window_attention(q, q, q, i32([0, 4, 3, 12]), out, err_flag=err)
    assert err.item() == dl.ERRBIT_OFFSETS
    assert torch.isfinite(out[:4]).all() and (out[:4] != 9).all() and (out[4:] == 9).all()
    empty = torch.empty(0, 1, 32, device="cuda")
    assert dl.window_attention(empty, empty, empty, i32([0, 0])).shape == (0, 1, 32)
    assert (dl.window_attention(q, empty, empty, i32([0, 10]), k_starts=i32([0, 0])) == 0).all()
