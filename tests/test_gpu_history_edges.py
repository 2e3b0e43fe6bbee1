"""Event-history operators on the GPU at the edges of their definitions: what a refused
request leaves behind, the largest windows, empty and infinite scores, layouts and
streams, and waits that run out. Bounds as in test_gpu_history.py."""
import numpy as np
import pytest

import history_ref as ref
import test_gpu_history as base

torch = pytest.importorskip("torch")
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402

pytestmark = pytest.mark.gpu
i32, f64, rows, make, fill, same_state, starts_of = (
    base.i32, base.f64, base.rows, base.make, base.fill, base.same_state, base.starts_of)
TYPES = base.TYPES


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    from dlrm_embedding_interaction_gb300 import build
    build.build()
    torch.cuda.set_device(0)


# ------------------------------------------------------------------ refused requests

def test_a_refused_copy_leaves_nothing_behind():
    rng = np.random.default_rng(40)
    cache, pool = make(32, 8, 3, 2, 32, 32)
    fill(cache, pool, rng, [0, 1], [40, 70])

    def copy(src, dst):
        dl.history_copy(cache, i32(src), i32(dst))
        pool.fork(src, dst, False)
        same_state(cache, pool)

    copy([8], [5])                                  # no such source
    assert cache.error() == dl.ERR_INDEX_OOB
    copy([0, 1], [4, 5])                            # slot 5 at a higher index than before
    assert cache.error() == dl.OK
    copy([-1, 0, 9], [6, 6, 7])                     # 6 is written twice: the first counts, and is refused
    assert cache.error() == dl.ERR_INDEX_OOB
    copy([0, 1, 0], [2, 7, 6])
    assert cache.error() == dl.OK


@pytest.mark.parametrize("batch", [129, 1500])
def test_a_refused_fork_of_many_leaves_nothing_behind(batch):
    """Sources out of range in a fork of many requests, then appends, copies and forks
    whose slots stand at other indices."""
    rng = np.random.default_rng(batch)
    cache, pool = make(4 * batch, 2 * batch, 2, 1, 32, 32)
    fill(cache, pool, rng, [0, 1], [40, 20])
    src = np.where(rng.random(batch) < 0.5, 0, 2 * batch).tolist()
    dst = (2 + np.arange(batch)).tolist()
    dl.history_fork(cache, i32(src), i32(dst))
    pool.fork(src, dst, True)
    assert cache.error() == dl.ERR_INDEX_OOB
    dl.history_free(cache, i32(dst))
    pool.release(dst)
    same_state(cache, pool, codes=False)
    # every slot at a higher index than before, but the first
    dst = dst[-1:] + dst[:-1]
    for step in range(3):
        if step == 0:
            fill(cache, pool, rng, dst, [1] * batch)
        else:
            (dl.history_copy if step == 1 else dl.history_fork)(cache, i32([1] * batch), i32(dst))
            pool.fork([1] * batch, dst, step == 2)
        same_state(cache, pool)
        assert cache.error() == dl.OK
        dl.history_free(cache, i32(dst))
        pool.release(dst)


@pytest.mark.parametrize("page", [64, 2 ** 31 - 1, -2])
def test_pages_that_a_table_cannot_hold_are_left_alone(page):
    """A table that names a page outside the pool: such an entry is no page to any call."""
    rng = np.random.default_rng(50)
    cache, pool = make(64, 300, 4, 1, 32, 32)
    fill(cache, pool, rng, [0, 1], [100, 40])
    cache.table[0, 1] = page
    dl.history_copy(cache, i32([0, 1]), i32([2, 3]))
    dl.history_fork(cache, i32([0, 1]), i32([4, 5]))
    dl.history_fork(cache, i32([0] * 200), i32(range(6, 206)))
    assert cache.error() == dl.ERR_OOM              # of the last call's pages
    assert cache.lengths[:7].tolist() == [100, 40, 100, 40, 100, 40, 100]
    assert cache.table[2, 1] == -1 and (cache.table[2, [0, 2, 3]] >= 0).all()
    assert cache.table[4, 1] == page
    q = rows(rng, 2, 1, 32, "fp32")
    got = dl.history_attention(cache, i32([1, 3, 5]), i32([0, 2, 2, 2]), q)
    assert cache.error() == dl.OK and torch.isfinite(got).all()
    dl.history_attention(cache, i32([4]), i32([0, 2]), q)
    assert cache.error() == dl.ERR_INDEX_OOB
    dl.history_free(cache, i32(range(0, 206)))
    assert int(cache.n_free) == 63                  # all but the one that the table lost
    assert cache.error() == dl.OK


def test_a_fork_of_a_page_of_half_a_gigabyte():
    """More pieces to copy than a grid has rows."""
    heads = 32768
    cache = dl.HistoryCache(3, 3, 1, heads, 128, page_tokens=128)
    k, v = (torch.randn(5, heads, 128, device="cuda", dtype=torch.float16) for _ in range(2))
    dl.history_append(cache, i32([0]), i32([0, 5]), k, v)
    dl.history_fork(cache, i32([0]), i32([2]))
    assert cache.error() == dl.OK and cache.lengths.tolist() == [5, 0, 5]
    a, b = (int(cache.table[s, 0]) for s in (0, 2))
    assert a != b
    for x in (cache.k_codes, cache.v_codes):
        assert torch.equal(x[a].view(torch.uint8), x[b].view(torch.uint8))
        assert x[b, :, :5].float().abs().amax(dim=(1, 2)).min() > 0
    for x in (cache.k_scales, cache.v_scales):
        assert torch.equal(x[a], x[b])


# ------------------------------------------------------------------ windows

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 40])
def test_the_largest_window_with_more_queries_than_events(dtype, dim, window):
    """The first rows stand before the first event: such a window's start lies below -2^31."""
    rng = np.random.default_rng(41)
    for counts, lens in (([4, 70, 300], [1, 20, 150]), ([33], [1])):
        for sinks in (0, 2, 2 ** 31 - 1):
            base.check_window(rng, counts, lens, 4, 2, dim, dtype, window, sinks)
    lens, counts = [1, 20, 150, 700], [4, 70, 300, 710]
    cache, pool = make(20, 4, 11, 2, dim, 64)
    fill(cache, pool, rng, [0, 1, 2, 3], lens)
    for n in (1, 3, 4):                             # the last: enough rows for the tensor-core kernel
        base.check_attention(cache, pool, rng, list(range(n)), counts[:n], 4, dtype, True, window, 1)
    assert cache.error() == dl.OK


# ------------------------------------------------------------------ scores and weights

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim,n", [(32, 3), (64, 40), (64, 700), (128, 300)])
def test_scores_of_minus_infinity_are_no_empty_rows(dtype, dim, n):
    """A row all of whose visible scores are -infinity is 0 / 0, as its definition says, not
    zeros like a row that sees nothing; with other events beside them they weigh nothing."""
    rng = np.random.default_rng(42)
    q, k, v = (rows(rng, n, h, dim, dtype, 0.3) for h in (4, 2, 2))
    q[:, :, 3] = q[:, :, 3].abs() + 0.5
    k[0, :, 3] = -float("inf")                      # what the first row sees
    k[1, 0, 3] = -float("inf")
    want, _ = ref.attention(f64(q), f64(k), f64(v), dim ** -0.5, True, 0, 0)
    assert np.isnan(want[0]).all() and np.isnan(want[1, :2]).all() and np.isfinite(want[2:]).all()
    lse = torch.empty(n, 4, device="cuda")
    got = dl.window_attention(q, k, v, i32([0, n]), lse=lse)
    np.testing.assert_array_equal(np.isnan(f64(got)), np.isnan(want))
    assert (lse[0] == -float("inf")).all() and (lse[1, :2] == -float("inf")).all()
    assert torch.isfinite(lse[1, 2:]).all() and torch.isfinite(lse[2:]).all()
    eps = {"fp32": 2.0 ** -16, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    bound = eps * np.abs(f64(v)).max() + base.half_ulp(dtype) * np.abs(want[2:])
    assert (np.abs(f64(got)[2:] - want[2:]) <= bound).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("count", [1, 2100])
def test_infinite_queries_over_a_cache(dtype, count):
    """Codes hold no infinities, queries may: scores are then infinite of either sign, and NaN
    where the code is zero."""
    rng = np.random.default_rng(43)
    cache, pool = make(8, 2, 4, 2, 64, 64)
    one = torch.ones(5, 2, 64, device="cuda")
    dl.history_append(cache, i32([0]), i32([0, 5]), one, one)
    pool.append([0], [0, 5], (f64(one), f64(one)))
    q = rows(rng, count, 4, 64, dtype, 0.3)
    q[0, :, 7] = -float("inf")
    q[count // 2, 1, 9] = float("inf")
    k, v = pool.events(0)
    want, _ = ref.attention(f64(q), k, v, 0.125, False, 0, 0)
    assert np.isnan(want[0]).all() and np.isnan(want[count // 2, 1]).all()
    got = dl.history_attention(cache, i32([0]), i32([0, count]), q)
    np.testing.assert_array_equal(np.isnan(f64(got)), np.isnan(want))


@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("n", [300, 4096, 16384, 65000])
@pytest.mark.parametrize("window,sinks", [(0, 0), (3000, 500)])
def test_sums_of_fp32_over_many_events(dim, n, window, sinks):
    """Values of one sign, where errors that point the same way add up: the output stays
    within 2^-16 of them, however many events it sums."""
    rng = np.random.default_rng(44)
    q = rows(rng, 70, 2, dim, "fp32", 0.3)
    k = rows(rng, n, 1, dim, "fp32", 0.3)
    v = torch.from_numpy(rng.random((n, 1, dim)) + 1.0).float().cuda()
    for rows_of in (1, 70):
        x = q[:rows_of]
        lse = torch.empty(rows_of, 2, device="cuda")
        got = dl.window_attention(x, k, v, i32([0, rows_of]), k_starts=i32([0, n]), window=window, sinks=sinks,
                                  lse=lse)
        pos = torch.arange(n - rows_of, n, device="cuda")[:, None]
        t = torch.arange(n, device="cuda")[None]
        see = (t <= pos) & ((t > pos - window) | (t < sinks) if window else t >= 0)
        s = torch.einsum("ihd,td->hit", x.double(), k[:, 0].double()) * dim ** -0.5
        s = s.masked_fill(~see, -float("inf"))
        want = torch.einsum("hit,td->ihd", s.softmax(-1), v[:, 0].double())
        assert (got.double() - want).abs().max().item() <= 2.0 ** -16 * 2.0
        sums = s.logsumexp(-1).T
        assert ((lse.double() - sums).abs() <= 2.0 ** -17 * (1 + sums.abs())).all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_many_small_weights_beside_a_large_one(dtype):
    """One event outweighs each of 65,000 others by 2^25.2, yet together they have 0.16% of
    the weight. Values are 0 for the one and 1 for the others, so the output is their share."""
    n, dim = 65000, 64
    for plain in (False, True):
        k, v = torch.zeros(n, 1, dim, device="cuda"), torch.ones(n, 1, dim, device="cuda")
        k[0, 0, 0], v[0] = 1.0, 0.0
        q = torch.zeros(1 if not plain else 40, 1, dim, device="cuda")
        q[:, 0, 0] = 17.5
        rest = (n - 1 - (np.arange(len(q))[::-1] if plain else np.zeros(1))) * np.exp(-17.5)
        want = rest / (1 + rest)
        if plain:
            q, k, v = (t.to(TYPES[dtype]) for t in (q, k, v))
            outs = [dl.window_attention(q[-c:], k, v, i32([0, c]), k_starts=i32([0, n]), scale=1.0)
                    for c in (1, 40)]               # up to head_dim 64 the number of rows picks the kernel
        else:
            cache = dl.HistoryCache(1100, 1, 1100, 1, dim)
            dl.history_append(cache, i32([0]), i32([0, n]), k, v)
            q = q.to(TYPES[dtype])
            outs = [dl.history_attention(cache, i32([0]), i32([0, len(x)]), x, scale=1.0)
                    for x in (q, q.expand(4200, 1, dim))]
        # every weight is off by at most its rounding (2^-22, 2^-12 or 2^-9 of it, as the type
        # of the weights may be), and so is their sum; and half an ulp of the output
        eps = {"fp32": 2.0 ** -16, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
        for out in outs:
            share = want[-len(out):] if plain else want
            err = np.abs(f64(out)[:, 0] - share[:, None])
            assert (err <= (eps + base.half_ulp(dtype)) * share[:, None]).all(), (plain, len(out), err.max())


# ------------------------------------------------------------------ streams

def test_a_call_on_another_stream_while_the_current_one_is_busy():
    """The cache, and an output that the call makes, belong to the call's stream: nothing that
    is still queued on the current one (a fill of freed memory too) reaches them."""
    rng = np.random.default_rng(49)
    side = torch.cuda.Stream()
    k = rows(rng, 200, 2, 64, "fp32")
    q = rows(rng, 5000, 4, 64, "fp32")
    plain = rows(rng, 5000, 4, 64, "bf16", 0.3)
    slots, at, q_at = i32([0]), i32([0, 200]), i32([0, 5000])
    want = dl.window_attention(plain, plain, plain, q_at)
    pool = ref.Pool(8, 2, 4, 2, 64, 64)
    pool.append([0], [0, 200], (f64(k), f64(k)))
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    freed = [torch.empty_like(x) for x in (q, plain)]
    torch.cuda._sleep(200_000_000)                  # a tenth of a second
    for x in freed:
        x.fill_(7.0)
    del freed, x
    cache = dl.HistoryCache(8, 2, 4, 2, 64, stream=side)
    dl.history_append(cache, slots, at, k, k, stream=side)
    out = dl.history_attention(cache, slots, q_at, q, stream=side)
    enc = dl.window_attention(plain, plain, plain, q_at, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    same_state(cache, pool)
    assert cache.error(side) == dl.OK
    assert torch.equal(enc, want)
    assert torch.equal(out, dl.history_attention(cache, slots, q_at, q))


def test_streams_by_their_handles():
    """A raw cudaStream_t: a stream's own, and the legacy and per-thread default streams'."""
    rng = np.random.default_rng(52)
    k = rows(rng, 40, 2, 64, "fp32")
    want = dl.window_attention(k, k, k, i32([0, 40]))
    at, one = i32([0, 40]), i32([0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for stream in (0, 1, 2, side.cuda_stream, side):
        cache = dl.HistoryCache(4, 2, 2, 2, 64, stream=stream)
        dl.history_append(cache, one, at, k, k, stream=stream)
        torch.cuda.synchronize()
        outs.append(dl.history_attention(cache, one, at, k, causal=True, stream=stream))
        got = dl.window_attention(k, k, k, at, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert cache.error(stream) == dl.OK
    assert all(torch.equal(x, outs[0]) for x in outs)


# ------------------------------------------------------------------ starts

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n", [1 << 20, 1 << 13])
def test_starts_that_claim_all_rows_many_times_over(dtype, n):
    """Every second request decreases and is refused, the others have all rows each. The
    longer rows make more work in all than 31 bits count. Over a cache such a call does
    nothing but say so, over plain rows no more than its rows are; the next is as ever."""
    rng = np.random.default_rng(48)
    cache, pool = make(70, 2, 65, 8, 32, 64)
    fill(cache, pool, rng, [0, 1], [4096, 100])
    batch = min(4096, n // 100)
    at = i32([0, n] * (batch // 2) + [0])
    q = rows(rng, 1, 8, 32, dtype).expand(n, 8, 32)
    out = torch.full((n, 8, 32), 9.0, dtype=TYPES[dtype], device="cuda")
    dl.history_attention(cache, i32([0] * (len(at) - 1)), at, q, out)
    assert cache.error() == dl.ERR_UNSUPPORTED
    assert (out == 9).all()
    base.check_attention(cache, pool, rng, [1, 0], [3, 2], 8, dtype, False, 0, 0)
    assert cache.error() == dl.OK
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = q.contiguous()
    dl.window_attention(q, q, q, at, out, window=64, err_flag=err)
    assert err.item() == dl.ERRBIT_OFFSETS


# ------------------------------------------------------------------ waits that run out

LIMIT_NS = 2_000_000      # 2 ms: far above any wait of a healthy call here


def stalled(call, error):
    """call(), with a piece of its work withheld: TIMEOUT after the limit, not the default's 2 s."""
    import time
    dl.attention_test_stall(LIMIT_NS, False)
    call()
    assert error() == dl.OK
    dl.attention_test_stall(LIMIT_NS, True)
    try:
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        call()
        status = error()                            # waits for the GPU
        elapsed = time.perf_counter() - t0
    finally:
        dl.attention_test_stall()
    assert status == dl.ERR_TIMEOUT
    assert elapsed < 0.5, elapsed


@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("counts", [[700], [40, 300, 5000, 64, 1000]])
def test_a_wait_of_window_attention_that_runs_out_reports_timeout(dim, counts):
    rng = np.random.default_rng(45)
    n = sum(counts)
    q, k, v = (rows(rng, n, h, dim, "bf16", 0.3) for h in (4, 2, 2))
    at, err = i32(starts_of(counts)), torch.zeros(1, dtype=torch.int32, device="cuda")
    want = dl.window_attention(q, k, v, at, window=300, sinks=3)

    def error():
        bits = err.item()
        err.zero_()
        return dl.ERR_TIMEOUT if bits == 1 << dl.ERR_TIMEOUT else bits

    stalled(lambda: dl.window_attention(q, k, v, at, window=300, sinks=3, err_flag=err), error)
    for _ in range(3):
        assert torch.equal(dl.window_attention(q, k, v, at, window=300, sinks=3, err_flag=err), want)
    assert err.item() == 0


@pytest.mark.parametrize("dim", [32, 64, 128])
def test_window_attention_that_gives_up_in_the_middle(dim):
    """A limit shorter than what its roles wait for one another in a long call: every CTA
    gives up with copies in flight, and calls after it are as ever."""
    rng = np.random.default_rng(46)
    n = 16384                                       # more units a CTA than it knows ahead
    q, k, v = (rows(rng, 3 * n, 8, dim, "bf16", 0.3) for _ in range(3))
    at, err = i32([0, n, 2 * n, 3 * n]), torch.zeros(1, dtype=torch.int32, device="cuda")
    want = dl.window_attention(q, k, v, at)
    for limit in (20_000, 50_000, 100_000):
        dl.attention_test_stall(limit)
        try:
            dl.window_attention(q, k, v, at, err_flag=err)
            assert err.item() == 1 << dl.ERR_TIMEOUT
        finally:
            dl.attention_test_stall()
        err.zero_()
        assert torch.equal(dl.window_attention(q, k, v, at, err_flag=err), want)
        assert err.item() == 0


@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("lens,counts", [([6000], [2100]), ([3000, 64, 5000, 900], [700, 1000, 500, 300])])
def test_a_cache_is_as_ever_after_a_wait_that_ran_out(dim, lens, counts):
    """Units that CTAs share: those that did their part must not count for the next call."""
    rng = np.random.default_rng(47)
    cache, pool = make(2 + sum(-(-n // 64) for n in lens), len(lens), 100, 2, dim, 64)
    fill(cache, pool, rng, list(range(len(lens))), lens)
    slots, at = i32(range(len(lens))), i32(starts_of(counts))
    q = rows(rng, sum(counts), 4, dim, "bf16", 0.3)
    one = rows(rng, len(lens), 4, dim, "bf16", 0.3)

    def many():
        return dl.history_attention(cache, slots, at, q)

    def few():                                      # the other kernel, over the same scratch
        return dl.history_attention(cache, slots, i32(range(len(lens) + 1)), one)

    want, want_few = many(), few()
    for turn in range(2):
        stalled(many, cache.error)
        for _ in range(2):
            got, got_few = (many(), few()) if turn else (few(), many())[::-1]
            assert torch.equal(got_few, want_few)
            assert torch.equal(got, want)
        assert cache.error() == dl.OK


@pytest.mark.parametrize("dim", [32, 64, 128])
def test_attention_over_a_cache_that_gives_up_in_the_middle(dim):
    """Limits about as long as one step of the pipeline: CTAs give up with parts of their
    units done, and calls after it are as ever."""
    rng = np.random.default_rng(51)
    lens, counts = [6000, 3000, 500, 6000], [2100, 1000, 300, 40]
    cache, pool = make(250, 4, 100, 2, dim, 64)
    fill(cache, pool, rng, [0, 1, 2, 3], lens)
    slots, at = i32(range(4)), i32(starts_of(counts))
    q = rows(rng, sum(counts), 4, dim, "bf16", 0.3)
    want = dl.history_attention(cache, slots, at, q)
    ran_out = 0
    for limit in (200, 1000, 3000, 10_000):
        dl.attention_test_stall(limit)
        try:
            dl.history_attention(cache, slots, at, q)
            status = cache.error()
        finally:
            dl.attention_test_stall()
        assert status in (dl.OK, dl.ERR_TIMEOUT)
        ran_out += status == dl.ERR_TIMEOUT
        for _ in range(2):
            assert torch.equal(dl.history_attention(cache, slots, at, q), want)
        assert cache.error() == dl.OK
    assert ran_out > 0


def test_the_stall_hook_checks_its_arguments():
    with pytest.raises(dl.DlrmError):
        dl.attention_test_stall(-1)
