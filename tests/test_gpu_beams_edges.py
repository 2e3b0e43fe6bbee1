"""The beam search's operators on the GPU at the edges of their definitions: layouts, empty
and infinite values, refused requests, many requests, streams and graphs, and the three of
them in a run. Bounds as in test_gpu_beams.py."""
import numpy as np
import pytest

import beam_ref
import test_gpu_beams as base

torch = pytest.importorskip("torch")
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES, append, beams, check_rows, check_select, f64, i32, make, rows, same_state, starts_of = (
    base.TYPES, base.append, base.beams, base.check_rows, base.check_select, base.f64, base.i32, base.make,
    base.rows, base.same_state, base.starts_of)


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    from dlrm_embedding_interaction_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def shared_attention(cache, slots, at, groups, q, **more):
    return dl.history_prefix_attention(cache, i32(slots), i32(at), i32(groups), q, **more)


# ------------------------------------------------------------------ attention with a shared prefix

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", ["heads first", "gaps", "odd"])
def test_strided_queries_and_outputs(dtype, layout):
    rng = np.random.default_rng(1)
    cache, pool, slots, groups = beams(rng, [200, 90], [5, 3], [2] * 8, 2, 64, 64)
    at = list(range(0, 17, 2))
    q = rows(rng, 16, 4, 64, dtype, 0.3)
    if layout == "heads first":
        have, out = q.transpose(0, 1).contiguous().transpose(0, 1), torch.full_like(q, 9.0).transpose(0, 1).contiguous().transpose(0, 1)
    else:
        wide = 80 if layout == "gaps" else 67
        have, out = (torch.full((16, 4, wide), 9.0, dtype=q.dtype, device="cuda") for _ in range(2))
        have[:, :, :64] = q
        have, out, rest = have[:, :, :64], out[:, :, :64], out[:, :, 64:]
    assert shared_attention(cache, slots, at, groups, have, out=out) is out
    check_rows(pool, slots, at, q, out, None, dtype)
    if layout != "heads first":
        assert (rest == 9).all()                  # between the rows: as it was
    assert cache.error() == dl.OK


@pytest.mark.parametrize("dtype", list(TYPES))
def test_what_masked_events_hold_has_no_influence(dtype):
    """NaN and infinities outside the window, in shared and in own pages, and behind the end."""
    rng = np.random.default_rng(2)
    idle = 3000
    cache, pool, slots, groups = beams(rng, [300], [4], [0] * 4, 1, 64, 32, spare=20, idle=idle)
    bad = torch.full((40, 1, 64), float("nan"), device="cuda")
    bad[::2] = float("inf")
    dl.history_append(cache, i32(slots), i32(range(0, 41, 10)), bad, bad)
    pool.append(slots, list(range(0, 41, 10)), (f64(bad), f64(bad)))
    append(cache, pool, rng, slots, [70] * 4)
    cache.v_codes.view(torch.uint8)[cache.refs == 0] = 0x7f
    at = starts_of([1, 2, 1, 1] + [0] * idle)
    q = rows(rng, 5, 2, 64, dtype, 0.3)
    for causal in (False, True):
        lse = torch.empty(5, 2, device="cuda")
        out = shared_attention(cache, slots + [0] * idle, at, [0, 4, 4 + idle], q, causal=causal, window=60, sinks=20, lse=lse)
        check_rows(pool, slots, at[:5], q, out, lse, dtype, causal=causal, window=60, sinks=20)
    assert cache.error() == dl.OK


@pytest.mark.parametrize("dtype", list(TYPES))
def test_one_requests_events_that_are_not_finite_reach_no_other(dtype):
    """The rows of a group share tiles, and 0 * NaN is NaN."""
    rng = np.random.default_rng(16)
    cache, pool, slots, groups = beams(rng, [130], [6], [9] * 6, 2, 64, 32, spare=10)
    bad = torch.full((2, 2, 64), float("nan"), device="cuda")
    append(cache, pool, rng, [slots[1]], [1])
    dl.history_append(cache, i32([slots[2]]), i32([0, 2]), bad, bad)
    pool.append([slots[2]], [0, 2], (f64(bad), f64(bad)))
    at = [0, 2, 4, 6, 8, 10, 12]
    q = rows(rng, 12, 8, 64, dtype, 0.3)
    lse = torch.empty(12, 8, device="cuda")
    out = shared_attention(cache, slots, at, groups, q, lse=lse)
    for b in (0, 1, 3, 4, 5):
        check_rows(pool, [slots[b]], [0, 2], q[2 * b:2 * b + 2], out[2 * b:2 * b + 2], lse[2 * b:2 * b + 2], dtype)
    assert out[4:6].isnan().all()
    # events that all of them see
    cache, pool, slots, groups = beams(rng, [130], [3], [0] * 3, 2, 64, 32)
    cache.v_codes.view(torch.uint8)[cache.table[slots[0], 1], 1, :, :] = 0x7f
    out = shared_attention(cache, slots, [0, 1, 2, 3], groups, q[:3])
    assert out[:, 4:].isnan().all() and not out[:, :4].isnan().any()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_infinite_queries_and_rows_without_weights(dtype):
    """As history_attention has them: NaN where a score is, 0 / 0 where all are -infinity."""
    rng = np.random.default_rng(3)
    cache, pool, slots, groups = beams(rng, [200], [3], [5] * 3, 1, 64, 64)
    q = rows(rng, 3, 1, 64, dtype, 0.3)
    q[0, 0, 3] = float("inf")
    q[1] = float("nan")
    at = [0, 1, 2, 3]
    lse, other = torch.empty(3, 1, device="cuda"), torch.empty(3, 1, device="cuda")
    out = shared_attention(cache, slots, at, groups, q, lse=lse)
    want = dl.history_attention(cache, i32(slots), i32(at), q, lse=other)
    np.testing.assert_array_equal(np.isnan(f64(out)), np.isnan(f64(want)))
    np.testing.assert_array_equal(np.isnan(f64(lse)), np.isnan(f64(other)))
    check_rows(pool, slots[2:], [0, 1], q[2:], out[2:], lse[2:], dtype)


def test_trimmed_pages_are_read_by_no_window_that_left_them():
    rng = np.random.default_rng(4)
    idle = 3000
    cache, pool, slots, groups = beams(rng, [500], [4], [3, 40, 3, 70], 1, 64, 32, spare=10, idle=idle)
    for where in (slots[:2], slots[2:]):
        dl.history_trim(cache, i32(where), 100, 10)
        pool.release(where, 100, 10)
    same_state(cache, pool)
    q = rows(rng, 4, 2, 64, "bf16", 0.3)
    at, groups = list(range(5)) + [4] * idle, [0, 4, 4 + idle]
    out = shared_attention(cache, slots + [0] * idle, at, groups, q, window=100, sinks=10)
    check_rows(pool, slots, at[:5], q, out, None, "bf16", window=100, sinks=10)
    assert cache.error() == dl.OK
    shared_attention(cache, slots + [0] * idle, at, groups, q, window=400)
    assert cache.error() == dl.ERR_INDEX_OOB


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shared", [True, False])
def test_rows_of_no_request_stay_and_slots_may_occur_twice(dtype, shared):
    rng = np.random.default_rng(17)
    cache, pool, slots, groups = beams(rng, [200, 90], [4, 3], [2] * 7, 2, 64, 64, shared=shared)
    slots = [slots[0], slots[0], slots[2], 0, slots[4], slots[5], slots[5]]   # (0: the user's own)
    at = [3, 4, 6, 6, 9, 10, 11, 12]
    q = rows(rng, 14, 4, 64, dtype, 0.3)
    out, lse = torch.full_like(q, 9.0), torch.full((14, 4), 9.0, device="cuda")
    shared_attention(cache, slots, at, groups, q, out=out, lse=lse)
    check_rows(pool, slots, at, q, out, lse, dtype)
    for x in (out, lse):
        assert (x[:3] == 9).all() and (x[12:] == 9).all()
    before = out.clone()
    shared_attention(cache, [], [0], [0], q[:0], out=out[:0])
    shared_attention(cache, slots, [5] * 8, groups, q, out=out)   # no rows at all
    shared_attention(cache, [], [0], [0, 0, 0], q, out=out)       # groups of nothing
    assert torch.equal(out, before) and cache.error() == dl.OK


@pytest.mark.parametrize("shared", [True, False])
def test_bad_requests_are_reported_and_the_next_call_is_as_ever(shared):
    rng = np.random.default_rng(5)
    cache, pool, slots, groups = beams(rng, [300, 100], [4, 3], [2] * 7, 2, 64, 64, shared=shared)
    at = list(range(8))
    q = rows(rng, 7, 4, 64, "fp32", 0.3)
    want = shared_attention(cache, slots, at, groups, q)
    check_rows(pool, slots, at, q, want, None, "fp32")
    # a slot that is none: its rows see nothing, the others are served
    broken = list(slots)
    broken[1], broken[5] = -1, cache.n_slots
    out = shared_attention(cache, broken, at, groups, q)
    assert cache.error() == dl.ERR_INDEX_OOB
    assert (out[[1, 5]] == 0).all()
    check_rows(pool, broken, at, q, out, None, "fp32")
    for starts, cut in (([0, 1, 2, 9, 4, 5, 6, 7], groups), ([0, 1, 2, 3, 4, 5, 6, 8], groups),
                        ([-1, 1, 2, 3, 4, 5, 6, 7], groups), (at, [0, 5, 4, 7]), (at, [0, 4, 8]), (at, [-1, 4, 7]),
                        (at, [1, 4, 7]), (at, [0, 4, 6])):
        shared_attention(cache, slots, starts, cut, q)
        assert cache.error() == dl.ERR_UNSUPPORTED, (starts, cut)
        assert torch.equal(shared_attention(cache, slots, at, groups, q), want)
        assert cache.error() == dl.OK
    same_state(cache, pool)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("counts,queries", [([700], 1), ([1] * 600, 1), ([300, 2, 400], 2)])
def test_many_requests_and_groups(dtype, counts, queries):
    rng = np.random.default_rng(6)
    n = sum(counts)
    cache, pool, slots, groups = beams(rng, [40 + i % 50 for i in range(len(counts))], counts, [i % 3 for i in range(n)],
                                       1, 32, 32)
    at = [queries * i for i in range(n + 1)]
    q = rows(rng, at[-1], 1, 32, dtype, 0.3)
    out = shared_attention(cache, slots, at, groups, q)
    check_rows(pool, slots, at, q, out, None, dtype)
    assert cache.error() == dl.OK


def test_pages_past_four_gigabytes():
    rng = np.random.default_rng(19)
    heads, dim, page = 8, 128, 128
    n = (1 << 32) // (heads * dim * page) + 40      # the last pages lie past 2^32 bytes
    cache = dl.HistoryCache(n, 8, 400, heads, dim, page_tokens=page)
    pool = beam_ref.Pool(40, 8, 400, heads, dim, page)
    cache.free_pages.copy_(torch.arange(n, dtype=torch.int32, device="cuda"))   # the last page first
    pool.free = list(range(40))
    append(cache, pool, rng, [0], [300])
    dl.history_fork(cache, i32([0] * 4), i32([1, 2, 3, 4]))
    pool.fork([0] * 4, [1, 2, 3, 4], True)
    append(cache, pool, rng, [1, 2, 3, 4], [3, 1, 200, 0])
    assert cache.table.max().item() == n - 1
    dl.history_reorder(cache, i32([1, 2, 3, 4]), i32([2, 2, 0, 0]))
    assert pool.reorder([1, 2, 3, 4], [2, 2, 0, 0])
    for dtype in TYPES:
        q = rows(rng, 4, 16, dim, dtype, 0.3)
        out = shared_attention(cache, [1, 2, 3, 4], [0, 1, 2, 3, 4], [0, 4], q)
        check_rows(pool, [1, 2, 3, 4], [0, 1, 2, 3, 4], q, out, None, dtype)
    assert cache.error() == dl.OK


# ------------------------------------------------------------------ reordering

@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("batch", [7, 60, 1300])
def test_any_parents_with_refusals_among_them(seed, batch):
    """Parents out of range, slots that are none or occur twice, empty slots, too few pages."""
    rng = np.random.default_rng(100 * batch + seed)
    slots_all, page = batch + 20, 32
    cache, pool = make(3 * batch if seed % 2 else 8 * batch, slots_all, 6, 1, 32, page)
    some = rng.permutation(slots_all)[:batch].tolist()
    append(cache, pool, rng, some, rng.integers(0, 2 * page, batch).tolist())
    cache.error()
    for step in range(3):
        slots = rng.permutation(slots_all)[:batch].tolist()
        parents = rng.integers(-1, batch, batch).tolist()
        want = dl.OK
        if step == 1:
            for i in rng.integers(0, batch, 3):
                slots[i] = [-1, slots_all, slots[0]][int(rng.integers(0, 3))]
            for i in rng.integers(0, batch, 2):
                parents[i] = [batch, -2][int(rng.integers(0, 2))]
        there = [s for s in slots if 0 <= s < slots_all]
        if len(there) < batch or any(not -1 <= p < batch or (p >= 0 and not 0 <= slots[p] < slots_all)
                                     for b, p in enumerate(parents) if 0 <= slots[b] < slots_all and slots[b] not in slots[:b]):
            want = dl.ERR_INDEX_OOB
        elif len(set(there)) < batch:
            want = dl.ERR_INVALID_ARG
        dl.history_reorder(cache, i32(slots), i32(parents))
        enough = pool.reorder(slots, parents)
        same_state(cache, pool)
        if not enough and want in (dl.OK, dl.ERR_INVALID_ARG):
            want = dl.ERR_OOM
        assert cache.error() == want
        new = rng.integers(0, 3, batch).tolist()
        live = [s for s in dict.fromkeys(slots) if 0 <= s < slots_all]
        append(cache, pool, rng, live, new[:len(live)])
        same_state(cache, pool)
        cache.error()


def test_too_few_pages_leave_everything_as_it_was():
    rng = np.random.default_rng(9)
    cache, pool = make(6, 8, 4, 1, 32, 32)
    append(cache, pool, rng, [0, 1], [40, 33])      # four pages of six, two of them not full
    slots, parents = [0, 1, 2, 3, 4], [0, 0, 0, 0, 1]
    dl.history_reorder(cache, i32(slots), i32(parents))
    assert not pool.reorder(slots, parents)
    # copies: 1, 2, 3 of slot 0's last page; given up: none, as 4 continues slot 1
    assert cache.error() == dl.ERR_OOM
    assert cache.lengths.tolist() == [40, 33, 0, 0, 0, 0, 0, 0] and int(cache.n_free) == 2
    same_state(cache, pool)
    slots, parents = [0, 1, 2, 3], [0, 0, 0, 0]     # one given up, two free: enough
    dl.history_reorder(cache, i32(slots), i32(parents))
    assert pool.reorder(slots, parents)
    same_state(cache, pool)
    assert cache.error() == dl.OK


@pytest.mark.parametrize("seed", range(4))
def test_reordering_among_the_other_operators(seed):
    """Forks, trims, frees, appends and compactions in between."""
    rng = np.random.default_rng(200 + seed)
    cache, pool = make(120, 12, 8, 1, 32, 32)
    for step in range(40):
        slots = rng.permutation(12)[:int(rng.integers(1, 13))].tolist()
        kind = int(rng.integers(0, 6))
        if kind == 0:
            parents = rng.integers(-1, len(slots), len(slots)).tolist()
            dl.history_reorder(cache, i32(slots), i32(parents))
            assert pool.reorder(slots, parents)
        elif kind == 1:
            window, sinks = int(rng.integers(1, 90)), int(rng.integers(0, 40))
            dl.history_trim(cache, i32(slots), window, sinks)
            pool.release(slots, window, sinks)
        elif kind == 2:
            dl.history_free(cache, i32(slots[:2]))
            pool.release(slots[:2])
        elif kind == 3:
            dl.history_fork(cache, i32(slots), i32(slots[::-1]))
            pool.fork(slots, slots[::-1], True)
        elif kind == 4:
            dl.history_compact(cache)
            pool.compact()
        else:
            append(cache, pool, rng, slots, rng.integers(0, 40, len(slots)).tolist())
        same_state(cache, pool)
    cache.error()


@pytest.mark.parametrize("page", [64, 2 ** 31 - 1, -2])
def test_reordering_past_pages_that_a_table_cannot_hold(page):
    rng = np.random.default_rng(10)
    cache, pool = make(64, 8, 4, 1, 32, 32)
    append(cache, pool, rng, [0, 1], [100, 40])
    cache.table[0, 1] = page
    cache.table[0, 3] = page                        # the last page, not full
    dl.history_reorder(cache, i32([0, 1, 2, 3]), i32([1, 0, 0, 1]))
    assert cache.error() == dl.OK
    assert cache.lengths[:4].tolist() == [40, 100, 100, 40]
    assert cache.table[1, 1] == page and cache.table[2, 3] == page
    dl.history_free(cache, i32(range(4)))
    assert int(cache.n_free) == 62                  # all but the two that the table lost
    assert cache.error() == dl.OK


# ------------------------------------------------------------------ selection

def test_strides_and_broadcast_masks():
    rng = np.random.default_rng(11)
    for vocab in (300, 5000):
        wide = torch.from_numpy(rng.standard_normal((6, vocab + 13))).float().cuda()
        logits, starts = wide[:, 5:5 + vocab], [0, 6]
        scores = torch.from_numpy(rng.standard_normal(6)).float().cuda()
        plain = dl.beam_select(logits, scores, i32(starts), 9)
        check_select(logits, scores, starts, 9, None, plain)
        again = dl.beam_select(logits.contiguous(), scores, i32(starts), 9)
        assert all(torch.equal(a, b) for a, b in zip(plain, again))   # alignment changes nothing
        mask = torch.from_numpy(rng.random(vocab) < 0.1).cuda()
        for allowed in (mask, mask[None], mask[None].expand(6, vocab), mask.repeat(6, 1)):
            got = dl.beam_select(logits, scores, i32(starts), 9, allowed=allowed)
            check_select(logits, scores, starts, 9, mask[None].expand(6, vocab), got)
        one = torch.zeros(6, vocab, dtype=torch.bool, device="cuda")
        one[2, 7] = True                            # a beam with one way on: at no cost
        got = dl.beam_select(logits, scores, i32(starts), 2, allowed=one)
        assert got[0][0, 0] == scores[2] and got[1].tolist() == [[2, -1]] and got[2].tolist() == [[7, -1]]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [4096, 8197, 16383, 40960])
def test_rows_may_begin_at_any_element(dtype, vocab):
    """Wherever logits and masks lie the result is the same bit for bit, and what lies before
    and behind a row is not the row's."""
    rng = np.random.default_rng(20)
    x = torch.from_numpy(rng.standard_normal((3, vocab))).to(TYPES[dtype]).cuda()
    mask = torch.from_numpy(rng.random((3, vocab)) < 0.5).cuda()
    starts = i32([0, 1, 3])
    want = [dl.beam_select(x, None, starts, 40, allowed=m) for m in (None, mask)]
    check_select(x, None, [0, 1, 3], 40, None, want[0])
    check_select(x, None, [0, 1, 3], 40, mask, want[1])
    for offset in range(9):
        wide = torch.full((3, vocab + 21), float("nan"), dtype=x.dtype, device="cuda")
        wide[:, offset:offset + vocab] = x
        wide_mask = torch.ones(3, vocab + 23, dtype=torch.bool, device="cuda")
        wide_mask[:, 2 * offset % 7:2 * offset % 7 + vocab] = mask
        for m, expected in ((None, want[0]), (wide_mask[:, 2 * offset % 7:2 * offset % 7 + vocab], want[1])):
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            got = dl.beam_select(wide[:, offset:offset + vocab], None, starts, 40, allowed=m, err_flag=err)
            assert int(err) == 0 and all(torch.equal(a, b) for a, b in zip(got, expected)), offset


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("width", [3, 27, 100])
def test_masks_of_ranges_and_logits_that_rise(dtype, width):
    """Tokens in a few places of a chunk only, and chunks whose last logits are the largest."""
    rng = np.random.default_rng(21)
    vocab = 20011
    x = torch.from_numpy(rng.standard_normal((9, vocab))).to(TYPES[dtype]).cuda()
    x[4] += torch.linspace(0, 30, vocab, device="cuda").to(x.dtype)
    x[5] -= torch.linspace(0, 30, vocab, device="cuda").to(x.dtype)
    mask = torch.zeros(9, vocab, dtype=torch.bool, device="cuda")
    for row, (a, b) in enumerate([(0, 700), (1000, 1030), (5000, 9000), (19990, vocab), (0, vocab), (0, vocab), (4090, 4100),
                                  (0, 2), (12000, 12900)]):
        mask[row, a:b] = True
    for starts in ([0, 9], list(range(10)), [0, 2, 4, 7, 9]):
        check_select(x, None, starts, width, mask, dl.beam_select(x, None, i32(starts), width, allowed=mask))
        check_select(x, None, starts, width, None, dl.beam_select(x, None, i32(starts), width))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [200, 70000])
def test_zeros_of_both_signs_are_equal(dtype, vocab):
    rng = np.random.default_rng(18)
    x = torch.zeros(3, vocab, dtype=TYPES[dtype], device="cuda")
    x[torch.from_numpy(rng.random((3, vocab)) < 0.5).cuda()] = -0.0
    got = dl.beam_select(x, None, i32([0, 3]), 100)
    assert (got[1] == 0).all() and got[2].tolist() == [list(range(100))]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [100, 9000])
def test_extreme_logits(dtype, vocab):
    """Of the type's lowest value, -infinity, and rows far from zero and from one another."""
    rng = np.random.default_rng(12)
    t = TYPES[dtype]
    x = torch.from_numpy(rng.standard_normal((8, vocab))).to(t).cuda()
    x[0] = torch.finfo(t).min
    x[1, ::2] = torch.finfo(t).min
    x[2, 3:] = -float("inf")
    x[3] = -float("inf")
    x[4] += 1000.0
    x[5] -= 1000.0
    x[6] = torch.linspace(-30000, 30000, vocab, device="cuda").to(t)
    if dtype != "fp16":
        x[7] = torch.linspace(-1e30, 1e30, vocab, device="cuda").to(t)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    starts = [0, 3, 8]
    got = dl.beam_select(x, None, i32(starts), 50, err_flag=err)
    best, parents, tokens = (y.cpu().numpy() for y in got)
    assert int(err) == 0
    want, want_rows, want_tokens, every = beam_ref.select(f64(x), np.zeros(8), starts, 50)
    there = want > -np.inf
    np.testing.assert_array_equal(best > -np.inf, there)
    # scores of 10^4 and more are fp32 numbers that far apart, and so are the logits
    assert (np.abs(best - want)[there] <= 2.0 ** -19 + 2.0 ** -23 * np.abs(want[there])).all()
    picked = every[parents[there], tokens[there]]
    assert (np.abs(picked - want[there]) <= 2.0 ** -19 + 2.0 ** -23 * np.abs(want[there])).all()


@pytest.mark.parametrize("vocab", [50, 20000])
def test_bad_rows_and_starts_are_reported_and_the_others_served(vocab):
    rng = np.random.default_rng(13)
    x = torch.from_numpy(rng.standard_normal((7, vocab))).float().cuda()
    scores = torch.zeros(7, device="cuda")
    good = dl.beam_select(x, scores, i32([0, 2, 4, 7]), 3)
    for what in ("nan", "inf", "score nan", "score inf"):
        y, s = x.clone(), scores.clone()
        if what.startswith("score"):
            s[3] = float(what.split()[1])
        else:
            y[3, vocab // 2] = float(what)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = dl.beam_select(y, s, i32([0, 2, 4, 7]), 3, err_flag=err)
        assert int(err) == 1 << dl.ERR_INVALID_ARG, what
        assert all(torch.equal(a[[0, 2]], b[[0, 2]]) for a, b in zip(got, good))
        assert (got[1][1] == 2).all()               # the group's other row
    err.zero_()
    got = dl.beam_select(x, scores, i32([0, 2, 9, 7]), 3, err_flag=err)
    assert int(err) == dl.ERRBIT_OFFSETS
    assert torch.equal(got[2][0], good[2][0]) and (got[1][1:] == -1).all() and (got[0][1:] == -float("inf")).all()
    none = dl.beam_select(x, scores, i32([3, 3]), 4)
    assert (none[0] == -float("inf")).all() and (none[1] == -1).all() and (none[2] == -1).all()
    assert dl.beam_select(x, scores, i32([0]), 4)[0].shape == (0, 4)
    assert (dl.beam_select(x[:0], scores[:0], i32([0, 0]), 4)[1] == -1).all()


@pytest.mark.parametrize("counts,vocab,width", [([700], 40, 200), ([1] * 3000, 30, 2), ([0, 300, 1], 5000, 256),
                                                ([40], 200000, 10), ([2], 3000017, 64),
                                                ([1, 2], 2 ** 24 + 9, 5), ([1500], 5000, 7), ([3, 2500], 4500, 100)])
def test_many_rows_groups_and_chunks(counts, vocab, width):
    g = torch.Generator(device="cuda")
    g.manual_seed(14)
    starts = starts_of(counts)
    x = (2 * torch.randn(starts[-1], vocab, generator=g, device="cuda")).half()
    scores = -3 * torch.rand(starts[-1], generator=g, device="cuda")
    got = dl.beam_select(x, scores, i32(starts), width)
    if starts[-1] * vocab < 1 << 22:
        check_select(x, scores, starts, width, None, got)
        return
    # the same on the GPU in 64 bits, where it is too much for the restatement
    every = (x.double() - torch.logsumexp(x.double(), 1, keepdim=True) + scores.double()[:, None])
    for i in range(len(counts)):
        if counts[i]:
            want = every[starts[i]:starts[i + 1]].reshape(-1).topk(width).values
            assert ((got[0][i].double() - want).abs() <= 2.0 ** -20 + 2.0 ** -24 * want.abs()).all()
            picked = every[got[1][i].long(), got[2][i].long()]
            assert ((picked - want).abs() <= 2.0 ** -19).all()
            assert len(set(zip(got[1][i].tolist(), got[2][i].tolist()))) == width


# ------------------------------------------------------------------ a run of them

def test_steps_of_a_search_on_another_stream_and_in_graphs():
    """Selection, reordering, the new events and their attention, as they are used; then the
    same from two graphs that take turns."""
    rng = np.random.default_rng(15)
    users, width, vocab = 3, 4, 500
    n = users * width
    cache, pool, slots, groups = beams(rng, [100, 37, 200], [width] * users, [0] * n, 2, 64, 32, spare=4 * n)
    logits = torch.from_numpy(rng.standard_normal((n, vocab))).bfloat16().cuda()
    kv = rows(rng, n, 2, 64, "bf16")
    q = rows(rng, n, 4, 64, "bf16", 0.3)
    scores = torch.zeros(n, device="cuda")
    slots_t, at, groups_t = i32(slots), i32(range(n + 1)), i32(groups)

    def step(stream=None):
        selected = dl.beam_select(logits, scores, groups_t, width, stream=stream)
        parents = selected[1]
        dl.history_reorder(cache, slots_t, parents.view(-1), stream=stream)
        dl.history_append(cache, slots_t, at, kv, kv, stream=stream)
        return selected, parents, dl.history_prefix_attention(cache, slots_t, at, groups_t, q, stream=stream)

    def after(got, turns):
        selected, parents, out = got
        check_select(logits, scores, groups, width, None, selected)
        for _ in range(turns):
            assert pool.reorder(slots, parents.view(-1).tolist())
            pool.append(slots, list(range(n + 1)), (f64(kv), f64(kv)))
        same_state(cache, pool)
        check_rows(pool, slots, list(range(n + 1)), q, out, None, "bf16")
        assert cache.error() == dl.OK

    after(step(), 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    after(got, 1)
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(step())
    for turn in (0, 1, 1, 0):
        graphs[turn].replay()
        torch.cuda.synchronize()
        after(outs[turn], 1)
