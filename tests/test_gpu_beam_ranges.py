"""The beam search's operators on the GPU over ranges of values and sizes where one way of
computing passes into another. Bounds as in test_gpu_beams.py."""
import numpy as np
import pytest

import beam_ref
import test_gpu_beams as base

torch = pytest.importorskip("torch")
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402

pytestmark = pytest.mark.gpu
f64, i32 = base.f64, base.i32


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    from dlrm_embedding_interaction_gb300 import build
    build.build()
    torch.cuda.set_device(0)


# ------------------------------------------------------------------ selection

@pytest.mark.parametrize("first,second", [(-1, 1), (1, -1), (-21, 1), (1, 1), (-1, -1)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("where", ["two chunks", "two warps", "two tiles"])
def test_logits_on_both_sides_of_65536(where, sign, first, second):
    """Sums of exponentials have one scale for references below 65,536 in magnitude and another
    from there on; parts of a row (chunks, a CTA's warps, a thread's tiles of 2048 tokens) may
    have either. A row's two logits that count stand on sides `first` and `second` of the edge
    or further below it. One candidate a group: its score is -log(1 + e^(difference)), within
    2^-20 and half an ulp of fp32."""
    rows = 96
    at = {"two chunks": (5, 20000), "two warps": (5, 1500), "two tiles": (5, 2048 + 5)}[where]
    near = np.linspace(1 / 128, 1.6, rows)
    x = np.full((rows, 30000), -1e9, np.float32)
    # (steps of 2^-7 and 2^-8: numbers of fp32 on either side)
    for column, side, gap in ((at[0], first, near), (at[1], second, near[::-1] + 1 / 128)):
        gap = gap if abs(side) == 1 else gap + abs(side)
        x[:, column] = (sign * 65536 + np.sign(side) * gap).astype(np.float32)
    logits = torch.from_numpy(x).cuda()
    starts = list(range(rows + 1))
    got = dl.beam_select(logits, None, i32(starts), 1)
    want, _, tokens, _ = beam_ref.select(f64(logits), np.zeros(rows), starts, 1)
    best = got[0].cpu().numpy().astype(np.float64)
    assert (np.abs(best - want) <= 2.0 ** -20 + 2.0 ** -24 * np.abs(want)).all(), np.abs(best - want).max()
    np.testing.assert_array_equal(got[2].cpu().numpy(), tokens)


@pytest.mark.parametrize("sign", [1, -1])
def test_rows_around_65536_keep_their_order(sign):
    """Rows of one group whose scores are the logarithms of their own sums: every candidate's
    score is its logit, so the order over all rows is that of the logits, which lie 2^-7 apart."""
    rng = np.random.default_rng(1)
    rows, vocab, width = 24, 20000, 48
    x = np.full((rows, vocab), -1e9, np.float32)
    steps = rng.permutation(rows * 8).reshape(rows, 8)
    columns = rng.permutation(vocab)[:rows * 8].reshape(rows, 8)
    np.put_along_axis(x, columns, (sign * 65536 + (steps - rows * 4) / 128.0).astype(np.float32), 1)
    d = x.astype(np.float64)
    top = d.max(1, keepdims=True)
    # a sum that is a number of fp32 (2^-7 apart) less: scores take the whole part of it
    lse = (np.log(np.exp(d - top).sum(1, keepdims=True)) + top)[:, 0]
    scores = torch.from_numpy(lse.astype(np.float32)).cuda()
    got = dl.beam_select(torch.from_numpy(x).cuda(), scores, i32([0, rows]), width)
    want, want_rows, want_tokens, every = beam_ref.select(d, f64(scores), [0, rows], width)
    picked = every[got[1].cpu().numpy(), got[2].cpu().numpy()]
    # (a score is the logit and up to 2^-8 that the row's logarithm lost as a number of fp32)
    assert (np.abs(picked - want) <= 2.0 ** -19).all(), np.abs(picked - want).max()
    assert (np.abs(got[0].cpu().numpy() - want) <= 2.0 ** -20 + 2.0 ** -24 * np.abs(want)).all()


def microseconds(call, turns=5):
    """The least of a few timings of the call."""
    times = []
    for _ in range(turns):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        call()
        end.record()
        torch.cuda.synchronize()
        times.append(1000 * begin.elapsed_time(end))
    return min(times)


# Beams that are not in use, as searches mark them.
UNUSED = [-1e4, -1e9, float(np.finfo(np.float32).min)]


@pytest.mark.parametrize("unused", UNUSED)
@pytest.mark.parametrize("dtype,vocab,width", [("fp32", 256, 8), ("fp32", 4096, 8), ("bf16", 32768, 16), ("fp16", 300007, 100)])
@pytest.mark.parametrize("used", [1, 7])
def test_beams_that_are_not_in_use(dtype, vocab, width, used, unused):
    """They lose to every continuation of the others, and cost no more than if they were in use
    (ten times, as calls of microseconds are noisy; where the farthest row's rounding is
    everybody's margin it is a hundred times)."""
    rng = np.random.default_rng(vocab + used)
    beams, groups = 8, 4
    starts = list(range(0, groups * beams + 1, beams))
    logits = torch.from_numpy(2 * rng.standard_normal((groups * beams, vocab))).to(base.TYPES[dtype]).cuda()
    scores = torch.from_numpy(-5 * rng.random(groups * beams)).float().cuda()
    at = i32(starts)
    before = microseconds(lambda: dl.beam_select(logits, scores, at, width))
    scores.view(groups, beams)[:, used:] = unused
    got = dl.beam_select(logits, scores, at, width)
    best, rows, tokens = (x.cpu().numpy() for x in got)
    want, want_rows, want_tokens, every = beam_ref.select(f64(logits), f64(scores), starts, width)
    assert ((rows - np.arange(groups)[:, None] * beams) < used).all()
    assert (np.abs(best - want) <= 2.0 ** -20 + 2.0 ** -24 * np.abs(want)).all()
    assert (np.abs(every[rows, tokens] - want) <= 2.0 ** -19).all()
    assert microseconds(lambda: dl.beam_select(logits, scores, at, width)) <= 10 * before


@pytest.mark.parametrize("dtype", list(base.TYPES))
@pytest.mark.parametrize("vocab", [500, 9001])
@pytest.mark.parametrize("spread", [1e3, 1e5, 1e9, 1e30])
def test_rows_far_apart_are_compared_exactly(dtype, vocab, spread):
    """Scores and logits of all magnitudes, among them rows whose score makes up for where their
    logits lie, so that candidates of every row are close to the bound: the order is that of 64
    bits, up to what the logarithms may be off (2^-19) and 64 bits round (2^-50 of the largest)."""
    rng = np.random.default_rng(vocab)
    rows, width = 40, 50
    x = rng.standard_normal((rows, vocab))
    if dtype == "fp32":
        x[::3] += np.float32(spread) * np.sign(rng.standard_normal((len(x[::3]), 1))) * 0.75
    logits = torch.from_numpy(x).to(base.TYPES[dtype]).cuda()
    s = -3 * rng.random(rows)
    s[1::4] -= spread
    s[2::4] = -rng.random(len(s[2::4])) * spread
    scores = torch.from_numpy(s).float().cuda()
    starts = [0, 4, 5, rows]
    best, parents, tokens = (y.cpu().numpy() for y in dl.beam_select(logits, scores, i32(starts), width))
    want, _, _, every = beam_ref.select(f64(logits), f64(scores), starts, width)
    tol = 2.0 ** -19 + 2.0 ** -50 * spread
    assert (np.abs(best - want) <= tol + 2.0 ** -24 * np.abs(want)).all()
    picked = every[parents, tokens]
    assert (np.abs(picked - want) <= tol + 2.0 ** -50 * np.abs(want)).all()
    for g in range(3):
        assert len(set(zip(parents[g].tolist(), tokens[g].tolist()))) == width


@pytest.mark.parametrize("unused", UNUSED)
@pytest.mark.parametrize("dtype,vocab,width", [("fp32", 300, 16), ("fp32", 4096, 16), ("bf16", 32768, 100), ("fp16", 300007, 16)])
def test_places_that_only_unused_beams_can_take(dtype, vocab, width, unused):
    """One beam in use may continue with three tokens; the other places go to beams whose
    scores agree in most of their bits, or in all 64 (numbers of 64 bits lie 2^75 apart at
    -3.4e38, so that a row's continuations are equal there, and the first row takes all
    places). (Thirty times: a part of the candidates is gone through a few times more, in 64
    bits. One bit of the score at a time takes hundreds of times.)"""
    rng = np.random.default_rng(vocab)
    beams, groups = 8, 3
    starts = list(range(0, groups * beams + 1, beams))
    logits = torch.from_numpy(2 * rng.standard_normal((groups * beams, vocab))).to(base.TYPES[dtype]).cuda()
    allowed = torch.ones(groups * beams, vocab, dtype=torch.bool, device="cuda")
    scores = torch.zeros(groups * beams, device="cuda")
    at = i32(starts)
    call = lambda: dl.beam_select(logits, scores, at, width, allowed=allowed)   # noqa: E731
    before = microseconds(call)
    used = 3
    allowed[used::beams] = False
    allowed[used::beams, ::vocab // 3 + 1] = True
    scores.view(groups, beams)[:] = unused
    scores[used::beams] = -1.0
    best, rows, tokens = (x.cpu().numpy() for x in call())
    want, want_rows, want_tokens, every = beam_ref.select(f64(logits), f64(scores), starts, width, allowed.cpu().numpy())
    assert (rows[:, :3] % beams == used).all() and (rows[:, 3:] % beams != used).all()
    if unused < -1e30:
        np.testing.assert_array_equal(rows[:, 3:], want_rows[:, 3:])
    for g in range(groups):
        assert len(set(zip(rows[g].tolist(), tokens[g].tolist()))) == width
    tol = 2.0 ** -19 + 2.0 ** -50 * np.abs(want)
    assert (np.abs(every[rows, tokens] - want) <= tol).all()
    assert (np.abs(best - want) <= tol + 2.0 ** -24 * np.abs(want)).all()
    assert microseconds(call) <= 30 * before, (microseconds(call), before)


@pytest.mark.parametrize("fill", ["lowest", -1e4, 0.0])
@pytest.mark.parametrize("dtype,vocab,width", [("fp32", 20011, 5), ("bf16", 32768, 16), ("fp16", 300007, 100), ("bf16", 300007, 256)])
@pytest.mark.parametrize("left", [0, 3, 200])
def test_tokens_masked_by_a_value(dtype, vocab, width, left, fill):
    """Most logits of a row are one number (tokens masked by a value of their own, or a head
    that saturates), so that it is the bound wherever a chunk has few others; ties go by token.
    Ten times as long as other logits take is the noise of short calls and some passes more; a
    pass for each bit of the value and of the index takes thirty to fifty times. Where a group
    has fewer tokens left than places (the group of one row has `left`), what the others' lists
    hold is equal, at most 11 rows of 37 lists of 256: 104,000 scores in 64 bits, of 7 operations
    each, 2 a clock and SM, are 190 us a pass, and four passes (range, places, counts, the taken
    ones) 770, 15 times the 50 us; thirty are allowed."""
    rng = np.random.default_rng(vocab + left)
    rows, t = 24, base.TYPES[dtype]
    logits = torch.from_numpy(2 * rng.standard_normal((rows, vocab))).to(t).cuda()
    starts = [0, 6, 12, 13, rows]
    at = i32(starts)
    before = microseconds(lambda: dl.beam_select(logits, None, at, width))
    value = torch.finfo(t).min if fill == "lowest" else fill
    x = torch.full_like(logits, value)
    for row in range(rows):                       # rows of their own tokens, some of them side by side
        keep = rng.permutation(vocab)[:left] if row % 2 else np.arange(left) + 37 * row
        x[row, torch.from_numpy(keep).cuda()] = logits[row, torch.from_numpy(keep).cuda()]
    got = dl.beam_select(x, None, at, width)
    best, parents, tokens = (y.cpu().numpy() for y in got)
    want, want_rows, want_tokens, every = beam_ref.select(f64(x), np.zeros(rows), starts, width)
    assert (np.abs(best - want) <= 2.0 ** -20 + 2.0 ** -24 * np.abs(want)).all()
    assert (np.abs(every[parents, tokens] - want) <= 2.0 ** -19).all()
    for g in range(len(starts) - 1):              # of each row: its largest logits, the first of equal ones
        for row in set(parents[g].tolist()):
            mine = tokens[g][parents[g] == row]
            order = np.argsort(-f64(x[row]), kind="stable")[:len(mine)]
            np.testing.assert_array_equal(mine, order)
    assert microseconds(lambda: dl.beam_select(x, None, at, width)) <= (10 if left >= width else 30) * before


@pytest.mark.parametrize("dtype", list(base.TYPES))
@pytest.mark.parametrize("kind", ["steps", "all rise", "two levels", "masked steps", "one above"])
@pytest.mark.parametrize("width", [1, 33, 256])
def test_chunks_that_overflow_their_lists(dtype, kind, width):
    """Rows in which every tile has larger logits than the one before, with and without ties."""
    vocab, t = 70001, base.TYPES[dtype]
    rng = np.random.default_rng(width)
    i = np.arange(vocab)
    x = {"steps": i // 700 * 0.125, "all rise": i * (40.0 / vocab), "two levels": (i % 3 == 1) * 5.0 + i // 30000,
         "masked steps": i // 300 * 0.0625, "one above": (i == 50000) * 1.0 - (i % 2) * 1e-3}[kind]
    logits = torch.from_numpy(np.stack([x, x[::-1].copy(), rng.permutation(x)] * 3)).to(t).cuda()
    allowed = torch.from_numpy(rng.random(logits.shape) < 0.7).cuda() if kind == "masked steps" else None
    starts = list(range(0, 10, 3))
    got = dl.beam_select(logits, None, i32(starts), width, allowed=allowed)
    best, parents, tokens = (y.cpu().numpy() for y in got)
    mask = None if allowed is None else allowed.cpu().numpy()
    want, _, _, every = beam_ref.select(f64(logits), np.zeros(9), starts, width, mask)
    assert (np.abs(best - want) <= 2.0 ** -20 + 2.0 ** -24 * np.abs(want)).all()
    assert (np.abs(every[parents, tokens] - want) <= 2.0 ** -19).all()
    for g in range(3):
        for row in set(parents[g].tolist()):
            mine = tokens[g][parents[g] == row]
            y = f64(logits[row])
            if mask is not None:
                y = np.where(mask[row], y, -np.inf)
            np.testing.assert_array_equal(mine, np.argsort(-y, kind="stable")[:len(mine)])


@pytest.mark.parametrize("vocab", [300, 5000])
@pytest.mark.parametrize("kind", ["equal", "spread", "unused"])
def test_groups_that_bad_starts_lay_over_one_another(vocab, kind):
    """Starts that decrease leave two groups with rows in common, more than shared memory holds
    the states of: what they write is undefined, but the call ends, reports them, and serves
    the group before them; the next call is as ever."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    logits = torch.zeros(900, vocab, device="cuda")
    if kind != "equal":
        logits.normal_(generator=g)
    scores = torch.zeros(900, device="cuda")
    if kind == "unused":
        scores[1::2] = -1e9
    more = [900] * 20 if vocab == 300 else []     # groups enough for one launch
    good = dl.beam_select(logits, scores, i32([0, 10, 600, 900] + more), 20)
    for _ in range(20):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = dl.beam_select(logits, scores, i32([0, 10, 600, 40, 900] + more), 20, err_flag=err)
        assert int(err) & dl.ERRBIT_OFFSETS
        assert all(torch.equal(a[0], b[0]) for a, b in zip(got, good))
        assert (got[1][2] == -1).all()            # from 600 to 40: none
    again = dl.beam_select(logits, scores, i32([0, 10, 600, 900] + more), 20)
    assert all(torch.equal(a, b) for a, b in zip(again, good))
