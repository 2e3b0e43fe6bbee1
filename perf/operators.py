"""Event-history operators, as cases that can be timed and compared.

A user's event history is kept as keys and values in 8 bits (e4m3, one power-of-two scale for each
page of tokens and head) in pages of a pool; a page table maps a history's slot to its pages.

  attend    history_attention: queries (a next event, or the candidates to rank) over cached histories
  encode    window_attention: causal self-attention of ragged histories, with a sliding window and a
            few first events that stay visible
  session   history_fork + history_append + history_free: a request's own events on top of a stored
            history, dropped afterwards
  rebuild   history_free + history_append: a history is replaced by a recomputed one
  forks     history_fork + history_free: one private view of a history per request
  defrag    history_copy, history_free, history_compact, history_fork, history_free: histories move
            through the pool and end where they began, packed at its front

`own` chooses between the plain forms below (elementary torch operations in 32 bits) and this
package's operators. The pool's contents, the queries and the events come from the seed; lengths come
from the case.
"""
import math

import torch

own = False

POOL = ("k_codes", "v_codes", "k_scales", "v_scales", "table", "lengths", "refs", "free_pages", "n_free")
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # one user online, one next-event query over a short history: latency
        dict(name="attend one user", kind="attend", users=1, low=150, high=150, queries=1, heads=4, kv_heads=4,
             dim=64, page=64, causal=False, window=0, sinks=0, dtype="fp32", lse=False),
        # a serving batch: one query a user, histories of all lengths, grouped heads
        dict(name="attend 64 users", kind="attend", users=64, low=37, high=4096, queries=1, heads=8, kv_heads=2,
             dim=64, page=64, causal=False, window=0, sinks=0, dtype="bf16", lse=False),
        # the newest three events of many users look back through a window, with first events kept
        dict(name="attend window", kind="attend", users=256, low=3, high=2000, queries=3, heads=4, kv_heads=1,
             dim=32, page=32, causal=True, window=256, sinks=4, dtype="fp32", lse=True),
        # lifelong logs: few users, all time goes into reading the cache
        dict(name="attend lifelong", kind="attend", users=4, low=65000, high=100001, queries=1, heads=8, kv_heads=8,
             dim=128, page=128, causal=False, window=0, sinks=0, dtype="fp16", lse=False),
        # ranking: hundreds of candidates of a user against the whole history
        dict(name="attend ranking", kind="attend", users=16, low=1000, high=4096, queries=500, heads=4, kv_heads=2,
             dim=64, page=64, causal=False, window=0, sinks=0, dtype="bf16", lse=False),
        # short histories in the library's default precision
        dict(name="encode short", kind="encode", users=32, low=1, high=512, heads=4, kv_heads=4,
             dim=32, window=64, sinks=2, dtype="fp32", lse=True),
        # a batch of ordinary histories
        dict(name="encode batch", kind="encode", users=64, low=100, high=1024, heads=8, kv_heads=2,
             dim=64, window=256, sinks=4, dtype="bf16", lse=False),
        # lifelong logs
        dict(name="encode lifelong", kind="encode", users=2, low=16000, high=16384, heads=8, kv_heads=8,
             dim=128, window=2048, sinks=16, dtype="fp16", lse=False),
        # a request's own event on top of each stored history
        dict(name="session one event", kind="session", users=32, low=5, high=1024, new=1, kv_heads=4,
             dim=64, page=64, dtype="fp32"),
        # histories recomputed offline are loaded again
        dict(name="rebuild histories", kind="rebuild", users=16, low=2000, high=4096, kv_heads=8,
             dim=128, page=64, dtype="bf16"),
        # a private view of a history for each request in flight
        dict(name="forks", kind="forks", users=64, low=100, high=4096, kv_heads=2, dim=64, page=64, spread=8),
        # the pool is packed after churn
        dict(name="defrag", kind="defrag", users=128, low=500, high=4096, kv_heads=4, dim=64, page=64),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(("attend", "attend", "attend", "encode", "encode", "session", "rebuild", "forks", "defrag"))
    dim = rng.choice((32, 64, 128))
    page = rng.choice((32, 64, 128))
    group = rng.choice((1, 2, 4))
    kv = rng.choice((1, 2, 4, 8))
    if kind == "attend":
        queries = rng.choice((1, 1, 2, _log(rng, 2, 600)))
        high = _log(rng, 20, 100000 if queries < 8 else 5000)
        users = _log(rng, 1, max(1, min(256, 400000 // high, 30000000 // (high * queries * group * kv))))
        masked = rng.choice((False, True))
        return dict(kind=kind, users=users, low=rng.randint(0, high), high=high, queries=queries, heads=group * kv,
                    kv_heads=kv, dim=dim, page=page, causal=rng.choice((False, True)),
                    window=_log(rng, 1, high) if masked else 0, sinks=rng.choice((0, 1, 4, 17)) if masked else 0,
                    dtype=rng.choice(tuple(DTYPES)), lse=rng.choice((False, True)))
    if kind == "encode":
        high = _log(rng, 8, 8192)
        users = _log(rng, 1, max(1, min(128, 200000000 // (high * high * group * kv), 65536 // high)))
        return dict(kind=kind, users=users, low=rng.randint(0, high), high=high, heads=group * kv, kv_heads=kv,
                    dim=dim, window=rng.choice((0, _log(rng, 1, high))), sinks=rng.choice((0, 1, 4, 17)),
                    dtype=rng.choice(tuple(DTYPES)), lse=rng.choice((False, True)))
    high = _log(rng, 30, 4096)
    users = _log(rng, 1, max(1, min(256, 16 * 4096 * 8 * 128 // (high * kv * dim))))
    case = dict(kind=kind, users=users, low=rng.randint(1, high), high=high, kv_heads=kv, dim=dim, page=page)
    if kind == "session":
        case.update(new=_log(rng, 1, 200), dtype=rng.choice(tuple(DTYPES)))
    elif kind == "rebuild":
        case.update(dtype=rng.choice(tuple(DTYPES)))
    elif kind == "forks":
        case.update(spread=rng.choice((1, 2, 8)))
    return case


def _lengths(case):
    """Histories' lengths, spread over [low, high]; the first is the longest."""
    low, high = case["low"], case["high"]
    return [high - int((high - low) * ((i * 0.6180339887498949) % 1.0)) for i in range(case["users"])]


def _queries(case):
    """Queries of each user: `queries`, and with many of them some users have fewer."""
    n = case["queries"]
    return [n if n < 4 else max(1, n - (i * n // 7) % (n // 2)) for i in range(case["users"])]


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _seen(rows, length, causal, window, sinks):
    """Pairs of a query and an event that it sees; the queries are the last `rows` positions, or all stand at the end."""
    pairs = 0
    if not causal and not window:
        return rows * length
    for i in range(rows) if causal else (rows - 1,):
        end = length - rows + i + 1  # events [0, end) are not in the query's future
        if end > 0:
            seen = end if not window else min(end, window + min(sinks, max(0, end - window)))
            pairs += seen if causal else seen * rows
    return pairs


def _read(rows, length, causal, window, sinks):
    """Events that some query sees."""
    if length <= 0 or rows <= 0:
        return 0
    if not window:
        return length
    first = max(0, (max(1, length - rows + 1) if causal else length) - window)
    return length - first + min(sinks, first)


def work(case):
    kind, lens, dim, kv = case["kind"], _lengths(case), case["dim"], case["kv_heads"]
    if kind in ("attend", "encode"):
        rows = _queries(case) if kind == "attend" else lens
        causal = case.get("causal", True)
        size = DTYPES[case["dtype"]].itemsize
        pairs = sum(_seen(r, n, causal, case["window"], case["sinks"]) for r, n in zip(rows, lens))
        read = sum(_read(r, n, causal, case["window"], case["sinks"]) for r, n in zip(rows, lens))
        each = 2 * kv * dim * (1 if kind == "attend" else size)
        if kind == "attend":
            each += 2 * kv * 4 / case["page"]
        moved = read * each + sum(rows) * case["heads"] * (2 * dim * size + (4 if case["lse"] else 0))
        return {"bytes": moved, "flops": 4 * dim * case["heads"] * pairs}
    page = 2 * kv * (case["page"] * dim + 4)  # codes and scales of one page
    pages = [-(-n // case["page"]) for n in lens]
    parts = sum(1 for n in lens if n % case["page"])
    if kind == "session":
        size = DTYPES[case["dtype"]].itemsize
        return {"bytes": 2 * parts * page + sum(pages) * 8 + case["users"] * case["new"] * 2 * kv * dim * (size + 1),
                "flops": 4 * case["users"] * case["new"] * kv * dim}
    if kind == "rebuild":
        size = DTYPES[case["dtype"]].itemsize
        return {"bytes": sum(lens) * 2 * kv * dim * (size + 1) + sum(pages) * (8 + 8 * kv), "flops": 4 * sum(lens) * kv * dim}
    if kind == "forks":
        return {"bytes": case["spread"] * (2 * parts * page + sum(pages) * 16), "flops": 0}
    return {"bytes": 4 * sum(pages) * page + 2 * parts * page + sum(pages) * 32, "flops": 0}


# ---------------------------------------------------------------------------------- inputs

def _power(amax):
    """The least power of two s with amax <= 448 s, from 2^-60 to 2^60."""
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), torch.full_like(e, -60))
    return torch.ldexp(torch.ones_like(amax), e.clamp(-60, 60))


def _pool(case, gen, slots, spare):
    """A pool in use: histories of _lengths(case) in slots 0.., pages in no order, `spare` free pages."""
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    lens = _lengths(case)
    pages = [-(-n // page) for n in lens]
    used = sum(pages)
    total = used + spare
    most = max(pages + [1]) + -(-case.get("new", 0) // page)
    dev = "cuda"
    c = {}
    for name in ("k", "v"):
        x = torch.randn(total, heads, page, dim, generator=gen, device=dev)
        x *= torch.exp(0.5 * torch.randn(total, heads, 1, 1, generator=gen, device=dev))
        s = _power(x.abs().amax((2, 3)))
        c[name + "_codes"] = (x / s[:, :, None, None]).to(E4M3)
        c[name + "_scales"] = s
        del x
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    at = torch.tensor(_starts(pages), device=dev)
    j = torch.arange(most, device=dev)
    has = j < (at[1:] - at[:-1])[:, None]
    table = torch.full((slots, most), -1, dtype=torch.int32, device=dev)
    table[: len(lens)] = torch.where(has, order[(at[:-1, None] + j).clamp(max=max(used - 1, 0))], -1)
    c["table"] = table
    c["lengths"] = torch.zeros(slots, dtype=torch.int32, device=dev)
    c["lengths"][: len(lens)] = torch.tensor(lens, dtype=torch.int32, device=dev)
    c["refs"] = torch.zeros(total, dtype=torch.int32, device=dev)
    c["refs"][order[:used].long()] = 1
    c["free_pages"] = torch.zeros(total, dtype=torch.int32, device=dev)
    c["free_pages"][:spare] = order[used:]
    c["n_free"] = torch.tensor([spare], dtype=torch.int32, device=dev)
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind, lens, dev = case["kind"], _lengths(case), "cuda"
    i32 = dict(dtype=torch.int32, device=dev)
    users = case["users"]
    s = dict(case=case)

    def rows(n, heads):
        return torch.randn(n, heads, case["dim"], generator=gen, device=dev).to(DTYPES[case["dtype"]])

    if kind == "encode":
        at = _starts(lens)
        s["starts"] = torch.tensor(at, **i32)
        s["q"], s["k"], s["v"] = rows(at[-1], case["heads"]), rows(at[-1], case["kv_heads"]), rows(at[-1], case["kv_heads"])
        return s
    pages = [-(-n // case["page"]) for n in lens]
    parts = sum(1 for n in lens if n % case["page"])
    s["slots"] = torch.arange(users, **i32)
    if kind == "attend":
        at = _starts(_queries(case))
        s["starts"] = torch.tensor(at, **i32)
        s["q"] = rows(at[-1], case["heads"])
        c = _pool(case, gen, users, 3)
    elif kind == "session":
        at = _starts([case["new"]] * users)
        s["starts"] = torch.tensor(at, **i32)
        s["k"], s["v"] = rows(at[-1], case["kv_heads"]), rows(at[-1], case["kv_heads"])
        s["work"] = s["slots"] + users
        c = _pool(case, gen, 2 * users, users * (2 + case["new"] // case["page"]) + 3)
    elif kind == "rebuild":
        at = _starts(lens)
        s["starts"] = torch.tensor(at, **i32)
        s["k"], s["v"] = rows(at[-1], case["kv_heads"]), rows(at[-1], case["kv_heads"])
        c = _pool(case, gen, users, 3)
    elif kind == "forks":
        s["src"] = s["slots"].repeat(case["spread"])
        s["work"] = torch.arange(users, users * (1 + case["spread"]), **i32)
        c = _pool(case, gen, users * (1 + case["spread"]), parts * case["spread"] + 3)
    else:
        s["work"] = s["slots"] + users
        c = _pool(case, gen, 2 * users, sum(pages) + parts + 3)
    s["pool"] = c
    if own:  # the handle that a user's program keeps: the same contents in a cache of the package's own
        import dlrm_embedding_interaction_gb300 as dl
        p, h, g, d = c["k_codes"].shape
        s["cache"] = dl.HistoryCache(p, c["table"].shape[0], c["table"].shape[1], h, d, page_tokens=g)
        for name in POOL:
            getattr(s["cache"], name).copy_(c[name])
        s["pool"] = {name: getattr(s["cache"], name) for name in POOL}
    return s


# ---------------------------------------------------------------------------------- plain forms

def _softmax_out(scores, mask, v):
    """softmax(scores) v over the visible events, and the log of the sum; zeros and -inf where nothing is visible."""
    scores = scores.masked_fill(~mask, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return out, (total.log() + top).squeeze(-1)


def _visible(pos, t, length, window, sinks):
    mask = (t < length) & (t <= pos)
    return mask & ((t > pos - window) | (t < sinks)) if window else mask


def _padded(x, starts, most):
    """(users, most, heads, dim) in 32 bits of ragged rows, zeros past each user's."""
    at = starts[:-1, None].long() + torch.arange(most, device=x.device)
    inside = at < starts[1:, None]
    return x[at.clamp(max=max(len(x) - 1, 0))].float() * inside[:, :, None, None], inside


def _attend(case, q, starts, k, v, lengths, causal, most):
    """k, v: (users, kv_heads, events, dim) in 32 bits."""
    users, kv, events, dim = k.shape
    rows, inside = _padded(q, starts, most)
    group = case["heads"] // kv
    rows = rows.view(users, most, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(users, kv, group * most, dim)
    scores = torch.matmul(rows, k.transpose(-1, -2)).mul_(dim ** -0.5)
    counts = (starts[1:] - starts[:-1])[:, None]
    pos = lengths[:, None] - counts + torch.arange(most, device=q.device) if causal else (lengths[:, None] - 1).expand(users, most)
    t = torch.arange(events, device=q.device)
    mask = _visible(pos[:, :, None], t, lengths[:, None, None], case["window"], case["sinks"])
    out, lse = _softmax_out(scores.view(users, kv, group, most, events), mask[:, None, None], v[:, :, None])
    out = out.permute(0, 3, 1, 2, 4).reshape(users, most, case["heads"], dim)[inside].to(q.dtype)
    lse = lse.permute(0, 3, 1, 2).reshape(users, most, case["heads"])[inside]
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _gather(codes, scales, rows):
    """(users, heads, events, dim) in 32 bits of the pages of `rows`."""
    at = rows.clamp(min=0).long()
    x = codes.view(torch.uint8)[at].view(E4M3).float() * scales[at][:, :, :, None, None]
    u, m, h, g, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(u, h, m * g, d)


def _fork(c, src, dst, share):
    page = c["k_codes"].shape[2]
    length = c["lengths"][src]
    full = length // page if share else torch.zeros_like(length)
    j = torch.arange(c["table"].shape[1], device=src.device)
    has = j < ((length + page - 1) // page)[:, None]
    fresh = has & (j >= full[:, None])
    need = fresh.sum(1)
    rank = (need.cumsum(0) - need)[:, None] + j - full[:, None]
    old = c["table"][src]
    new = c["free_pages"][(c["n_free"] - 1 - rank).clamp(min=0)]
    c["table"][dst] = torch.where(fresh, new, torch.where(has, old, -1))
    c["refs"].index_add_(0, old.clamp(min=0).view(-1).long(), (has & ~fresh).view(-1).to(torch.int32))
    to, of = new[fresh].long(), old[fresh].long()
    c["refs"][to] = 1
    for name in ("k", "v"):
        codes = c[name + "_codes"].view(torch.uint8)
        codes[to] = codes[of]
        c[name + "_scales"][to] = c[name + "_scales"][of]
    c["n_free"] -= need.sum()
    c["lengths"][dst] = length


def _free(c, slots):
    row = c["table"][slots].view(-1)
    pages = row[row >= 0].long()
    place = torch.arange(len(pages), device=row.device)
    c["refs"].index_add_(0, pages, torch.full_like(pages, -1, dtype=torch.int32))
    last = torch.full((len(c["refs"]),), -1, device=row.device).scatter_reduce(0, pages, place, "amax")
    gone = pages[(c["refs"][pages] == 0) & (last[pages] == place)].to(torch.int32)
    c["free_pages"][c["n_free"] + torch.arange(len(gone), device=row.device)] = gone.flip(0)
    c["n_free"] += len(gone)
    c["table"][slots] = -1
    c["lengths"][slots] = 0


def _append(c, slots, starts, new):
    pages, heads, page, dim = c["k_codes"].shape
    count = starts[1:] - starts[:-1]
    before = c["lengths"][slots]
    after = before + count
    first, end = (before + page - 1) // page, (after + page - 1) // page
    need = end - first
    j = torch.arange(c["table"].shape[1], device=slots.device)
    fresh = (j >= first[:, None]) & (j < end[:, None])
    rank = (need.cumsum(0) - need)[:, None] + j - first[:, None]
    row = torch.where(fresh, c["free_pages"][(c["n_free"] - 1 - rank).clamp(min=0)], c["table"][slots])
    c["table"][slots] = row
    c["refs"][row[fresh].long()] = 1
    c["n_free"] -= need.sum()
    c["lengths"][slots] = after
    t = torch.arange(len(new["k"]), device=slots.device)
    user = torch.searchsorted(starts[1:].contiguous(), t.to(torch.int32), right=True)
    pos = before[user] + t - starts[user]
    at = row[user, pos // page].long()
    off = pos % page
    kept = torch.zeros(pages, dtype=torch.int32, device=slots.device)  # events that a page holds already
    part = before % page
    some = (part > 0) & (count > 0)
    kept[row.gather(1, (before // page).clamp(max=row.shape[1] - 1)[:, None].long())[:, 0][some].long()] = part[some].to(torch.int32)
    touched = torch.zeros(pages, dtype=torch.bool, device=slots.device)
    touched[at] = True
    held = kept.nonzero().view(-1)
    for name in ("k", "v"):
        x = new[name].float()
        codes, scales = c[name + "_codes"], c[name + "_scales"]
        amax = torch.zeros(pages, heads, device=x.device).scatter_reduce(0, at[:, None].expand(-1, heads), x.abs().amax(-1), "amax")
        s = torch.where((kept > 0)[:, None], torch.maximum(scales, _power(amax)), _power(amax))
        s = torch.where(touched[:, None], s, scales)
        was = codes.view(torch.uint8)[held].view(E4M3).float()
        now = was * (scales[held] / s[held])[:, :, None, None]
        live = torch.arange(page, device=x.device) < kept[held][:, None]
        codes.view(torch.uint8)[held] = torch.where(live[:, None, :, None], now, was).to(E4M3).view(torch.uint8)
        scales.copy_(s)
        codes.view(torch.uint8)[at, :, off] = (x / s[at][:, :, None]).to(E4M3).view(torch.uint8)


def _compact(c):
    ids = torch.arange(len(c["refs"]), device=c["refs"].device)
    live = c["refs"] > 0
    n = live.sum()
    to, of = ids[~live & (ids < n)], ids[live & (ids >= n)]
    for name in ("k", "v"):
        codes = c[name + "_codes"].view(torch.uint8)
        codes[to] = codes[of]
        c[name + "_scales"][to] = c[name + "_scales"][of]
    c["refs"][to] = c["refs"][of]
    c["refs"][of] = 0
    name = ids.to(torch.int32)
    name[of] = to.to(torch.int32)
    c["table"].copy_(torch.where(c["table"] >= 0, name[c["table"].clamp(min=0).long()], -1))
    free = len(ids) - n
    c["free_pages"].copy_(torch.where(ids < free, len(ids) - 1 - ids, c["free_pages"]))
    c["n_free"].copy_(free.view(1))


def _plain(s):
    case, c = s["case"], s.get("pool")
    kind = case["kind"]
    if kind == "attend":
        rows = c["table"][s["slots"]]
        length = c["lengths"][s["slots"]]
        k, v = _gather(c["k_codes"], c["k_scales"], rows), _gather(c["v_codes"], c["v_scales"], rows)
        v = v * (torch.arange(v.shape[2], device=v.device) < length[:, None])[:, None, :, None]
        return _attend(case, s["q"], s["starts"], k, v, length, case["causal"], max(_queries(case)))
    if kind == "encode":
        most = case["high"]
        k, v = (_padded(s[n], s["starts"], most)[0].permute(0, 2, 1, 3) for n in ("k", "v"))
        return _attend(case, s["q"], s["starts"], k, v, s["starts"][1:] - s["starts"][:-1], True, most)
    if kind == "session":
        _fork(c, s["slots"], s["work"], True)
        _append(c, s["work"], s["starts"], s)
        _free(c, s["work"])
    elif kind == "rebuild":
        _free(c, s["slots"])
        _append(c, s["slots"], s["starts"], s)
    elif kind == "forks":
        _fork(c, s["src"], s["work"], True)
        view = c["table"].clone()
        _free(c, s["work"])
        return dict(c, view=view)
    else:
        _fork(c, s["slots"], s["work"], False)
        _free(c, s["slots"])
        _compact(c)
        _fork(c, s["work"], s["slots"], True)
        _free(c, s["work"])
    return dict(c)


# ---------------------------------------------------------------------------------- one pass

def run(s):
    if not own:
        return _plain(s)
    import dlrm_embedding_interaction_gb300 as dl
    case, cache, kind = s["case"], s.get("cache"), s["case"]["kind"]
    if kind in ("attend", "encode"):
        got = {"out": torch.empty_like(s["q"])}
        if case["lse"]:
            got["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
        if kind == "attend":
            dl.history_attention(cache, s["slots"], s["starts"], s["q"], got["out"], causal=case["causal"],
                                 window=case["window"], sinks=case["sinks"], lse=got.get("lse"))
        else:
            dl.window_attention(s["q"], s["k"], s["v"], s["starts"], got["out"], window=case["window"],
                                sinks=case["sinks"], lse=got.get("lse"))
        return got
    if kind == "session":
        dl.history_fork(cache, s["slots"], s["work"])
        dl.history_append(cache, s["work"], s["starts"], s["k"], s["v"])
        dl.history_free(cache, s["work"])
    elif kind == "rebuild":
        dl.history_free(cache, s["slots"])
        dl.history_append(cache, s["slots"], s["starts"], s["k"], s["v"])
    elif kind == "forks":
        dl.history_fork(cache, s["src"], s["work"])
        view = cache.table.clone()
        dl.history_free(cache, s["work"])
        return dict(s["pool"], view=view)
    else:
        dl.history_copy(cache, s["slots"], s["work"])
        dl.history_free(cache, s["slots"])
        dl.history_compact(cache)
        dl.history_fork(cache, s["work"], s["slots"])
        dl.history_free(cache, s["work"])
    return dict(s["pool"])


# ---------------------------------------------------------------------------------- in 64 bits

def _exact_rows(q, k, v, ends, case):
    """Attention in 64 bits of one user: q (rows, heads, dim), k and v (events, kv_heads, dim); row i sees events
    before ends[i], of those the last `window` and the first `sinks`. Rows go in blocks, each over its events alone."""
    rows, heads, dim = q.shape
    group = heads // k.shape[1]
    window, sinks = case["window"], case["sinks"]
    out = torch.zeros(rows, heads, dim, dtype=torch.float64, device=q.device)
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64, device=q.device)
    step = max(1, min(2048, 400_000_000 // (8 * heads * max(1, len(k)))))
    for a in range(0, rows, step):
        b = min(rows, a + step)
        end = torch.tensor(ends[a:b], device=q.device)
        last = max(ends[a:b])
        if last <= 0:
            continue
        first = max(0, min(ends[a:b]) - window) if window else 0
        at = torch.cat([torch.arange(min(sinks, first)), torch.arange(first, last)]).to(q.device)
        ok = at < end[:, None]
        if window:
            ok &= (at >= end[:, None] - window) | (at < sinks)
        for h in range(heads):
            x = (q[a:b, h].double() @ k[at, h // group].double().T) / math.sqrt(dim)
            x[~ok] = -math.inf
            total = torch.logsumexp(x, 1)
            w = torch.exp(x - total[:, None])
            w[~ok] = 0
            out[a:b, h] = w @ v[at, h // group].double()
            lse[a:b, h] = total
    return out, lse


def _exact_e4m3(x):
    """The e4m3 value nearest to x (even on ties): 4 bits from 2^-6 up, steps of 2^-9 below, at most 448."""
    m, _ = torch.frexp(x)  # x = m 2^e, 0.5 <= |m| < 1, so x / m is 2^e exactly
    step = torch.where(x == 0, torch.ones_like(x), x / m / 16).clamp(min=2.0 ** -9)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    kind = case["kind"]
    if kind in ("forks", "defrag"):
        return None  # pages move, nothing is computed
    lens = _lengths(case)
    if kind == "rebuild" and sum(lens) > 8000 * case["page"]:
        return None  # page by page below: too long
    s = prepare(case, seed)
    if kind in ("attend", "encode"):
        got = [], []
        at = s["starts"].tolist()
        for u, n in enumerate(lens):
            q = s["q"][at[u]:at[u + 1]]
            if kind == "attend":
                ids = s["pool"]["table"][u, : -(-n // case["page"])].long()
                k, v = (
                    (s["pool"][x + "_codes"].view(torch.uint8)[ids].view(E4M3).double() * s["pool"][x + "_scales"][ids][:, :, None, None].double())
                    .permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], case["dim"])[:n] for x in ("k", "v"))
            else:
                k, v = s["k"][at[u]:at[u + 1]], s["v"][at[u]:at[u + 1]]
            causal = kind == "encode" or case["causal"]
            ends = [n - len(q) + i + 1 if causal else n for i in range(len(q))]
            if len(q):
                for x, y in zip(got, _exact_rows(q, k, v, ends, case)):
                    x.append(y)
        out, lse = (torch.cat(x) if x else None for x in got)
        return {"out": out, "lse": lse} if case["lse"] else {"out": out}
    # session and rebuild: the pages as the definition leaves them
    c = s["pool"]
    page, at = case["page"], s["starts"].tolist()
    free = c["free_pages"][: int(c["n_free"])].tolist()
    codes = {n: c[n + "_codes"].double() for n in ("k", "v")}
    scales = {n: c[n + "_scales"].double() for n in ("k", "v")}
    rows = [[int(p) for p in r if p >= 0] for r in c["table"][: case["users"]].tolist()]
    if kind == "rebuild":
        free += [p for r in reversed(rows) for p in reversed(r)]
        rows, lens = [[] for _ in rows], [0] * len(rows)
    else:
        for u, n in enumerate(lens):  # the forks' own copies of pages that are not full
            if n % page:
                old, new = rows[u][-1], free.pop()
                for d in (codes, scales):
                    for x in d.values():
                        x[new] = x[old]
                rows[u][-1] = new
    for u, n in enumerate(lens):
        rows[u] += [free.pop() for _ in range(-(-(n + at[u + 1] - at[u]) // page) - len(rows[u]))]
        for name in ("k", "v"):
            new = s[name][at[u]:at[u + 1]].double()
            done = 0
            while done < len(new):
                pos = n + done
                p, off = rows[u][pos // page], pos % page
                part = new[done: done + page - off].permute(1, 0, 2)
                big = part.abs().amax((1, 2))
                scale = torch.pow(2.0, torch.ceil(torch.log2(big / 448)).clamp(-60, 60))
                if off:
                    scale = torch.maximum(scale, scales[name][p])
                    codes[name][p, :, :off] = _exact_e4m3(codes[name][p, :, :off] * (scales[name][p] / scale)[:, None, None])
                scales[name][p] = scale
                codes[name][p, :, off: off + part.shape[1]] = _exact_e4m3(part / scale[:, None, None])
                done += part.shape[1]
    return {"k_codes": codes["k"], "v_codes": codes["v"], "k_scales": scales["k"], "v_scales": scales["v"],
            "table": None, "lengths": None, "refs": None, "free_pages": None, "n_free": None}
