"""Beam search over event histories, as cases that can be timed and compared.

A model that proposes a user's next items (or the codes that spell an item) keeps a few
continuations of the user's history alive. Each is a slot of the event-history cache that was forked
from the user's own: their first pages are the same pages, and only their last ones differ.

  prefix    history_prefix_attention: queries of all beams over their histories; what the beams of a
            user share is read once for all of them
  select    beam_select: the best continuations of each user over all its beams and the whole
            vocabulary, by the sum of log-probabilities, some tokens not allowed
  reorder   history_reorder: every beam's slot takes over the history of the beam it continues

`own` chooses between the plain forms below (elementary torch operations) and this package's
operators. The pool's contents, queries, logits and scores come from the seed; lengths and the beams'
parents come from the case.
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
        # one user online, four beams over a short history: latency
        dict(name="prefix one user", kind="prefix", users=1, beams=4, low=150, high=150, new=3, queries=1, heads=4,
             kv_heads=4, dim=64, page=64, causal=False, window=0, sinks=0, dtype="fp32", lse=False),
        # a serving batch: histories of all lengths, up to 16 beams, grouped heads
        dict(name="prefix 64 users", kind="prefix", users=64, beams=16, low=37, high=4096, new=3, queries=1, heads=8,
             kv_heads=2, dim=64, page=64, causal=False, window=0, sinks=0, dtype="bf16", lse=False),
        # each beam's newest two events look back through a window, with first events kept
        dict(name="prefix window", kind="prefix", users=32, beams=10, low=3, high=2000, new=5, queries=2, heads=4,
             kv_heads=1, dim=32, page=32, causal=True, window=512, sinks=4, dtype="fp32", lse=True),
        # lifelong logs: few users, all time goes into reading the cache
        dict(name="prefix lifelong", kind="prefix", users=4, beams=8, low=65000, high=100001, new=4, queries=1, heads=8,
             kv_heads=8, dim=128, page=128, causal=False, window=0, sinks=0, dtype="fp16", lse=False),
        # many beams a user: the products count
        dict(name="prefix wide", kind="prefix", users=16, beams=64, low=1000, high=4096, new=3, queries=1, heads=8,
             kv_heads=2, dim=64, page=64, causal=False, window=0, sinks=0, dtype="bf16", lse=False),
        # one user's next code of an item, out of a codebook: latency
        dict(name="select one user", kind="select", users=1, beams=4, vocab=256, width=4, dtype="fp32", keep=0),
        # the codes of many users, where only codes that continue some item are allowed
        dict(name="select codes", kind="select", users=256, beams=32, vocab=256, width=32, dtype="fp32", keep=8),
        # a serving batch over a vocabulary of item tokens
        dict(name="select items", kind="select", users=64, beams=32, vocab=32768, width=32, dtype="bf16", keep=0),
        # few users over a whole catalogue, an odd number of items, some of them not for this user
        dict(name="select catalogue", kind="select", users=4, beams=10, vocab=1000003, width=100, dtype="fp16", keep=2),
        # one user's beams after a step
        dict(name="reorder one user", kind="reorder", users=1, beams=4, low=150, high=150, new=3, kv_heads=4, dim=64,
             page=64),
        # a serving batch's beams after a step
        dict(name="reorder 64 users", kind="reorder", users=64, beams=16, low=37, high=4096, new=3, kv_heads=2, dim=64,
             page=64),
        # beams that have gone apart by several pages
        dict(name="reorder long beams", kind="reorder", users=16, beams=10, low=1000, high=4096, new=300, kv_heads=8,
             dim=128, page=64),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(("prefix", "prefix", "prefix", "select", "select", "reorder"))
    dim = rng.choice((32, 64, 128))
    page = rng.choice((32, 64, 128))
    group = rng.choice((1, 2, 4))
    kv = rng.choice((1, 2, 4, 8))
    beams = _log(rng, 1, 64)
    if kind == "prefix":
        queries = rng.choice((1, 1, 1, 2, 5))
        high = _log(rng, 20, 100000 if beams <= 8 else 5000)
        most = min(256, 3000000000 // (beams * high * kv * dim), 40000000 // (beams * queries * high * group * kv))
        masked = rng.choice((False, False, True))
        return dict(kind=kind, users=_log(rng, 1, max(1, most)), beams=beams, low=rng.randint(0, high), high=high,
                    new=_log(rng, 1, 2 * page), queries=queries, heads=group * kv, kv_heads=kv, dim=dim, page=page,
                    causal=rng.choice((False, True)), window=_log(rng, 1, high) if masked else 0,
                    sinks=rng.choice((0, 1, 4, 17)) if masked else 0, dtype=rng.choice(tuple(DTYPES)),
                    lse=rng.choice((False, True)))
    if kind == "select":
        vocab = _log(rng, 2, 1000003)
        return dict(kind=kind, users=_log(rng, 1, max(1, min(256, 64000000 // (beams * vocab)))), beams=beams, vocab=vocab,
                    width=_log(rng, 1, 128), dtype=rng.choice(tuple(DTYPES)), keep=rng.choice((0, 0, 2, 8)))
    high = _log(rng, 30, 4096)
    new = _log(rng, 1, 300)
    most = min(256, 100000000 // (beams * kv * dim * (new + page) + high * kv * dim))
    return dict(kind=kind, users=_log(rng, 1, max(1, most)), beams=beams, low=rng.randint(0, high), high=high, new=new,
                kv_heads=kv, dim=dim, page=page)


def _lengths(case):
    """Stored histories' lengths, spread over [low, high]; the first is the longest."""
    low, high = case["low"], case["high"]
    return [high - int((high - low) * ((i * 0.6180339887498949) % 1.0)) for i in range(case["users"])]


def _beams(case):
    """Beams of each user: `beams`, and with many of them some users have fewer left."""
    n = case["beams"]
    return [n if n < 4 else max(1, n - (i * n // 7) % (n // 2)) for i in range(case["users"])]


def _parents(case):
    """The beam that each beam continues, as an index into all beams: more often one of the first of its user."""
    got, at = [], 0
    for u, n in enumerate(_beams(case)):
        got += [at + int(n * ((i + 0.37 + u) * 0.6180339887498949 % 1.0) ** 2) for i in range(n)]
        at += n
    return got


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _pairs(rows, length, causal, window, sinks):
    """Pairs of a query and an event that it sees; the queries are the last `rows` positions, or all stand at the end."""
    total = 0
    for i in range(rows):
        end = length - rows + i + 1 if causal else length
        if end > 0:
            total += end if not window else min(end, window + min(sinks, max(0, end - window)))
    return total


def work(case):
    kind = case["kind"]
    if kind == "select":
        rows = sum(_beams(case))
        places = rows * case["vocab"]
        return {"bytes": places * (DTYPES[case["dtype"]].itemsize + (1 if case["keep"] else 0)) + rows * 4 + case["users"] * case["width"] * 12,
                "flops": 4 * places}
    kv, dim, page, new = case["kv_heads"], case["dim"], case["page"], case["new"]
    if kind == "prefix":
        rows, window, sinks = case["queries"], case["window"], case["sinks"]
        size = DTYPES[case["dtype"]].itemsize
        read = pairs = 0
        for n, beams in zip(_lengths(case), _beams(case)):
            shared, end = n // page * page, n + new
            first = max(0, (end - rows + 1 if case["causal"] else end) - window) if window else 0
            kept = min(sinks, first)
            read += max(0, shared - first) + min(kept, shared) + beams * (end - max(first, shared) + max(0, kept - shared))
            pairs += beams * _pairs(rows, end, case["causal"], window, sinks)
        queries = sum(_beams(case)) * rows
        return {"bytes": read * 2 * kv * (dim + 4 / page) + queries * case["heads"] * (2 * dim * size + (4 if case["lse"] else 0)),
                "flops": 4 * dim * case["heads"] * pairs}
    parents, moved, entries, at = _parents(case), 0, 0, 0
    for n, beams in zip(_lengths(case), _beams(case)):
        mine = parents[at: at + beams]
        if (n + new) % page:
            moved += beams - len(set(mine))
        entries += sum(1 for i, p in enumerate(mine) if p != at + i) * (-(-(n + new) // page) - n // page)
        at += beams
    return {"bytes": moved * 2 * 2 * kv * (page * dim + 4) + entries * 24 + len(parents) * 16, "flops": 0}


# ---------------------------------------------------------------------------------- inputs

def _power(amax):
    """The least power of two s with amax <= 448 s, from 2^-60 to 2^60."""
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), torch.full_like(e, -60))
    return torch.ldexp(torch.ones_like(amax), e.clamp(-60, 60))


def _pool(case, gen, spare):
    """A pool in use: a slot for each beam; the beams of a user share the full pages of its stored history and have
    pages of their own from there on; pages in no order, `spare` of them free."""
    page, heads, dim, new = case["page"], case["kv_heads"], case["dim"], case["new"]
    dev = "cuda"
    lens, beams = _lengths(case), _beams(case)
    users, slots = len(lens), sum(beams)
    shared = torch.tensor([n // page for n in lens], device=dev)
    tails = torch.tensor([-(-(n + new) // page) - n // page for n in lens], device=dev)
    most = max(-(-(n + new) // page) for n in lens)
    n_beams = torch.tensor(beams, device=dev)
    user = torch.repeat_interleave(torch.arange(users, device=dev), n_beams)
    of_user = shared.cumsum(0) - shared                    # a user's first page
    of_beam = shared.sum() + tails[user].cumsum(0) - tails[user]
    used = sum(n // page + b * (-(-(n + new) // page) - n // page) for n, b in zip(lens, beams))
    total = used + spare
    c = {}
    for name in ("k", "v"):
        x = torch.randn(total, heads, page, dim, generator=gen, device=dev)
        x *= torch.exp(0.5 * torch.randn(total, heads, 1, 1, generator=gen, device=dev))
        s = _power(x.abs().amax((2, 3)))
        c[name + "_codes"] = (x / s[:, :, None, None]).to(E4M3)
        c[name + "_scales"] = s
        del x
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    j = torch.arange(most, device=dev)
    own_page = j >= shared[user][:, None]
    at = torch.where(own_page, of_beam[:, None] + j - shared[user][:, None], of_user[user][:, None] + j)
    has = j < (shared + tails)[user][:, None]
    c["table"] = torch.where(has, order[at.clamp(max=total - 1)], -1).to(torch.int32).contiguous()
    c["lengths"] = (torch.tensor(lens, device=dev)[user] + new).to(torch.int32)
    refs = torch.zeros(total, dtype=torch.int32, device=dev)
    c["refs"] = refs.index_add_(0, c["table"].clamp(min=0).view(-1).long(), has.view(-1).to(torch.int32))
    c["free_pages"] = torch.zeros(total, dtype=torch.int32, device=dev)
    c["free_pages"][:spare] = order[used:]
    c["n_free"] = torch.tensor([spare], dtype=torch.int32, device=dev)
    assert c["table"].shape == (slots, most)
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev = "cuda"
    i32 = dict(dtype=torch.int32, device=dev)
    beams = _beams(case)
    s = dict(case=case)
    s["groups"] = torch.tensor(_starts(beams), **i32)
    if case["kind"] == "select":
        rows, vocab = sum(beams), case["vocab"]
        s["logits"] = (2.0 * torch.randn(rows, vocab, generator=gen, device=dev)).to(DTYPES[case["dtype"]])
        s["scores"] = -5.0 * torch.rand(rows, generator=gen, device=dev)
        if case["keep"]:
            s["allowed"] = torch.rand(rows, vocab, generator=gen, device=dev) < 1.0 / case["keep"]
            s["allowed"][5::11] = False  # a beam that continues no item
        return s
    s["slots"] = torch.arange(sum(beams), **i32)
    if case["kind"] == "prefix":
        s["starts"] = torch.arange(0, sum(beams) * case["queries"] + 1, case["queries"], **i32)
        s["q"] = torch.randn(sum(beams) * case["queries"], case["heads"], case["dim"], generator=gen, device=dev).to(DTYPES[case["dtype"]])
    else:
        s["parents"] = torch.tensor(_parents(case), **i32)
    c = s["pool"] = _pool(case, gen, 3)
    if own:  # the handle that a user's program keeps: the same contents in a cache of the package's own
        import dlrm_embedding_interaction_gb300 as dl
        p, h, g, d = c["k_codes"].shape
        s["cache"] = dl.HistoryCache(p, c["table"].shape[0], c["table"].shape[1], h, d, page_tokens=g)
        for name in POOL:
            getattr(s["cache"], name).copy_(c[name])
        s["pool"] = {name: getattr(s["cache"], name) for name in POOL}
    return s


# ---------------------------------------------------------------------------------- plain forms

def _gather(codes, scales, rows):
    """(slots, heads, events, dim) in 32 bits of the pages of `rows`."""
    at = rows.clamp(min=0).long()
    x = codes.view(torch.uint8)[at].view(E4M3).float()
    x *= scales[at][:, :, :, None, None]
    u, m, h, g, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(u, h, m * g, d)


def _prefix(s):
    case, c = s["case"], s["pool"]
    kv, dim, queries, window = case["kv_heads"], case["dim"], case["queries"], case["window"]
    group = case["heads"] // kv
    rows, length = c["table"][s["slots"]], c["lengths"][s["slots"]].long()
    k = _gather(c["k_codes"], c["k_scales"], rows)
    n, events = k.shape[0], k.shape[2]
    q = s["q"].float().view(n, queries, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(n, kv, group * queries, dim)
    scores = torch.matmul(q, k.transpose(-1, -2)).mul_(dim ** -0.5).view(n, kv, group, queries, events)
    del k
    pos = length[:, None] - queries + torch.arange(queries, device=q.device) if case["causal"] else (length - 1)[:, None].expand(n, queries)
    t = torch.arange(events, device=q.device)
    mask = (t < length[:, None, None]) & (t <= pos[:, :, None])
    if window:
        mask &= (t > pos[:, :, None] - window) | (t < case["sinks"])
    scores.masked_fill_(~mask[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = _gather(c["v_codes"], c["v_scales"], rows)
    v *= (t < length[:, None])[:, None, :, None]  # what stands behind the last event is no value
    out = torch.matmul(p.view(n, kv, group * queries, events), v).view(n, kv, group, queries, dim)
    out /= torch.where(total > 0, total, torch.ones_like(total))
    out = out.permute(0, 3, 1, 2, 4).reshape(n * queries, case["heads"], dim).to(s["q"].dtype)
    if not case["lse"]:
        return {"out": out}
    return {"out": out, "lse": (total.log() + top).squeeze(-1).permute(0, 3, 1, 2).reshape(n * queries, case["heads"])}


def _select(s):
    """In 64 bits: whether one candidate stands before another may hang by the last digits of 32."""
    width, starts = s["case"]["width"], s["groups"].long()
    x = s["logits"].double()
    if "allowed" in s:
        x.masked_fill_(~s["allowed"], -math.inf)
    rows, vocab = x.shape
    dev = x.device
    top = x.amax(1, keepdim=True)
    total = torch.where(top > -math.inf, top, torch.zeros_like(top))
    total = total + torch.exp(x - total).sum(1, keepdim=True).log()
    x.sub_(torch.where(total > -math.inf, total, torch.zeros_like(total))).add_(s["scores"].double()[:, None])
    users = len(starts) - 1
    of = torch.searchsorted(starts[1:].contiguous(), torch.arange(rows, device=dev), right=True)
    most = s["case"]["beams"]
    flat = torch.full((users, most, vocab), -math.inf, dtype=torch.float64, device=dev)
    flat[of, torch.arange(rows, device=dev) - starts[of]] = x
    flat = flat.view(users, most * vocab)
    kth = flat.topk(min(width, most * vocab), dim=1).values[:, -1:]
    user, place = ((flat >= kth) & (flat > -math.inf)).nonzero().unbind(1)
    value = flat[user, place]
    order = torch.sort(value, descending=True, stable=True).indices
    order = order[torch.sort(user[order], stable=True).indices]  # by user, then value, then place
    user, place, value = user[order], place[order], value[order]
    rank = torch.arange(len(user), device=dev) - torch.searchsorted(user, user)
    first = rank < width
    user, place, value, rank = user[first], place[first], value[first], rank[first]
    scores = torch.full((users, width), -math.inf, device=dev)
    parents = torch.full((users, width), -1, dtype=torch.int32, device=dev)
    tokens = torch.full((users, width), -1, dtype=torch.int32, device=dev)
    scores[user, rank] = value.float()
    parents[user, rank] = (starts[user] + place // vocab).to(torch.int32)
    tokens[user, rank] = (place % vocab).to(torch.int32)
    return {"scores": scores, "parents": parents, "tokens": tokens}


def _reorder(s):
    c = s["pool"]
    slots, parents = s["slots"].long(), s["parents"].long()
    page, dev = c["k_codes"].shape[2], slots.device
    n, most = len(slots), c["table"].shape[1]
    b, j = torch.arange(n, device=dev), torch.arange(most, device=dev)
    old, length = c["table"][slots], c["lengths"][slots].long()
    new, after = old[parents], length[parents]
    part = after % page > 0
    last = (after // page).clamp(max=most - 1)
    # of the requests that continue a beam, its own or the first one keeps a last page that is not full
    keeper = torch.full((n,), n, device=dev).scatter_reduce(0, parents, torch.where(parents == b, -1, b), "amin")
    copies = part & (keeper[parents] != torch.where(parents == b, -1, b))
    given = (length % page > 0) & (keeper == n)            # last pages that nobody continues
    spare = old[b, (length // page).clamp(max=most - 1)][given]
    n_copies, n_given, n_free = copies.sum(), given.sum(), c["n_free"][0].long()
    rank = copies.cumsum(0) - 1
    from_stack = c["free_pages"][(n_free - 1 - (rank - n_given).clamp(min=0)).clamp(min=0)]
    padded = torch.cat([spare, spare.new_zeros(1)])
    page_of = torch.where(rank < n_given, padded[rank.clamp(min=0).minimum(n_given)], from_stack)
    was = new[b, last]
    new = torch.where(copies[:, None] & (j == last[:, None]), page_of[:, None], new)
    taken = (n_copies - n_given).clamp(min=0)
    # references, and the pages that lose their last: the last entry of the last request on top of none
    change = old != new
    refs = c["refs"]
    refs.index_add_(0, old.clamp(min=0).view(-1).long(), -(change & (old >= 0)).view(-1).to(torch.int32))
    refs.index_add_(0, new.clamp(min=0).view(-1).long(), (change & (new >= 0)).view(-1).to(torch.int32))
    drop = (change & (old >= 0)).view(-1).nonzero().view(-1)
    pages = old.view(-1)[drop].long()
    final = torch.full((len(refs),), -1, device=dev).scatter_reduce(0, pages, drop, "amax")
    gone = pages[(refs[pages] == 0) & (final[pages] == drop)].to(torch.int32)
    c["free_pages"][n_free - taken + torch.arange(len(gone), device=dev)] = gone.flip(0)
    c["n_free"][0] = n_free - taken + len(gone)
    to, of = page_of[copies].long(), was[copies].long()
    for name in ("k", "v"):
        codes = c[name + "_codes"].view(torch.uint8)
        codes[to] = codes[of]
        c[name + "_scales"][to] = c[name + "_scales"][of]
    c["table"][slots] = new
    c["lengths"][slots] = after.to(torch.int32)
    return dict(c)


# ---------------------------------------------------------------------------------- one pass

def run(s):
    case, kind = s["case"], s["case"]["kind"]
    if not own:
        return _prefix(s) if kind == "prefix" else _select(s) if kind == "select" else _reorder(s)
    import dlrm_embedding_interaction_gb300 as dl
    if kind == "prefix":
        got = {"out": torch.empty_like(s["q"])}
        if case["lse"]:
            got["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
        dl.history_prefix_attention(s["cache"], s["slots"], s["starts"], s["groups"], s["q"], got["out"],
                                    causal=case["causal"], window=case["window"], sinks=case["sinks"], lse=got.get("lse"))
        return got
    if kind == "select":
        scores, parents, tokens = dl.beam_select(s["logits"], s["scores"], s["groups"], case["width"], allowed=s.get("allowed"))
        return {"scores": scores, "parents": parents, "tokens": tokens}
    dl.history_reorder(s["cache"], s["slots"], s["parents"])
    return dict(s["pool"])


# ---------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    kind = case["kind"]
    if kind == "reorder":
        return None  # pages move, nothing is computed
    s = prepare(case, seed)
    beams = _beams(case)
    if kind == "select":
        best = torch.full((len(beams), case["width"]), -math.inf, dtype=torch.float64, device="cuda")
        at = 0
        for u, n in enumerate(beams):
            values = []
            for r in range(at, at + n):
                x = s["logits"][r]
                x = (x[s["allowed"][r]] if "allowed" in s else x).double()
                if len(x):
                    x = x - torch.logsumexp(x, 0) + s["scores"][r].double()
                    values.append(x.topk(min(len(x), case["width"])).values)
            if values:
                x = torch.sort(torch.cat(values), descending=True).values[: case["width"]]
                best[u, : len(x)] = x
            at += n
        return {"scores": best, "parents": None, "tokens": None}
    c, queries, group, page = s["pool"], case["queries"], case["heads"] // case["kv_heads"], case["page"]
    window, sinks = case["window"], case["sinks"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    lens = [n + case["new"] for n, b in zip(_lengths(case), beams) for _ in range(b)]
    for b, n in enumerate(lens):
        ids = c["table"][b, : -(-n // page)].long()
        k, v = ((c[x + "_codes"].view(torch.uint8)[ids].view(E4M3).double() * c[x + "_scales"][ids][:, :, None, None].double())
                .permute(1, 0, 2, 3).reshape(case["kv_heads"], -1, case["dim"])[:, :n] for x in ("k", "v"))
        for i in range(queries):
            end = n - queries + i + 1 if case["causal"] else n
            if end <= 0:
                continue
            first = max(0, end - window) if window else 0
            near = slice(first, end)
            kept = min(sinks, first)
            kk, vv = (torch.cat([x[:, :kept], x[:, near]], 1) if kept else x[:, near] for x in (k, v))
            r = b * queries + i
            x = torch.einsum("hgd,htd->hgt", s["q"][r].double().view(-1, group, case["dim"]), kk) / math.sqrt(case["dim"])
            total = torch.logsumexp(x, 2)
            out[r] = torch.einsum("hgt,htd->hgd", torch.exp(x - total[:, :, None]), vv).reshape(-1, case["dim"])
            lse[r] = total.view(-1)
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
