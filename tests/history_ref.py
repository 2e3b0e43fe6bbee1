"""Plain float64 restatement of the event-history operators, written from their
definitions in include/dlrm.h (test infrastructure, no GPU)."""
import numpy as np


def e4m3_values():
    """The value of each of the 256 codes (NaN for 0x7f and 0xff)."""
    code = np.arange(256)
    sign = np.where(code & 0x80, -1.0, 1.0)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = sign * v
    v[(code & 0x7f) == 0x7f] = np.nan
    return v


VALUES = e4m3_values()
_POSITIVE = VALUES[:127]                          # codes 0 .. 0x7e, ascending


def to_e4m3(x):
    """Codes of the nearest values (ties to the even code), saturating, NaN kept."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= 448, 126, code)
    code = np.where(np.isnan(x), 0x7f, code)
    return (code | np.where(np.signbit(x) & ~np.isnan(x), 0x80, 0)).astype(np.uint8)


def scale_of(x):
    """2^e, e the least integer in [-60, 60] with |x| <= 448 * 2^e for the finite x."""
    a = np.abs(np.asarray(x, np.float64))
    a = a[np.isfinite(a)]
    top = a.max() if a.size else 0.0
    e = -60
    while e < 60 and top > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Pool:
    """The state that the operators act on, as plain arrays and lists."""

    def __init__(self, n_pages, n_slots, max_pages, n_heads, head_dim, page_tokens):
        self.G, self.M, self.P = page_tokens, max_pages, n_pages
        shape = (n_pages, n_heads, page_tokens, head_dim)
        self.codes = [np.zeros(shape, np.uint8), np.zeros(shape, np.uint8)]
        self.scales = [np.zeros(shape[:2]), np.zeros(shape[:2])]
        self.table = np.full((n_slots, max_pages), -1)
        self.lengths = np.zeros(n_slots, int)
        self.refs = np.zeros(n_pages, int)
        self.free = list(range(n_pages - 1, -1, -1))

    def pages(self, length):
        return -(-int(length) // self.G)

    def _grant(self, needs):
        """Which requests get pages: all until one finds too few."""
        ok, short, at = [], False, 0
        for n in needs:
            at += n
            ok.append(n == 0 or at <= len(self.free))
        return ok

    def append(self, slots, starts, kv):
        plan, seen = [], set()
        for b, s in enumerate(slots):
            n = starts[b + 1] - starts[b]
            good = (0 <= s < len(self.lengths) and s not in seen and n >= 0 and starts[b] >= 0
                    and starts[b + 1] <= len(kv[0])
                    and self.lengths[s] + n <= self.M * self.G)
            seen.add(s)
            need = self.pages(self.lengths[s] + n) - self.pages(self.lengths[s]) if good else 0
            plan.append((s, starts[b], n, need, good))
        ok = self._grant([p[3] for p in plan])
        for (s, t0, n, need, good), has in zip(plan, ok):
            if not good or not has:
                continue
            old = int(self.lengths[s])
            for j in range(self.pages(old), self.pages(old) + need):
                self.table[s, j] = self.free.pop()
                self.refs[self.table[s, j]] = 1
            self.lengths[s] = old + n
            for j in range(old // self.G, self.pages(old + n)):
                kept, end = max(old - j * self.G, 0), min(old + n - j * self.G, self.G)
                if end <= kept:
                    continue
                page = self.table[s, j]
                for side in (0, 1):
                    x = np.asarray(kv[side][t0 + j * self.G + kept - old: t0 + j * self.G + end - old], np.float64)
                    for h in range(x.shape[1]):
                        c, sc = self.codes[side][page, h], scale_of(x[:, h])
                        if kept:
                            was = self.scales[side][page, h]
                            sc = max(sc, was)
                            c[:kept] = to_e4m3(VALUES[c[:kept]] * (was / sc))
                        self.scales[side][page, h] = sc
                        c[kept:end] = to_e4m3(x[:, h] / sc)

    def fork(self, src, dst, share):
        rows, lens = self.table.copy(), self.lengths.copy()
        plan, seen = [], set()
        for s, d in zip(src, dst):
            good = 0 <= s < len(lens) and 0 <= d < len(lens) and d not in seen and lens[d] == 0
            seen.add(d)
            n = self.pages(lens[s]) if good else 0
            fresh = [j for j in range(n) if rows[s, j] >= 0 and (not share or (j + 1) * self.G > lens[s])]
            plan.append((s, d, n, fresh, good))
        ok = self._grant([len(p[3]) for p in plan])
        for (s, d, n, fresh, good), has in zip(plan, ok):
            if not good or not has:
                continue
            for j in range(n):
                old = rows[s, j]
                if j in fresh:
                    new = self.free.pop()
                    for x in self.codes + self.scales:
                        x[new] = x[old]
                    self.refs[new] = 1
                    self.table[d, j] = new
                else:
                    self.table[d, j] = old
                    if old >= 0:
                        self.refs[old] += 1
            self.lengths[d] = lens[s]

    def release(self, slots, window=0, sinks=0):
        out, seen = [], set()
        for s in slots:
            if not 0 <= s < len(self.lengths) or s in seen:
                continue
            seen.add(s)
            n = int(self.lengths[s])
            first, last = 0, self.pages(n)
            if window:
                first, last = min(self.pages(sinks), last), max(0, (n - window) // self.G)
            for j in range(first, last):
                if self.table[s, j] >= 0:
                    out.append(self.table[s, j])
                    self.refs[self.table[s, j]] -= 1
                    self.table[s, j] = -1
            if not window:
                self.lengths[s] = 0
        last = {p: i for i, p in enumerate(out)}
        for i in range(len(out) - 1, -1, -1):
            if self.refs[out[i]] == 0 and last[out[i]] == i:
                self.free.append(out[i])

    def compact(self):
        n = int((self.refs > 0).sum())
        holes = [p for p in range(n) if self.refs[p] == 0]
        movers = [p for p in range(n, self.P) if self.refs[p] > 0]
        for to, of in zip(holes, movers):
            for x in self.codes + self.scales:
                x[to] = x[of]
            self.refs[to], self.refs[of] = self.refs[of], 0
            self.table[self.table == of] = to
        self.free = list(range(self.P - 1, n - 1, -1))

    def events(self, slot):
        """Keys and values of a history, (events, heads, dim), from its codes."""
        out = []
        n = int(self.lengths[slot])
        for side in (0, 1):
            at = [self.table[slot, t // self.G] for t in range(n)]
            x = VALUES[self.codes[side][at, :, np.arange(n) % self.G]] * self.scales[side][at][:, :, None]
            out.append(x.reshape((n,) + self.codes[0].shape[1::2]))
        return out


def attention(q, k, v, scale, causal, window, sinks):
    """q (rows, heads, dim) over k, v (events, kv heads, dim), all float64: out, lse.
    Masked events take no part, whatever they hold."""
    rows, heads, dim = q.shape
    n, group = len(k), heads // max(k.shape[1], 1)
    out, lse = np.zeros(q.shape), np.full((rows, heads), -np.inf)
    for i in range(rows):
        pos = n - rows + i if causal else n - 1
        t = np.arange(n)
        see = t <= pos
        if window:
            see &= (t > pos - window) | (t < sinks)
        if not see.any():
            continue
        for h in range(heads):
            x = k[see, h // group] @ q[i, h] * scale
            m = x.max() if not np.isnan(x).any() else np.nan
            w = np.exp(x - m)
            out[i, h] = w @ v[see, h // group] / w.sum()
            lse[i, h] = m + np.log(w.sum())
    return out, lse
