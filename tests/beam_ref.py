"""Plain float64 restatement of the beam search's operators, written from their definitions in
include/dlrm.h (test infrastructure, no GPU)."""
import numpy as np

import history_ref as ref


class Pool(ref.Pool):
    def reorder(self, slots, parents):
        """Returns whether there were pages enough; without them nothing changes."""
        rows, lens, n = self.table.copy(), self.lengths.copy(), len(slots)

        def there(s):
            return 0 <= s < len(lens)

        source = {}                                          # request -> slot whose history it takes, or -1
        for b, d in enumerate(slots):
            if not there(d) or d in slots[:b]:
                continue
            p = parents[b]
            source[b] = -1 if p == -1 else slots[p] if 0 <= p < n and there(slots[p]) else d

        def last(s):                                         # place and page of a last page that is not full
            j = int(lens[s]) // self.G
            return (j, rows[s, j]) if lens[s] % self.G and rows[s, j] >= 0 else (j, -1)

        keeper = {}
        for b, s in source.items():
            if s >= 0 and (s not in keeper or s == slots[b]):
                keeper[s] = b
        copies = [b for b, s in source.items() if s >= 0 and last(s)[1] >= 0 and keeper[s] != b]
        given = [last(slots[b])[1] for b in source if slots[b] not in keeper and last(slots[b])[1] >= 0]
        if len(copies) - len(given) > len(self.free):
            return False
        pages = {}
        for i, b in enumerate(copies):
            pages[b] = given[i] if i < len(given) else self.free.pop()
        was = [x.copy() for x in self.codes + self.scales]
        dropped = []
        for b, s in source.items():
            d = slots[b]
            if s == d:
                continue
            new = np.full(self.M, -1)
            if s >= 0:
                m = self.pages(lens[s])
                new[:m] = rows[s, :m]
                if b in pages:
                    j, old = last(s)
                    new[j] = pages[b]
                    for x, y in zip(self.codes + self.scales, was):
                        x[pages[b]] = y[old]
            for j in range(self.M):
                old = rows[d, j] if j < self.pages(lens[d]) else -1
                if old != new[j]:
                    if old >= 0:
                        self.refs[old] -= 1
                        dropped.append(old)
                    if new[j] >= 0:
                        self.refs[new[j]] += 1
            self.table[d] = new
            self.lengths[d] = lens[s] if s >= 0 else 0
        place = {p: i for i, p in enumerate(dropped)}
        for i in range(len(dropped) - 1, -1, -1):
            if self.refs[dropped[i]] == 0 and place[dropped[i]] == i:
                self.free.append(dropped[i])
        return True


def log_probabilities(logits, allowed=None):
    """Of each token among the row's allowed ones; -infinity for the others."""
    x = np.asarray(logits, np.float64).copy()
    if allowed is not None:
        x[~np.broadcast_to(allowed, x.shape)] = -np.inf
    top = x.max(1, keepdims=True)
    base = np.where(np.isfinite(top), top, 0.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        out = (x - base) - np.log(np.exp(x - base).sum(1, keepdims=True))   # (log n stays beside any base)
    return np.where(np.isneginf(x), -np.inf, out)


def select(logits, scores, starts, width, allowed=None):
    """scores, rows and tokens of each group, and the scores of all candidates."""
    every = log_probabilities(logits, allowed) + np.asarray(scores, np.float64)[:, None]
    every[~(np.asarray(scores, np.float64) > -np.inf)] = -np.inf
    groups, vocab = len(starts) - 1, every.shape[1]
    best = np.full((groups, width), -np.inf)
    rows, tokens = np.full((groups, width), -1), np.full((groups, width), -1)
    for g in range(groups):
        s0, s1 = starts[g], starts[g + 1]
        flat = every[s0:s1].reshape(-1)
        order = np.argsort(-flat, kind="stable")
        order = order[flat[order] > -np.inf][:width]
        best[g, :len(order)] = flat[order]
        rows[g, :len(order)] = s0 + order // vocab
        tokens[g, :len(order)] = order % vocab
    return best, rows, tokens, every
