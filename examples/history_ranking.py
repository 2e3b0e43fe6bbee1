"""Ranking candidates against users' event histories with the event-history operators.

A user's past items go through one layer of windowed self-attention and are kept, as
keys and values in 8 bits, in a cache between requests. A request forks the user's
history, adds the events of its own session, lets every candidate attend over it, and
scores [candidate, <candidate, what it found>] with the interaction and a top MLP; the
fork is dropped afterwards. Run it on a GB300:

    python examples/history_ranking.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402


def starts_of(counts):
    at = torch.zeros(len(counts) + 1, dtype=torch.int32)
    at[1:] = torch.tensor(list(counts), dtype=torch.int32).cumsum(0)
    return at.cuda()


class HistoryRanker:
    """items: (rows, dim) float32 embeddings; heads * head_dim == dim."""

    def __init__(self, items, heads, n_users, max_events, window=256, sinks=4, page_tokens=64, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        dim = items.shape[1]
        self.items, self.dim, self.heads = items, dim, heads
        self.window, self.sinks = window, sinks

        def weight(n, k):
            return torch.randn(n, k, generator=g, device="cuda") * k ** -0.5

        # encoder (q, k, v), cache (k, v) and candidate (q) projections, top MLP
        self.enc = [weight(dim, dim) for _ in range(3)]
        self.kv = [weight(dim, dim) for _ in range(2)]
        self.query = weight(dim, dim)
        self.top = [(weight(64, dim + 1), torch.zeros(64, device="cuda"), dl.ACT_RELU),
                    (weight(1, 64), torch.zeros(1, device="cuda"), dl.ACT_SIGMOID)]
        # slots [0, n_users) hold histories, [n_users, 2 n_users) the forks of requests
        self.n_users = n_users
        pages = -(-max_events // page_tokens)
        self.cache = dl.HistoryCache(n_users * (pages + 2), 2 * n_users, pages + 1, heads, dim // heads,
                                     page_tokens=page_tokens)

    def _linear(self, x, w, bias=None, act=dl.ACT_NONE):
        y = torch.empty(x.shape[0], w.shape[0], device="cuda")
        dl.linear_bias_act(x, w, bias, y, act)
        return y

    def _rows(self, ids):
        """Embeddings of items: bags of one row."""
        out = torch.empty(len(ids), 1, self.dim, device="cuda")
        at = torch.arange(len(ids), dtype=torch.int64, device="cuda").unsqueeze(0)
        dl.embedding_bag_sum_multi([self.items], ids.to(torch.int64).unsqueeze(0), at, out, 1)
        return out.view(-1, self.dim)

    def _heads(self, x):
        return x.view(-1, self.heads, self.dim // self.heads)

    def encode(self, ids, starts):
        """Keys and values, (events, heads, head_dim), of ragged histories of items."""
        x = self._rows(ids)
        q, k, v = (self._heads(self._linear(x, w)) for w in self.enc)
        h = dl.window_attention(q, k, v, starts, window=self.window, sinks=self.sinks)
        return [self._heads(self._linear(h.reshape(-1, self.dim), w)) for w in self.kv]

    def load(self, users, ids, starts):
        """Replaces the histories of ``users``."""
        dl.history_free(self.cache, users)
        dl.history_append(self.cache, users, starts, *self.encode(ids, starts))

    def rank(self, users, session_ids, session_starts, candidate_ids, candidate_starts):
        """Click probabilities of the candidates of each user, whose own session
        events count and are forgotten afterwards."""
        forks = users + self.n_users
        dl.history_fork(self.cache, users, forks)
        dl.history_append(self.cache, forks, session_starts, *self.encode(session_ids, session_starts))
        x = self._rows(candidate_ids)
        q = self._heads(self._linear(x, self.query))
        found = dl.history_attention(self.cache, forks, candidate_starts, q)
        dl.history_free(self.cache, forks)
        r = torch.empty(len(x), self.dim + 1, device="cuda")
        dl.pairwise_dot_lower_tri(x, found.view(-1, 1, self.dim), r)
        for w, bias, act in self.top:
            r = self._linear(r, w, bias, act)
        return r.view(-1)


def main():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rows, dim, users = 100_000, 128, 64
    items = torch.randn(rows, dim, generator=g, device="cuda")
    ranker = HistoryRanker(items, heads=2, n_users=users, max_events=2048)

    def some(counts):
        return torch.randint(rows, (sum(counts),), generator=g, device="cuda"), starts_of(counts)

    lengths = [50 + 31 * i for i in range(users)]
    everyone = torch.arange(users, dtype=torch.int32, device="cuda")
    ranker.load(everyone, *some(lengths))
    p = ranker.rank(everyone, *some([3] * users), *some([100] * users))
    dl.history_compact(ranker.cache)
    assert ranker.cache.error() == dl.OK
    print(f"{users} users, {sum(lengths)} events, {len(p)} candidates: "
          f"probabilities {p.min():.3f} to {p.max():.3f}, "
          f"{int(ranker.cache.n_free)} of {len(ranker.cache.refs)} pages free")


if __name__ == "__main__":
    main()
