"""Finding items by beam search over their codes, next to users' event histories.

An item is a tuple of codes, one a level (such as the cluster of its embedding, then the
cluster inside that one, and so on). A small decoder says the next code from the user's
past events and the codes so far: the history is read through attention, and each chosen
code becomes an event that only its own beam sees. All beams of a user are forks of the
user's history, so its pages are held, and read, once for all of them. A step is

    best continuations (beam_select, where the catalogue allows them)
    -> beams that continue others (history_reorder)
    -> the chosen codes' keys and values (history_append)
    -> what the beams find (history_prefix_attention)

and nothing in it waits for the host. Run it on a GB300:

    python examples/beam_search.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402


class Catalogue:
    """Which codes continue which: codes is (items, levels), each below n_codes."""

    def __init__(self, codes, n_codes):
        self.n_codes, self.levels = n_codes, codes.shape[1]
        self.allowed, self.child = [], []
        node, nodes = torch.zeros(len(codes), dtype=torch.int64, device=codes.device), 1
        for level in range(self.levels):
            key = node * n_codes + codes[:, level]
            found, node = key.unique(return_inverse=True)
            child = torch.zeros(nodes * n_codes, dtype=torch.int64, device=codes.device)
            child[found] = torch.arange(len(found), device=codes.device)
            allowed = torch.zeros(nodes * n_codes, dtype=torch.bool, device=codes.device)
            allowed[found] = True
            self.child.append(child.view(nodes, n_codes))
            self.allowed.append(allowed.view(nodes, n_codes))
            nodes = len(found)
        self.item = torch.zeros(nodes, dtype=torch.int64, device=codes.device)
        self.item[node] = torch.arange(len(codes), device=codes.device)


class BeamRetriever:
    """heads query heads over kv_heads; slots [0, n_users) of the cache hold the users'
    histories, the following n_users * width ones their beams."""

    def __init__(self, catalogue, n_users, width, max_events, heads=8, kv_heads=2, head_dim=64, page_tokens=64, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        dim = heads * head_dim

        def weight(n, k):
            return torch.randn(n, k, generator=g, device="cuda") * k ** -0.5

        self.catalogue, self.n_users, self.width, self.dim = catalogue, n_users, width, dim
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.codes = torch.randn(catalogue.levels, catalogue.n_codes, dim, generator=g, device="cuda")
        self.begin = torch.randn(dim, generator=g, device="cuda")
        self.q, self.o = weight(dim, dim), weight(dim, dim)
        self.kv = [weight(kv_heads * head_dim, dim) for _ in range(2)]
        self.head = [weight(catalogue.n_codes, dim) for _ in range(catalogue.levels)]
        # whole pages are shared, and each beam has its last one, and one more, to itself
        pages = -(-max_events // page_tokens)
        self.cache = dl.HistoryCache(n_users * (pages + 3 * width), n_users * (1 + width), pages + 1, kv_heads,
                                     head_dim, page_tokens=page_tokens)

    def _linear(self, x, w):
        y = torch.empty(x.shape[0], w.shape[0], device="cuda")
        dl.linear_bias_act(x, w, None, y, dl.ACT_NONE)
        return y

    def _events(self, x):
        return [self._linear(x, w).view(-1, self.kv_heads, self.head_dim) for w in self.kv]

    def load(self, users, events, starts):
        """Replaces the histories of ``users`` by ragged rows (events, dim)."""
        dl.history_free(self.cache, users)
        dl.history_append(self.cache, users, starts, *self._events(events))

    def retrieve(self, users):
        """The ``width`` most probable items of each user and their log-probabilities, best
        first, of those that the search met: (len(users), width) each, -1 past the last."""
        n, W, cat = len(users), self.width, self.catalogue
        beams = (self.n_users + users.view(-1, 1) * W + torch.arange(W, dtype=torch.int32, device="cuda")).view(-1)
        at = torch.arange(n * W + 1, dtype=torch.int32, device="cuda")
        groups = at[::W].contiguous()
        dl.history_fork(self.cache, users.repeat_interleave(W), beams)
        # the first step is the users' own: a beam each
        x = self.begin.expand(n, self.dim).contiguous()
        found = dl.history_attention(self.cache, users, at[:n + 1], self._linear(x, self.q).view(n, self.heads, -1))
        scores, starts = None, at[:n + 1]
        node = torch.zeros(n, dtype=torch.int64, device="cuda")
        for level in range(cat.levels):
            logits = self._linear(x + self._linear(found.reshape(-1, self.dim), self.o), self.head[level])
            best, rows, tokens = dl.beam_select(logits, scores, starts, W, allowed=cat.allowed[level][node])
            scores, rows, tokens = best.view(-1), rows.view(-1), tokens.view(-1)
            some = rows.clamp(min=0).long(), tokens.clamp(min=0).long()   # (a beam that is none stays at -inf)
            node = cat.child[level][node[some[0]], some[1]]
            if level == cat.levels - 1:
                break
            if level > 0:                           # (the first beams continue the same history)
                dl.history_reorder(self.cache, beams, rows)
            x = self.codes[level][some[1]]
            dl.history_append(self.cache, beams, at, *self._events(x))
            q = self._linear(x, self.q).view(n * W, self.heads, -1)
            found = dl.history_prefix_attention(self.cache, beams, at, groups, q)
            starts = groups
        dl.history_free(self.cache, beams)
        items = torch.where(rows >= 0, cat.item[node], -1)
        return items.view(n, W), scores.view(n, W)


def main():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    users, width, n_codes, levels, n_items = 64, 16, 256, 4, 100_000
    codes = torch.randint(n_codes, (n_items, levels), generator=g, device="cuda").unique(dim=0)
    retriever = BeamRetriever(Catalogue(codes, n_codes), users, width, max_events=2048)
    lengths = torch.tensor([0] + [50 + 31 * i for i in range(users)], device="cuda")
    everyone = torch.arange(users, dtype=torch.int32, device="cuda")
    starts = lengths.cumsum(0).int()
    retriever.load(everyone, torch.randn(int(starts[-1]), retriever.dim, generator=g, device="cuda"), starts)
    items, scores = retriever.retrieve(everyone)
    assert retriever.cache.error() == dl.OK
    print(f"{users} users, {int(starts[-1])} events, {len(codes)} items of {levels} codes: best {width} of each, "
          f"log-probabilities {scores.min():.3f} to {scores.max():.3f}, "
          f"{int(retriever.cache.n_free)} of {len(retriever.cache.refs)} pages free")
    return items, scores


if __name__ == "__main__":
    main()
