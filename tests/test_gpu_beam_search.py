"""The beam search example on the GPU: it runs, and a search that is wide enough to leave
nothing out finds every item, with the probabilities of a decoder without a cache."""
import importlib.util
import os

import pytest

import beam_ref
import test_gpu_beams as base

torch = pytest.importorskip("torch")
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    from dlrm_embedding_interaction_gb300 import build
    build.build()
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location("beam_search", os.path.join(ROOT, "examples", "beam_search.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_example_runs(example, capsys):
    items, scores = example.main()
    assert "64 users" in capsys.readouterr().out
    assert items.shape == (64, 16) and (items >= 0).all()
    assert all(len(set(row.tolist())) == 16 for row in items)
    assert (scores[:, :-1] >= scores[:, 1:]).all() and (scores < 0).all()


def plain(r, pool, slot, codes):
    """Log-probabilities of items (codes: (items, levels)) after a history, in 64 bits but
    for the cache's own 8 bits: pool's slot 1 becomes each beam in turn."""
    f = lambda x: torch.from_numpy(base.f64(x)) if isinstance(x, torch.Tensor) else torch.from_numpy(x)   # noqa: E731
    cat, group, out = r.catalogue, r.heads // r.kv_heads, []
    for item in codes.tolist():
        x, node, total = r.begin, 0, 0.0
        pool.fork([slot], [0], True)
        for level in range(cat.levels):
            k, v = (f(y) for y in pool.events(0))
            q = (f(x) @ f(r.q).t()).view(r.heads, r.head_dim)
            s = torch.einsum("hd,nhd->nh", q, k.repeat_interleave(group, 1)) * r.head_dim ** -0.5
            found = torch.einsum("nh,nhd->hd", s.softmax(0), v.repeat_interleave(group, 1)).reshape(-1)
            logits = (f(x) + found @ f(r.o).t()) @ f(r.head[level]).t()
            logits[~cat.allowed[level][node].cpu()] = -float("inf")
            total += logits.log_softmax(0)[item[level]].item()
            node = int(cat.child[level][node, item[level]])
            x = r.codes[level][item[level]]
            pool.append([0], [0, 1], [base.f64(y) for y in r._events(x[None])])
        pool.release([0])
        out.append(total)
    return torch.tensor(out)


def test_a_wide_search_finds_every_item(example):
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    codes = torch.randint(5, (40, 3), generator=g, device="cuda").unique(dim=0)
    r = example.BeamRetriever(example.Catalogue(codes, 5), n_users=3, width=64, max_events=200, heads=4, kv_heads=2,
                              head_dim=32, page_tokens=32)
    starts = torch.tensor([0, 130, 137, 201], dtype=torch.int32, device="cuda")
    events = torch.randn(201, r.dim, generator=g, device="cuda")
    users = torch.arange(3, dtype=torch.int32, device="cuda")
    r.load(users, events, starts)
    free = int(r.cache.n_free)
    kv, pool = r._events(events), beam_ref.Pool(40, 4, 8, 2, 32, 32)
    items, scores = r.retrieve(users)
    assert r.cache.error() == dl.OK and int(r.cache.n_free) == free
    for u in range(3):
        assert sorted(items[u].tolist()) == [-1] * (64 - len(codes)) + list(range(len(codes)))
        there = items[u] >= 0
        assert abs(scores[u][there].double().exp().sum().item() - 1) < 1e-4   # 40 rounded probabilities
        mine = slice(int(starts[u]), int(starts[u + 1]))
        pool.append([u + 1], [0, mine.stop - mine.start], [base.f64(y[mine]) for y in kv])
        want = plain(r, pool, u + 1, codes)
        # fp32 steps are off by some 2^-18. One may turn a key's code to the next one: a step
        # of 2^-3 of a component below 4, times as much of a query over 32^(1/2) moves a score
        # by 2^-2 at most, a row found among 7 events or more by 2^-4 of one value's part
        assert (scores[u][there].cpu().double() - want[items[u][there].cpu()]).abs().max() < 2.0 ** -4
    again = r.retrieve(users)
    assert torch.equal(again[0], items) and torch.equal(again[1], scores)
