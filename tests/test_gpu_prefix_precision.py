"""Attention with a shared prefix: the bits that its weights carry (include/dlrm.h), at sizes
where history_attention's own way would be another. Bounds as in test_gpu_beams.py, whose 2^-16 V
for weights of 22 bits holds for fp16 rows, too: the other factors of its products are exact
(fp16 queries, 8-bit codes)."""
import numpy as np
import pytest

import history_ref as ref
import test_gpu_beams as base

torch = pytest.importorskip("torch")
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402

pytestmark = pytest.mark.gpu
f64, i32, starts_of = base.f64, base.i32, base.starts_of


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    from dlrm_embedding_interaction_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def rounded_weights(q, k, v, scale):
    """Rows over all events with weights of 11 bits, the softmax's sum in full: what a product
    with fp16 weights and without their rests makes."""
    out = np.zeros(q.shape)
    group = q.shape[1] // k.shape[1]
    for h in range(q.shape[1]):
        x = (q[:, h] @ k[:, h // group].T) * scale
        w = np.exp2((x - x.max(1, keepdims=True)) * np.log2(np.e))
        out[:, h] = w.astype(np.float16).astype(np.float64) @ v[:, h // group] / w.sum(1, keepdims=True)
    return out


@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("users,beams,queries,group", [(40, 4, 1, 1), (40, 8, 1, 1), (6, 24, 1, 2), (4, 5, 7, 4)])
@pytest.mark.parametrize("length", [5, 40])
def test_fp16_rows_have_weights_of_22_bits(dim, users, beams, queries, group, length):
    """Up to 8 rows a group, whose rests lie in the other rows of a product, and more, whose rests
    have one of their own. Values are 1 and -1, so that many outputs are small, and what weights
    round is not hidden by the outputs' own rounding."""
    rng = np.random.default_rng(dim + beams + length)
    n = users * beams
    cache, pool, slots, groups = base.beams(rng, [length] * users, [beams] * users, [0] * n, 1, dim, 32, spare=n)
    k = 0.5 * torch.from_numpy(rng.standard_normal((4 * n, 1, dim))).float().cuda()
    v = torch.from_numpy(np.sign(rng.standard_normal((4 * n, 1, dim)))).float().cuda()
    own = [4 * i for i in range(n + 1)]
    dl.history_append(cache, i32(slots), i32(own), k, v)
    pool.append(slots, own, (f64(k), f64(v)))
    cache.v_codes.view(torch.uint8)[:] = torch.where(cache.v_codes.float() < 0, 0xb8, 0x38).to(torch.uint8)   # -1, 1
    cache.v_scales.fill_(1.0)
    pool.codes[1][:] = cache.v_codes.view(torch.uint8).cpu().numpy()
    pool.scales[1][:] = 1.0
    at = [queries * i for i in range(n + 1)]
    q = base.rows(rng, at[-1], group, dim, "fp16", 0.3)
    out = f64(dl.history_prefix_attention(cache, i32(slots), i32(at), i32(groups), q))
    assert cache.error() == dl.OK
    told = False
    for b, s in enumerate(slots):
        rows = f64(q[at[b]:at[b + 1]])
        ks, vs = pool.events(s)
        assert len(ks) == length + 4 and (np.abs(vs) == 1).all()
        want, _ = ref.attention(rows, ks, vs, dim ** -0.5, False, 0, 0)
        tol = 2.0 ** -16 + base.half_ulp("fp16") * np.abs(want)
        assert (np.abs(out[at[b]:at[b + 1]] - want) <= tol).all(), (b, np.abs(out[at[b]:at[b + 1]] - want).max())
        told |= (np.abs(rounded_weights(rows, ks, vs, dim ** -0.5) - want) > tol).any()
    assert told                                   # weights of 11 bits would not pass


@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("queries,beams", [(64, 16), (512, 2), (70, 9)])
@pytest.mark.parametrize("cut", ["groups", "each"])
@pytest.mark.parametrize("causal", [False, True])
def test_bf16_requests_of_many_rows(dim, queries, beams, cut, causal):
    """Requests of 64 rows and more and 4096 in all, for which history_attention has weights of 8
    bits: here they have 11, with histories that are shared and with a request a group."""
    rng = np.random.default_rng(dim + queries)
    n = 2 * beams
    cache, pool, slots, groups = base.beams(rng, [300, 37], [beams, beams], [3 + i % 40 for i in range(n)], 2, dim, 64)
    groups = groups if cut == "groups" else list(range(n + 1))
    at = [queries * i for i in range(n + 1)]
    q = base.rows(rng, at[-1], 4, dim, "bf16", 0.3)
    lse = torch.empty(q.shape[:2], device="cuda")
    out = dl.history_prefix_attention(cache, i32(slots), i32(at), i32(groups), q, causal=causal, lse=lse)
    for b in sorted({0, 1, beams, n - 1}):
        a, e = at[b], at[b + 1]
        if causal:                                # the last rows stand at the last events
            few = slice(e - 40, e)
            base.check_rows(pool, [slots[b]], [0, 40], q[few], out[few], lse[few], "bf16", causal=True)
        else:
            few = slice(a, a + 60)
            base.check_rows(pool, [slots[b]], [0, 60], q[few], out[few], lse[few], "bf16")
    assert cache.error() == dl.OK
