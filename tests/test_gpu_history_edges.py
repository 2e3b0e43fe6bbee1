"""Event-history operators on the GPU at the edges of their definitions: what a refused
request leaves behind, the largest windows, empty and infinite scores, layouts and
streams, and waits that run out. Bounds as in test_gpu_history.py."""
import numpy as np
import pytest

import history_ref as ref
import test_gpu_history as base

torch = pytest.importorskip("torch")
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402

pytestmark = pytest.mark.gpu
i32, f64, rows, make, fill, same_state, starts_of = (
    base.i32, base.f64, base.rows, base.make, base.fill, base.same_state, base.starts_of)
TYPES = base.TYPES


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    from dlrm_embedding_interaction_gb300 import build
    build.build()
    torch.cuda.set_device(0)


# ------------------------------------------------------------------ refused requests

def test_a_refused_copy_leaves_nothing_behind():
    rng = np.random.default_rng(40)
    cache, pool = make(32, 8, 3, 2, 32, 32)
    fill(cache, pool, rng, [0, 1], [40, 70])

    def copy(src, dst):
        dl.history_copy(cache, i32(src), i32(dst))
        pool.fork(src, dst, False)
        same_state(cache, pool)

    copy([8], [5])                                  # no such source
    assert cache.error() == dl.ERR_INDEX_OOB
    copy([0, 1], [4, 5])                            # slot 5 at a higher index than before
    assert cache.error() == dl.OK
    copy([-1, 0, 9], [6, 6, 7])                     # 6 is written twice: the first counts, and is refused
    assert cache.error() == dl.ERR_INDEX_OOB
    copy([0, 1, 0], [2, 7, 6])
    assert cache.error() == dl.OK


@pytest.mark.parametrize("batch", [129, 1500])
def test_a_refused_fork_of_many_leaves_nothing_behind(batch):
    """Sources out of range in a fork of many requests, then appends, copies and forks
    whose slots stand at other indices."""
    rng = np.random.default_rng(batch)
    cache, pool = make(4 * batch, 2 * batch, 2, 1, 32, 32)
    fill(cache, pool, rng, [0, 1], [40, 20])
    src = np.where(rng.random(batch) < 0.5, 0, 2 * batch).tolist()
    dst = (2 + np.arange(batch)).tolist()
    dl.history_fork(cache, i32(src), i32(dst))
    pool.fork(src, dst, True)
    assert cache.error() == dl.ERR_INDEX_OOB
    dl.history_free(cache, i32(dst))
    pool.release(dst)
    same_state(cache, pool, codes=False)
    # every slot at a higher index than before, but the first
    dst = dst[-1:] + dst[:-1]
    for step in range(3):
        if step == 0:
            fill(cache, pool, rng, dst, [1] * batch)
        else:
            (dl.history_copy if step == 1 else dl.history_fork)(cache, i32([1] * batch), i32(dst))
            pool.fork([1] * batch, dst, step == 2)
        same_state(cache, pool)
        assert cache.error() == dl.OK
        dl.history_free(cache, i32(dst))
        pool.release(dst)


# ------------------------------------------------------------------ windows

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 40])
def test_the_largest_window_with_more_queries_than_events(dtype, dim, window):
    """The first rows stand before the first event: such a window's start lies below -2^31."""
    rng = np.random.default_rng(41)
    for counts, lens in (([4, 70, 300], [1, 20, 150]), ([33], [1])):
        for sinks in (0, 2, 2 ** 31 - 1):
            base.check_window(rng, counts, lens, 4, 2, dim, dtype, window, sinks)
    lens, counts = [1, 20, 150, 700], [4, 70, 300, 710]
    cache, pool = make(20, 4, 11, 2, dim, 64)
    fill(cache, pool, rng, [0, 1, 2, 3], lens)
    for n in (1, 3, 4):                             # the last: enough rows for the tensor-core kernel
        base.check_attention(cache, pool, rng, list(range(n)), counts[:n], 4, dtype, True, window, 1)
    assert cache.error() == dl.OK
