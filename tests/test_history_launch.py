"""The launch code of the event-history operators on the host, against a stand-in for the
CUDA runtime (fake_cudart.cpp): no kernel runs, no GPU is needed."""
import ctypes
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402
from dlrm_embedding_interaction_gb300 import history  # noqa: E402
from test_history_checks import attention, pool  # noqa: E402

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    """The library's own objects over the stand-in."""
    from dlrm_embedding_interaction_gb300 import build
    if not (shutil.which("g++") and os.path.exists(build.nvcc())):
        pytest.skip("no compilers")
    build.build()
    out = str(tmp_path_factory.mktemp("fake") / "libfake.so")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    objects = [os.path.join(build.OBJ_DIR, os.path.basename(s)[:-3] + ".o") for s in build.sources()]
    # what the stand-in lacks is not called here: left unresolved
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I", include, "-Wl,-z,lazy",
                        "-Wl,-Bsymbolic", os.path.join(HERE, "fake_cudart.cpp"), *objects, "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    lib = ctypes.CDLL(out, mode=os.RTLD_LAZY | os.RTLD_LOCAL)
    history._bind(lib)
    return lib


@pytest.mark.parametrize("head_dim", [32, 64, 128])
@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("rows", [5, 5000])
def test_attention_launches_on_every_device_of_a_process(lib, head_dim, dtype, rows):
    """The shared memory that a kernel may take is an attribute of each device."""
    h = ctypes.byref(pool(head_dim=head_dim))
    ld = 4 * head_dim
    a = ctypes.byref(attention(head_dim=head_dim, dtype=dtype, q_rows=rows, k_rows=rows, ld_q=ld,
                               ld_q_head=head_dim, ld_out=ld, ld_out_head=head_dim, ld_k=ld // 2,
                               ld_k_head=head_dim, ld_v=ld // 2, ld_v_head=head_dim))
    for device in (0, 1, 0, 2, 63, 64, 65):
        lib.fake_set_device(device)
        before = lib.fake_launches()
        assert lib.history_attention(h, a, None) == dl.OK, device
        assert lib.window_attention(a, None) == dl.OK, device
        assert lib.fake_launches() == before + 2
    lib.fake_set_device(0)


@pytest.mark.parametrize("rows,heads,ld,ld_head,good", [
    (5, 4, 256, 64, True), (5, 4, 0, 64, False), (5, 4, 256, 0, False), (5, 4, 63, 64, False),
    (1, 4, 0, 64, True), (5, 1, 64, 0, True), (1, 1, 0, 0, True), (5, 4, 64, 320, True), (5, 4, 64, 64, False),
    (5, 4, 64, 319, False), (5, 4, 255, 64, False), (5, 4, 300, 70, True), (4, 2, 128, 192, True),
    (4, 2, 128, 191, False), (4, 2, 128, 193, False), (4, 8, 128, 192, False), (1 << 20, 4, 256, 64, True),
    (1 << 20, 2, 128, 64, True), (1 << 20, 4, 128, 64, False)])
def test_outputs_that_lie_over_one_another_are_refused(lib, rows, heads, ld, ld_head, good):
    """Against every pair of places, for few rows."""
    if rows < 100:
        at = sorted(t * ld + h * ld_head for t in range(rows) for h in range(heads))
        assert good == all(b - a >= 64 for a, b in zip(at, at[1:]))
    h = ctypes.byref(pool(n_heads=1))
    a = ctypes.byref(attention(q_rows=rows, k_rows=rows, n_heads=heads, n_kv_heads=1, ld_q=64 * heads,
                               ld_q_head=64, ld_k=64, ld_k_head=64, ld_v=64, ld_v_head=64, ld_out=ld,
                               ld_out_head=ld_head))
    want = dl.OK if good else dl.ERR_INVALID_ARG
    assert lib.history_attention(h, a, None) == want
    assert lib.window_attention(a, None) == want


@pytest.mark.parametrize("n_heads", [1, 16384, 32768, 131071])
@pytest.mark.parametrize("batch", [1, 200])
def test_pages_of_any_size_can_be_forked(lib, n_heads, batch):
    """A page of 2^29 bytes a side has more pieces to copy than a grid has rows."""
    h = ctypes.byref(pool(n_heads=n_heads, page_tokens=128, head_dim=128, n_slots=300))
    assert lib.history_append(h, 0x10000, 0x10000, batch, 0x10000, 128, 128, 0x10000, 128, 128, 5, 0,
                              None) == dl.OK
    for call in (lib.history_fork, lib.history_copy):
        assert call(h, 0x10000, 0x10000, batch, None) == dl.OK
    assert lib.history_compact(h, None) == dl.OK


@pytest.mark.parametrize("change", [dict(k_rows=2 ** 31 - 1), dict(k_rows=2 ** 31 - 256), dict(k_rows=2 ** 62),
                                    dict(q_rows=2 ** 31 - 1), dict(q_rows=2 ** 31 - 256),
                                    dict(q_rows=2 ** 30, n_heads=2), dict(q_rows=2 ** 62, n_heads=2),
                                    dict(q_rows=2 ** 62, n_heads=4), dict(q_rows=2 ** 63 - 1)])
def test_row_counts_near_2_to_the_31_are_refused(lib, change):
    """A step past the last tile would leave 32 bits, and a kernel's loop over keys would
    start again from below zero."""
    h = ctypes.byref(pool(n_heads=1))
    good = dict(n_heads=1, n_kv_heads=1, ld_q=256, ld_q_head=64, ld_out=256, ld_out_head=64, q_rows=3, k_rows=5)
    small = ctypes.byref(attention(**good))
    assert lib.window_attention(small, None) == dl.OK and lib.history_attention(h, small, None) == dl.OK
    a = ctypes.byref(attention(**dict(good, **change)))
    assert lib.window_attention(a, None) == dl.ERR_UNSUPPORTED
    if "q_rows" in change:
        assert lib.history_attention(h, a, None) == dl.ERR_UNSUPPORTED
