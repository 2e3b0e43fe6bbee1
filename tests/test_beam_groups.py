"""The groups of attention with a shared prefix, as the binding checks them (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")
import dlrm_embedding_interaction_gb300 as dl  # noqa: E402
from test_history_edges import fake  # noqa: E402, F401


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.mark.parametrize("out", [None, torch.zeros(3, 4, 64)])
@pytest.mark.parametrize("starts", [(0, 3), (0, 0), (0, 1, 3)])
def test_requests_in_no_group_are_refused(fake, starts, out):  # noqa: F811
    """Nothing would be written, and an output that the call makes holds what memory held."""
    cache, lib = fake
    slots = i32(*range(len(starts) - 1))
    with pytest.raises(ValueError, match="no group"):
        dl.history_prefix_attention(cache, slots, i32(*starts), i32(0), torch.zeros(3, 4, 64), out=out)
    assert not lib.calls


def test_no_requests_need_no_group(fake):  # noqa: F811
    cache, lib = fake
    for groups in (i32(0), i32(0, 0)):
        dl.history_prefix_attention(cache, i32(), i32(0), groups, torch.zeros(0, 4, 64))
        assert lib.calls.pop() == "history_prefix_attention"
