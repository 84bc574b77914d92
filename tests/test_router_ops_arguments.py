"""Arguments that ctypes would cut to 32 bits without a word, and configurations that a cache may not keep: no
GPU needed."""
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe


@pytest.mark.parametrize("name", ["n_group", "topk_group", "group_top"])
@pytest.mark.parametrize("value", [2 ** 32 + 1, 2 ** 31, -2 ** 31 - 1, -2 ** 32 + 1])
def test_route_config_refuses_what_does_not_fit(name, value):
    with pytest.raises(ValueError, match="2\\^31"):
        moe.route_config(**{name: value})
    with pytest.raises(ValueError, match="2\\^31"):
        moe.moe_route_grouped(torch.zeros((4, 16)), 2, **{name: value})
    assert getattr(moe.route_config(**{name: 2 ** 31 - 1}), name) == 2 ** 31 - 1


def test_workspace_sizes_refuse_what_does_not_fit(moelib):
    for M, N, K in ((2 ** 32 + 5, 8, 64), (5, 2 ** 32 + 8, 64), (5, 8, 2 ** 31), (-2 ** 32 + 5, 8, 64)):
        with pytest.raises(ValueError, match="2\\^31"):
            moe.linear_backward_workspace_size(M, N, K)
    for T, H in ((2 ** 32 + 4, 64), (4, 2 ** 31), (4, -2 ** 32 + 64)):
        with pytest.raises(ValueError, match="2\\^31"):
            moe.finalize_backward_workspace_size(T, H)


@pytest.fixture
def calls(monkeypatch):
    """The configurations that reach the library, which runs nothing."""
    seen = []

    class Lib:
        def moe_route_grouped(self, *a):
            seen.append(a[6]._obj)
            return 0

        def moe_route_grouped_backward(self, *a):
            seen.append(a[8]._obj)
            return 0

    monkeypatch.setattr(moe, "lib", Lib)
    monkeypatch.setattr(moe, "_launch", lambda stream: (-1, None))  # (the tensors below are the host's)
    return seen


LOGITS, WEIGHTS, IDS = torch.zeros((4, 16)), torch.zeros((4, 2)), torch.zeros((4, 2), dtype=torch.int32)


def test_scale_is_read_at_each_call(calls):
    """A scale that the caller holds in a tensor and changes is the one of the call, not of the first call."""
    scale = torch.tensor(1.5)
    for want in (1.5, 3.0):
        moe.moe_route_grouped(LOGITS, 2, scale=scale)
        moe.moe_route_grouped_backward(WEIGHTS, LOGITS, IDS, scale=scale)
        assert [c.scale for c in calls[-2:]] == [want, want]
        scale.mul_(2)


@pytest.mark.parametrize("name", ["n_group", "topk_group", "group_top"])
def test_group_counts_are_read_at_each_call(calls, name):
    count = torch.tensor(1)
    for want in (1, 2):
        moe.moe_route_grouped(LOGITS, 2, **{name: count})
        assert getattr(calls[-1], name) == want
        count.mul_(2)
    with pytest.raises(TypeError):
        moe.moe_route_grouped(LOGITS, 2, **{name: 2.0})
