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
    for M, N, K in ((2 ** 32 + 5, 8, 64), (5, 2 ** 32 + 8, 64), (5, 8, 2 ** 31)):
        with pytest.raises(ValueError, match="2\\^31"):
            moe.linear_backward_workspace_size(M, N, K)
    for T, H in ((2 ** 32 + 4, 64), (4, 2 ** 31)):
        with pytest.raises(ValueError, match="2\\^31"):
            moe.finalize_backward_workspace_size(T, H)


def test_scale_is_read_at_each_call(moelib, monkeypatch):
    """A scale that the caller holds in a tensor and changes is the one of the call, not of the first call."""
    seen = []

    class Lib:
        def moe_route_grouped(self, *a):
            seen.append(a[6]._obj.scale)
            return 0

        def moe_route_grouped_backward(self, *a):
            seen.append(a[8]._obj.scale)
            return 0

    monkeypatch.setattr(moe, "lib", Lib)
    monkeypatch.setattr(moe, "_launch", lambda stream: (-1, None))  # (the tensors below are the host's)
    logits, w, ids = torch.zeros((4, 16)), torch.zeros((4, 2)), torch.zeros((4, 2), dtype=torch.int32)
    scale = torch.tensor(1.5)
    for want in (1.5, 3.0):
        moe.moe_route_grouped(logits, 2, scale=scale)
        moe.moe_route_grouped_backward(w, logits, ids, scale=scale)
        assert seen[-2:] == [want, want]
        scale.mul_(2)
