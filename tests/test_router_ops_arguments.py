"""Arguments that ctypes would cut to 32 bits without a word: no GPU needed."""
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
