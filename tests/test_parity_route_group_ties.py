"""moe_route_grouped where the kept groups hang on what fp32 cannot tell: groups with fewer usable
experts than group_top, and group scores near the smallest fp32 numbers.  The choice is the one of
fp64 arithmetic (no case below holds two scores that fp64 cannot order but for equal ones, which go
to the lower group), so ids are compared for equality."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe
from oracle import router_ref as rr

pytestmark = pytest.mark.gpu

NONE = float("-inf")


def _same_choice(dev, l, k, bias=None, **kw):
    ids, w = moe.moe_route_grouped(l.to(dev), k, None if bias is None else bias.to(dev), **kw)
    torch.cuda.synchronize()
    rid, rw = rr.route_grouped(l, k, bias, **kw)
    bad = (ids.cpu().numpy() != rid).any(1).nonzero()[0]
    assert len(bad) == 0, f"rows {bad[:5]}: {ids.cpu().numpy()[bad[:2]]} for {rid[bad[:2]]}"
    assert (np.abs(w.cpu().double().numpy() - rw) <= np.abs(rw) * 2.0 ** -20 + 2.0 ** -140).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("size,k", [(4, 2), (4, 5), (16, 8), (60, 20)])
def test_group_with_one_usable_expert(cuda_dev, score, with_bias, size, k):
    """Two groups whose best experts are equal: the one with a second expert wins by it, however little that
    adds, a logit of 0 included."""
    low = {"sigmoid": [0.0, -14.0, -40.0], "softmax": [0.0, 5.0, -30.0]}[score]
    rows = []
    for second in low:
        for top in (20.0, 20.5):
            for first in (False, True):
                l = torch.full((4 * size,), NONE)
                one, two = (size, 0) if first else (0, size)
                l[one] = top
                l[two], l[two + 1] = top, second
                l[two + 2:two + size] = second - 5.0
                l[2 * size:3 * size] = -60.0
                rows.append(l)
                bare = l.clone()  # nothing beside the compared ones
                bare[two + 2:two + size] = NONE
                bare[2 * size:3 * size] = NONE
                rows.append(bare)
    l = torch.stack(rows)
    bias = torch.zeros(4 * size) if with_bias else None
    k = min(k, size)
    _same_choice(cuda_dev, l, k, bias, score=score, n_group=4, topk_group=1, group_top=2)
    if with_bias:  # a zero of score and bias together, and biases that are equal
        _same_choice(cuda_dev, l, k, torch.full((4 * size,), 0.25), score=score, n_group=4, topk_group=1, group_top=2)
        _same_choice(cuda_dev, l, k, torch.full((4 * size,), -1e-3), score=score, n_group=4, topk_group=2, group_top=2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size,k", [(4, 3), (60, 20)])
def test_group_scores_near_the_smallest_numbers(cuda_dev, score, size, k):
    """Sums of scores about 2^-126, some terms below it: e^-86.64 is 2^-125, e^-87.34 is below 2^-126."""
    g = torch.Generator().manual_seed(4)
    l = torch.full((64, 4 * size), -300.0)
    l[:, 0] = 0.0 if score == "softmax" else -60.0  # a group that is kept in any case
    for t in range(64):
        for grp in (1, 2, 3):
            l[t, grp * size:grp * size + 2] = -86.6 - torch.rand(2, generator=g) * 1.2
    l[0, size:size + 2] = torch.tensor([-86.64, -87.35])
    l[0, 2 * size:2 * size + 2] = -87.14
    _same_choice(cuda_dev, l, k, score=score, n_group=4, topk_group=2, group_top=2)
