"""moe_grouped_linear and its gradients where sorted rows lie outside every group, in front of the first and behind the
last: neither they nor their slots are read, nor their rows of an output written.

Tolerances: as in test_parity_grouped."""
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe
from test_parity_grouped import BF, ORDERS, Problem

pytestmark = pytest.mark.gpu


class Outside(Problem):
    """`front` and `over` sorted rows of no group, with values that are NaN and slots on the device that are out of range."""

    def __init__(self, counts, N, K, front, over, orders, poison):
        x_rows, rows, d_rows = ("slot" if o == "token" else o for o in orders)
        super().__init__(counts, N, K, 1, BF, x_rows, rows, d_rows, over=front + over)
        nan = float("nan")
        g = torch.Generator().manual_seed(front + over)
        self.x, self.dout = (torch.randn(t.shape, generator=g).to(BF) for t in (self.x, self.dout))
        self.slots = torch.randperm(self.S, generator=g).to(torch.int32)
        self.offsets = self.offsets + front
        self.out = torch.tensor([*range(front), *range(self.S - over, self.S)], dtype=torch.long)
        for t, order in ((self.x, x_rows), (self.dout, d_rows)):
            t[self.slots[self.out].long() if order == "slot" else self.out] = nan
        self.poison = poison

    def dev(self, dev):
        x, w, o, slots = super().dev(dev)
        if slots is not None:
            slots[self.out.to(dev)] = self.poison
        return x, w, o, slots


# small groups, whose rows are fetched where they are, and larger ones, which are put in order first
@pytest.mark.parametrize("counts", [[3, 0, 5], [20, 24, 0, 26], [70, 0, 90], [300, 129, 0]])
@pytest.mark.parametrize("front,over", [(5, 0), (0, 13), (40, 70)])
@pytest.mark.parametrize("orders", ORDERS)
def test_rows_and_slots_outside_the_groups(cuda_dev, counts, front, over, orders):
    for poison in (-1, 1 << 30):
        p = Outside(counts, 136, 72, front, over, orders, poison)
        p.check_forward(p.forward(cuda_dev))
        p.check_backward(*p.backward(cuda_dev, torch.float32))
        assert moe.moe_device_status() == moe.MOE_OK


def test_many_rows_in_front_off_128_bytes(cuda_dev):
    """Sorted rows that are moved to a pitch of 128 bytes."""
    p = Outside([1000, 0, 940], 2072, 2056, 33, 72, ("sorted", "sorted", "sorted"), -1)
    assert moe.grouped_linear_workspace_size(p.S, p.E, p.N, p.K) > 0
    p.check_forward(p.forward(cuda_dev))
    p.check_backward(*p.backward(cuda_dev))
    assert moe.moe_device_status() == moe.MOE_OK
