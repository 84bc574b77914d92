"""moe_rmsnorm of rows whose squares vanish in fp32, with an eps of 0 or next to it.

Tolerances: as in test_parity_rmsnorm (the rows are multiplied by a power of 2, which rounds nothing)."""
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe
from test_parity_rmsnorm import BF, _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-38, 1e-30, 7e-25, 1e-24, 1e-20])
@pytest.mark.parametrize("T,H", [(8, 256), (40, 7168), (300, 72), (1200, 1000), (2304, 1032)])
def test_small_values(cuda_dev, T, H, eps):
    """Rows from the smallest values of bf16 to ordinary ones, side by side."""
    x, res, w = _inputs(T, H)
    for residual in (None, res):
        v = x.clone()
        by = torch.exp2(torch.linspace(-126, 0, T).round())[:, None]
        v, r = (v.float() * by).to(BF), None if residual is None else (residual.float() * by).to(BF)
        for quant in ("fp8", "fp8_token"):
            outs = moe.moe_rmsnorm(v.to(cuda_dev), w.to(cuda_dev), residual=None if r is None else r.to(cuda_dev), eps=eps,
                                   quant=quant)
            _check(outs, v, r, w, quant, eps=float(torch.tensor(eps)))  # (as the call takes it, in fp32)


def test_a_row_of_zeros_without_eps(cuda_dev):
    """0 / 0 is NaN, in that row alone; with the smallest eps it is 0."""
    x, _, w = _inputs(5, 512, residual=False)
    x[2] = 0
    rows = [0, 1, 3, 4]
    n = moe.moe_rmsnorm(x.to(cuda_dev), w.to(cuda_dev), eps=0.0)[0].cpu()
    assert torch.isnan(n[2]).all() and torch.isfinite(n[rows]).all()
    n = moe.moe_rmsnorm(x.to(cuda_dev), w.to(cuda_dev), eps=1e-45)[0].cpu()
    assert (n[2] == 0).all() and torch.isfinite(n[rows]).all()
