"""GELU in moe_linear over the range of its arguments.

The product is an exact one: x picks the first column of w, which holds z, so z itself reaches the
epilogue.  GELU is z times the normal distribution's part below z: for z < 0 that is exp(-z^2 / 2) times a
smooth factor.  Half of z^2 carries one rounding, 2^-24 of z^2 / 2, the product with log2 e as much and its
constant no more, which the exponential turns into 3 z^2 2^-25; its own error and that of a factor of a dozen
operations stay below 8 2^-23: within (z^2 + 1) 2^-23 + 2^-20 of the value."""
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe
from oracle import router_ref as rr

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _outputs(dev, z, act, M, dtype):
    """act(z) in fp32 for M rows of the same z [N] (bf16 or fp16 values, N a multiple of 8)."""
    N = z.numel()
    x = torch.eye(N, dtype=dtype)[:1].repeat(M, 1)  # picks the first column of w
    w = torch.zeros((N, N), dtype=dtype)
    w[:, 0] = z.to(dtype)
    out = moe.moe_linear(x.to(dev), w.to(dev), activation=act, out_dtype=F32)
    assert moe.moe_device_status() == moe.MOE_OK
    return out.cpu().double()


@pytest.mark.parametrize("M", [1, 8, 40])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_gelu_keeps_its_digits_below_zero(cuda_dev, M, dtype):
    z = torch.cat([-torch.arange(4.0, 8.0, 1 / 32), torch.arange(-4.0, 4.0, 1 / 16)]).to(dtype).double()
    ref = rr.act(z, "gelu")
    got = _outputs(cuda_dev, z, "gelu", M, dtype)
    rel = ((got - ref).abs() / ref.abs().clamp_min(1e-30)).max(0).values
    assert (rel <= (z * z + 1) * 2.0 ** -23 + 2.0 ** -20).all(), f"{float(rel.max()):.3e}"
    # (beside a residual and by columns of two and one, the other epilogues of it)
    N = 41
    x = torch.eye(48, dtype=dtype)[:1].repeat(M, 1)
    w = torch.zeros((N, 48), dtype=dtype)
    w[:, 0] = z[:N].to(dtype)
    got = moe.moe_linear(x.to(cuda_dev), w.to(cuda_dev), activation="gelu", out_dtype=F32,
                         residual=torch.zeros((M, N), device=cuda_dev)).cpu().double()
    assert ((got - ref[:N]).abs() <= ((z[:N] ** 2 + 1) * 2.0 ** -23 + 2.0 ** -20) * ref[:N].abs()).all()


def test_gelu_slope_keeps_its_digits_below_zero(cuda_dev):
    """The slope is the part below z plus z times the density, of opposite signs there: together at most 1.6 of the
    slope for z <= -2, each within (z^2 + 8) 2^-23; then half a bf16 step."""
    z = torch.arange(-8.0, -2.0, 1 / 32).to(BF).double()
    N = z.numel()
    pre = z.to(BF).repeat(3, 1)
    dx, _, _ = moe.moe_linear_backward(torch.ones((3, N), dtype=BF, device=cuda_dev),
                                       torch.zeros((3, N), dtype=BF, device=cuda_dev),
                                       torch.eye(N, dtype=BF, device=cuda_dev), pre.to(cuda_dev), "gelu", need_dw=False)
    ref = rr.act_grad(z, "gelu")
    assert moe.moe_device_status() == moe.MOE_OK
    tol = (2.0 ** -8 + 1.6 * (z * z + 8) * 2.0 ** -23) * ref.abs()
    assert ((dx.cpu().double() - ref).abs() <= tol).all()
