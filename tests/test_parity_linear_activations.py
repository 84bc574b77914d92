"""The activations of moe_linear and of its gradients over the range of their arguments.

The product is an exact one: x = the identity's rows scaled to hold z in its columns, so z itself
reaches the epilogue.  GELU is z/2 erfc(-z / sqrt 2): the argument carries two roundings (of 1 / sqrt 2 and
of the product, 2^-24 each), which erfc turns into 2 u^2 + 1 times as much for u = |z| / sqrt 2 (its
logarithmic slope lies below 2 u + 1 / u), its own error is 4 last places (2^-21) and the products add two roundings: within
(z^2 + 1) 2^-23 + 2^-20 of the value."""
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


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype,big", [(BF, [20.0, 100.0, 1e4, 1e10, 5e18, 1e19, 1e20, 1e30, 3e38, float("inf")]),
                                       (HF, [20.0, 88.0, 104.0, 1000.0, 65504.0, float("inf")])])
def test_gradients_far_out(cuda_dev, act, dtype, big):
    """Far from 0 the slope is 1 or 0; a pre-activation of the type's infinity (a sum that overflowed it) has these
    slopes too.  The terms that decay are below 2^-23 there (20 e^-20 is 4e-8)."""
    z = torch.tensor([s * v for v in big for s in (1, -1)]).to(dtype)
    pre = z.repeat(3, 8)
    M, N = pre.shape
    dout = torch.linspace(-1, 1, M * N).view(M, N).to(dtype)
    w = torch.eye(N, dtype=dtype)
    x = torch.ones((M, 8), dtype=dtype)
    # dx = dz against the identity
    dx, dw, db = moe.moe_linear_backward(dout.to(cuda_dev), torch.zeros((M, N), dtype=dtype, device=cuda_dev),
                                         w.to(cuda_dev), pre.to(cuda_dev), act, need_dw=True, need_dbias=True)
    want = torch.where(pre > 0, dout.double(), 0.0)
    assert moe.moe_device_status() == moe.MOE_OK
    assert ((dx.cpu().double() - want).abs() <= want.abs() * (torch.finfo(dtype).eps / 2) + 2.0 ** -23).all()
    s = want.sum(0)
    assert ((db.cpu().double() - s).abs() <= s.abs() * torch.finfo(dtype).eps / 2 + 1e-6).all()
    # a NaN stays one
    pre[1, 2] = float("nan")
    dx, _, _ = moe.moe_linear_backward(dout.to(cuda_dev), x.new_zeros((M, N)).to(cuda_dev), w.to(cuda_dev),
                                       pre.to(cuda_dev), act, need_dw=False)
    assert torch.isnan(dx[1]).all() and torch.isfinite(dx[0]).all()
