"""The gradients of moe_linear's activations over the range of their arguments."""
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


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
