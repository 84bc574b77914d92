"""MoELayer.router_backward where the next block reads the residual stream too: the gradient of
<out, d> + <residual_out, dr> with respect to the router's weights, and on to the gate."""
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe
from mixture_experts_layer_tokens_gb300.inputs import CONFIGS, make_inputs, scaled
from mixture_experts_layer_tokens_gb300.layer import MoELayer, MoERouter

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("rms", [True, False])
def test_gradient_through_the_residual_stream(cuda_dev, rms):
    T, H, E, k = 40, 256, 16, 3
    cfg = scaled(CONFIGS["tiny"], name="router", T=T, H=H, I=256, E=E, top_k=k, residual=True, rms=rms)
    inp = make_inputs(cfg, seed=5)
    g = torch.Generator().manual_seed(17)
    gate_w = (torch.randn((E, H), generator=g) / H ** 0.5).to(BF)
    router = MoERouter(T, gate_w.to(cuda_dev), k, score="sigmoid", n_group=4, topk_group=2, group_top=2, scale=2.5)
    layer = MoELayer(inp.to(cuda_dev), router=router, keep_residual=True)
    layer.forward(None, layer.inp.a1)
    d, dr = (torch.randn((T, H), generator=g).to(BF) for _ in range(2))
    fin, (dgw, _, da1, dl) = layer.router_backward(d.to(cuda_dev), layer.inp.a1, dresidual_out=dr.to(cuda_dev))
    torch.cuda.synchronize()
    assert moe.moe_device_status() == moe.MOE_OK

    # fp64 autograd over the same rows and choice, the normalised stream as the forward call rounded it
    y = layer.y.cpu().double().view(T, k, H)
    logits = layer.router.logits.cpu().double().requires_grad_(True)
    p = torch.sigmoid(logits).gather(1, layer.topk_ids.cpu().long())
    w = p / p.sum(1, keepdim=True) * 2.5
    w.retain_grad()
    o = (w[:, :, None] * y).sum(1) + inp.residual.double()
    s = o + (layer.residual_out.cpu().double() - o).detach()
    out = s * (s.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt() * inp.rms_weight.double() if rms else s
    ((out * d.double()).sum() + (s * dr.double()).sum()).backward()
    near = lambda got, ref, tol: float((got.cpu().double() - ref).norm() / ref.norm()) <= tol  # noqa: E731
    # fp32 throughout (sums of 256 terms, a dozen roundings a term); then dlogits and the outputs to bf16
    assert near(fin[1], w.grad, 2.0 ** -16)
    assert near(dl, logits.grad, 2.0 ** -15)
    assert near(dgw, logits.grad.T @ inp.a1.double(), 2 * 2.0 ** -8 + 2.0 ** -14)
    assert near(da1, logits.grad @ gate_w.double(), 2 * 2.0 ** -8 + 2.0 ** -14)
    # without it: the gradient of out alone
    plain = layer.router_backward(d.to(cuda_dev), layer.inp.a1)[0]
    zero = layer.router_backward(d.to(cuda_dev), layer.inp.a1, dresidual_out=torch.zeros_like(dr).to(cuda_dev))[0]
    assert all(torch.equal(a, b) for a, b in zip(plain, zero) if a is not None)  # (no dy, without a norm no drms)
