"""The router's calls as they are used together: hidden states -> gate logits -> grouped choice ->
experts -> finalize, and the gradients back to the gate, eager, captured and on two streams."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe
from mixture_experts_layer_tokens_gb300.inputs import CONFIGS, make_inputs, scaled
from mixture_experts_layer_tokens_gb300.layer import MoELayer, MoERouter
from oracle import moe_ref, router_ref as rr
from parity_util import check_bf16

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _layer(dev, T=40, H=256, I=256, E=16, k=3, rms=True, seed=1, **router):
    cfg = scaled(CONFIGS["tiny"], name="router", T=T, H=H, I=I, E=E, top_k=k, residual=True, rms=rms)
    inp = make_inputs(cfg, seed=seed)
    g = torch.Generator().manual_seed(seed + 100)
    gate_w = (torch.randn((E, H), generator=g) / H ** 0.5).to(BF)
    gate_bias = (torch.randn((E,), generator=g) * 0.1).to(BF)
    balance = torch.randint(-50, 51, (E,), generator=g).float() * 1e-3
    kw = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2, scale=2.5)
    kw.update(router)
    r = MoERouter(T, gate_w.to(dev), k, gate_bias.to(dev), balance.to(dev), **kw)
    return cfg, inp, MoELayer(inp.to(dev), router=r), gate_w, gate_bias, balance, kw, g


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_layer_with_router_forward(cuda_dev, score):
    cfg, inp, layer, gate_w, gate_bias, balance, kw, _ = _layer(cuda_dev, score=score)
    out = layer.forward(None, layer.inp.a1)
    torch.cuda.synchronize()
    assert moe.moe_device_status() == moe.MOE_OK
    z, _, mag = rr.linear(inp.a1, gate_w, gate_bias)
    logits = layer.router.logits.cpu()
    assert (logits.double() - z).abs().le(2.0 ** -22 * (cfg.H / 16 + 16) * mag + 2.0 ** -23 * z.abs()).all()
    # from the GPU's own logits on, the choice is exact
    ids, w = rr.route_grouped(logits, cfg.top_k, balance, **kw)
    assert np.array_equal(layer.topk_ids.cpu().numpy(), ids)
    assert np.allclose(layer.topk_weights.cpu().numpy(), w, rtol=2.0 ** -20, atol=0)
    al = moe_ref.align(torch.from_numpy(ids), cfg.E, moe.MOE_BLOCK_M)
    y = moe_ref.experts(inp.a1, None, inp.w13, None, inp.w2, None, al, cfg.top_k, "bf16")
    ref = moe_ref.finalize(y, layer.topk_weights.cpu(), cfg.top_k, False, residual=inp.residual,
                           rms_weight=inp.rms_weight, eps=1e-6)
    # (element by element against the oracle's own bf16 experts rows, as the other layer tests)
    got = out.double().cpu().numpy()
    assert np.linalg.norm(got - ref.out) <= 5e-3 * np.linalg.norm(ref.out)


@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("softmax", True), ("softmax", False)])
@pytest.mark.parametrize("rms", [True, False])
def test_router_gradients_through_the_layer(cuda_dev, score, renorm, rms):
    """dout -> dweights -> dlogits -> dgate_w, dgate_bias, da1 against autograd in fp64 over the same y, logits
    and choice.  The chain's only roundings are dlogits to bf16 (half a step, 2^-8, of each term) and the
    outputs to bf16; everything else is fp32.  In the 2-norm: 2^-8 for the terms, 2^-8 for the outputs,
    2^-14 for the fp32 parts."""
    cfg, inp, layer, gate_w, gate_bias, balance, kw, g = _layer(cuda_dev, score=score, renormalize=renorm, rms=rms)
    layer.forward(None, layer.inp.a1)
    T, H, k = cfg.T, cfg.H, cfg.top_k
    dout = torch.randn((T, H), generator=g).to(BF)
    w64 = layer.topk_weights.cpu().double()
    y = layer.y.cpu().double().view(T, k, H)
    o = ((w64[:, :, None] * y).sum(1) + inp.residual.double()).to(BF)  # the residual stream, as the finalize rounds it
    fin, (dgw, dgb, da1, dl) = layer.router_backward(dout.to(cuda_dev), layer.inp.a1, o.to(cuda_dev) if rms else None)
    torch.cuda.synchronize()
    assert moe.moe_device_status() == moe.MOE_OK

    refs, _ = rr.finalize_backward(dout, layer.y.cpu(), layer.topk_weights.cpu(), k, o if rms else None,
                                   inp.rms_weight if rms else None)
    assert torch.allclose(fin[1].cpu().double(), refs["dweights"], rtol=1e-4, atol=1e-4 * refs["dweights"].abs().max())
    logits = layer.router.logits.cpu().double().requires_grad_(True)
    p = torch.sigmoid(logits) if score == "sigmoid" else torch.softmax(logits, 1)
    w = p.gather(1, layer.topk_ids.cpu().long())
    if renorm:
        w = w / w.sum(1, keepdim=True)
    want, = torch.autograd.grad((w * kw["scale"] * fin[1].cpu().double()).sum(), logits)
    near = lambda got, ref, tol: (got.cpu().double() - ref).norm() <= tol * ref.norm()  # noqa: E731
    assert near(dl, want, 2.0 ** -18)
    tol = 2 * 2.0 ** -8 + 2.0 ** -14
    assert near(dgw, want.T @ inp.a1.double(), tol)
    assert near(da1, want @ gate_w.double(), tol)
    assert near(dgb, want.sum(0), 2.0 ** -8 + 2.0 ** -14)


def test_layer_keeps_its_residual_for_the_gradients(cuda_dev):
    """keep_residual: the same output, the residual stream that moe_finalize writes, and the gradients that
    this stream gives when handed in."""
    cfg, _, layer, *_, g = _layer(cuda_dev)
    keep = MoELayer(layer.inp, router=layer.router, keep_residual=True)
    out = layer.forward(None, layer.inp.a1).clone()
    assert torch.equal(keep.forward(None, layer.inp.a1), out)
    o = torch.empty_like(out)
    moe.moe_finalize(layer.y, layer.topk_weights, cfg.top_k, False, residual=layer.inp.residual,
                     rms_weight=layer.inp.rms_weight, residual_out=o)
    assert torch.equal(keep.residual_out, o)
    dout = torch.randn((cfg.T, cfg.H), generator=g).to(BF).to(cuda_dev)
    want = [t.clone() for t in layer.router_backward(dout, layer.inp.a1, o)[1]]
    assert all(torch.equal(a, b) for a, b in zip(keep.router_backward(dout, layer.inp.a1)[1], want))
    with pytest.raises(ValueError):
        layer.router_backward(dout, layer.inp.a1)


def test_router_step_captured_beside_eager_ones_and_on_two_streams(cuda_dev):
    """Two layers' steps with their own buffers, one captured and replayed, one eager on another stream at the
    same time, give what they give alone."""
    layers = [_layer(cuda_dev, seed=s) for s in (1, 2)]
    douts = [torch.randn((c.T, c.H), generator=g).to(BF).to(cuda_dev) for c, *_, g in layers]
    steps, wants = [], []
    for (cfg, inp, layer, *_), dout in zip(layers, douts):
        def step(layer=layer, dout=dout):
            out = layer.forward(None, layer.inp.a1)
            fin, grads = layer.router_backward(dout, layer.inp.a1, residual_out=layer.inp.residual)
            return [out, fin[1], fin[2], fin[3], *grads]
        steps.append(step)
        wants.append([t.clone() for t in step()])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = steps[0]()
    side = torch.cuda.Stream()
    for t in captured:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graph.replay()
        with torch.cuda.stream(side):
            eager = steps[1]()
    torch.cuda.synchronize()
    assert moe.moe_device_status() == moe.MOE_OK
    for got, want in ((captured, wants[0]), (eager, wants[1])):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_router_gradients_on_another_stream_and_after_a_refused_call(cuda_dev):
    """The router's gradient buffers are made by its first call: one that is refused leaves them fit for the
    next, and one on another stream takes none that the current stream still works on."""
    (cfg, _, layer, *_, g), (_, _, ref, *_) = _layer(cuda_dev), _layer(cuda_dev)
    dw = torch.randn((cfg.T, cfg.top_k), generator=g).to(cuda_dev)
    layer.forward(None, layer.inp.a1)
    ref.forward(None, ref.inp.a1)
    want = [t.clone() for t in ref.router.backward(dw, ref.inp.a1, ref.topk_ids)]
    with pytest.raises(ValueError):
        layer.router.backward(dw, layer.inp.a1[:, :64].contiguous(), layer.topk_ids)
    got = layer.router.backward(dw, layer.inp.a1, layer.topk_ids)
    assert all(torch.equal(a, w) for a, w in zip(got, want))
    torch.cuda.synchronize()
    layer.router._grads = None
    side = torch.cuda.Stream()
    n = layer.router.gate_w.numel()
    junk = torch.empty(n, dtype=BF, device=cuda_dev)
    torch.cuda._sleep(20_000_000)
    junk.fill_(7.0)
    del junk  # (the current stream still has it to write)
    got = layer.router.backward(dw, layer.inp.a1, layer.topk_ids, stream=side)
    side.synchronize()
    early = [t.cpu() for t in got]
    torch.cuda.synchronize()
    for a, b, w in zip(got, early, want):
        assert torch.equal(a, w) and torch.equal(b, w.cpu())


def test_layer_and_router_refusals(cuda_dev):
    cfg, inp, layer, *_ = _layer(cuda_dev)
    other = MoERouter(cfg.T + 1, layer.router.gate_w, cfg.top_k)
    with pytest.raises(ValueError):
        MoELayer(layer.inp, router=other)
    with pytest.raises(ValueError):
        MoELayer(layer.inp).router_backward(layer.out, layer.inp.a1)
    with pytest.raises(ValueError):  # a batch of another size than the router's
        layer.router.forward(layer.inp.a1[:8])
    with pytest.raises(moe.MoeError):
        moe.moe_route_grouped(layer.router.logits, 3, n_group=3)
    with pytest.raises(ValueError):
        moe.moe_route_grouped(layer.router.logits.T, 3)
    with pytest.raises(ValueError):
        moe.moe_linear(layer.inp.a1[:, ::2], layer.router.gate_w[:, ::2])
    with pytest.raises(ValueError):
        moe.moe_linear(layer.inp.a1, layer.router.gate_w.cpu())
