"""The norm, the experts' products and the activation as they are used together: a layer that normalises its input, and
the training step of the experts, eager and captured.

Tolerances against fp64 autograd, in the 2-norm, count the roundings on the way to bf16, each at most half a step, 2^-8
(fp16 2^-11): [g | u] (twice: its two halves meet in a product), h, and the output for y and dw2; dh, [g | u] (twice, in
the slope and the factor), dgu and the output for dw13; one more for the sum of the slots in da1."""
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe
from mixture_experts_layer_tokens_gb300.inputs import CONFIGS, make_inputs, scaled
from mixture_experts_layer_tokens_gb300.layer import MoEExperts, MoELayer, MoERouter
from oracle import experts_ref as er
from oracle import moe_ref

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _close(got, ref, roundings, dtype, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    err, most = float((got - ref).norm()), roundings * torch.finfo(dtype).eps / 2 * float(ref.norm())
    assert err <= most, f"{what}: {err:.3e} > {most:.3e}"


def _experts(T, top_k, E, H, I, act, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    rows = I if act.endswith("no_mul") else 2 * I
    ids = torch.rand((T, E), generator=g).argsort(1)[:, :top_k].to(torch.int32)
    a1 = torch.randn((T, H), generator=g).to(dtype)
    w13 = (torch.randn((E, rows, H), generator=g) / H ** 0.5).to(dtype)
    w2 = (torch.randn((E, H, I), generator=g) / I ** 0.5).to(dtype)
    dy = torch.randn((T * top_k, H), generator=g).to(dtype)
    return ids, a1, w13, w2, dy


def _autograd(ids, a1, w13, w2, dy, act):
    """(y, dw13, dw2, da1) in fp64."""
    x, a, b = (t.double().requires_grad_(True) for t in (a1, w13, w2))
    T, top_k = ids.shape
    y = torch.zeros((T * top_k, a1.shape[1]), dtype=torch.float64)
    for e in range(w13.shape[0]):
        f = (ids.view(-1) == e).nonzero().flatten()
        y = y.index_copy(0, f, moe_ref.activation(x[f // top_k] @ a[e].T, act) @ b[e].T)
    return (y.detach(), *torch.autograd.grad((y * dy.double()).sum(), (a, b, x)))


@pytest.mark.parametrize("act", sorted(moe.ACTIVATIONS))
@pytest.mark.parametrize("dtype", [BF, HF])
def test_experts_training_step(cuda_dev, act, dtype):
    ids, a1, w13, w2, dy = _experts(150, 3, 12, 264, 136, act, dtype)
    y, dw13, dw2, da1 = _autograd(ids, a1, w13, w2, dy, act)
    al = moe.moe_align(ids.to(cuda_dev), 12)
    ex = MoEExperts(w13.to(cuda_dev), w2.to(cuda_dev), 150, 3, act, dw_dtype=torch.float32 if dtype is HF else None)
    d1 = a1.to(cuda_dev)
    _close(ex.forward(d1, al), y, 4.2, dtype, "y")
    g13, g2, gx = (t if t is None else t.clone() for t in ex.backward(dy.to(cuda_dev), d1, al))
    _close(g2, dw2, 4.2, dtype, "dw2")
    _close(g13, dw13, 5, dtype, "dw13")
    assert (gx is None) == (dtype is HF)
    if gx is not None:
        _close(gx, da1, 6, dtype, "da1")
    # once more, added: twice the gradient, but for the additions' roundings
    ex.forward(d1, al)
    t13, t2, _ = ex.backward(dy.to(cuda_dev), d1, al, accumulate=True)
    for got, one in ((t13, g13), (t2, g2)):
        assert ((got.double() - 2 * one.double()).abs() <= 2 * one.double().abs() * torch.finfo(got.dtype).eps / 2
                + (2.0 ** -20 if got.dtype is torch.float32 else 2.0 ** -8 * float(one.double().abs().max()))).all()
    assert moe.moe_device_status() == moe.MOE_OK


def test_workspace_of_many_rows_off_128_bytes(cuda_dev):
    """Enough rows of an odd width that the products move them first: the object's one workspace is enough for each."""
    T, k, E, H, I = 2100, 1, 2, 2056, 2072
    ids, a1, w13, w2, dy = (t.to(cuda_dev) for t in _experts(T, k, E, H, I, "silu_no_mul", BF, seed=4))
    assert moe.grouped_linear_workspace_size(T, E, H, I) > 0
    al = moe.moe_align(ids, E)
    ex = MoEExperts(w13, w2, T, k, "silu_no_mul")
    y = ex.forward(a1, al)
    assert torch.equal(y, moe.moe_grouped_linear(ex.h, w2, al.expert_offsets, al.sorted_slot, k, out_rows="slot"))
    h = ex.h.clone()
    dw13, dw2, _ = ex.backward(dy, a1, al)
    dh, want = moe.moe_grouped_linear_backward(dy, h, w2, al.expert_offsets, al.sorted_slot, k, dout_rows="slot")
    assert torch.equal(dw2, want) and torch.equal(ex.dh, dh)
    _, want = moe.moe_grouped_linear_backward(ex.gu, a1, w13, al.expert_offsets, al.sorted_slot, k, x_rows="token")
    assert torch.equal(dw13, want)


def test_layer_step_trains_router_and_experts(cuda_dev):
    """forward, the finalize's gradients, the router's and the experts': the experts' against autograd over the whole
    sum (dy is rounded once more on the way)."""
    T, H, I, E, k = 60, 256, 128, 8, 2
    cfg = scaled(CONFIGS["tiny"], name="train", T=T, H=H, I=I, E=E, top_k=k, residual=True)
    inp = make_inputs(cfg, seed=3)
    g = torch.Generator().manual_seed(11)
    gate = (torch.randn((E, H), generator=g) / H ** 0.5).to(BF).to(cuda_dev)
    layer = MoELayer(inp.to(cuda_dev), router=MoERouter(T, gate, k))
    a1 = layer.inp.a1
    layer.forward(None, a1)
    dout = torch.randn((T, H), generator=g).to(BF)
    fin, router = layer.router_backward(dout.to(cuda_dev), a1, need_dy=True)
    assert router[0].shape == gate.shape
    dw13, dw2, da1 = layer.experts_backward(fin[0], a1, dw_dtype=torch.float32)
    ids, w = layer.topk_ids.cpu(), layer.topk_weights.cpu().double()
    dy = (dout.double()[:, None, :] * w[:, :, None]).view(T * k, H)
    _, r13, r2, rx = _autograd(ids, inp.a1, inp.w13, inp.w2, dy, "silu")
    _close(dw2, r2, 4.2, BF, "dw2")  # (fp32: one rounding fewer, dy's in its place)
    _close(dw13, r13, 5, BF, "dw13")
    _close(da1, rx, 7, BF, "da1")
    with pytest.raises(ValueError, match="dw_dtype"):
        layer.experts_backward(fin[0], a1, dw_dtype=BF)
    # the layer's own forward and the separate calls agree to the roundings of y (h is rounded in both)
    y = layer.y.double().cpu()
    _close(layer.trainer.forward(a1, layer.al), y, 2 * 4.2, BF, "y")


@pytest.mark.parametrize("quant", ["fp8", "nvfp4", "fp8_tensor"])
def test_experts_backward_refuses(cuda_dev, quant):
    cfg = scaled(CONFIGS["deepseek" if quant != "nvfp4" else "mixtral_nvfp4"], name="no", T=4, H=256, I=256, E=4, top_k=2,
                 quant=quant, shared_I=0)
    layer = MoELayer(make_inputs(cfg).to(cuda_dev))
    with pytest.raises(ValueError, match="bf16 layer"):
        layer.experts_backward(layer.y, layer.inp.a1)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("quant", ["bf16", "fp8", "fp8_token", "fp8_tensor", "nvfp4"])
def test_layer_with_input_norm(cuda_dev, quant, residual):
    """The layer on what the norm gives, bit for bit: the same calls on moe_rmsnorm's outputs."""
    T, H = 37, 512
    cfg = scaled(CONFIGS["tiny"], name="norm", T=T, H=H, I=256, E=8, top_k=2, quant=quant, residual=True, rms=True,
                 shared_I=256)
    inp = make_inputs(cfg, seed=5)
    g = torch.Generator().manual_seed(6)
    gamma = (torch.rand((H,), generator=g) + 0.5).to(BF).to(cuda_dev)
    x = torch.randn((T, H), generator=g).to(BF).to(cuda_dev)
    res = torch.randn((T, H), generator=g).to(BF).to(cuda_dev) if residual else None
    layer = MoELayer(inp.to(cuda_dev), input_norm=gamma, keep_residual=True)
    got = layer.forward(layer.inp.logits, x, residual=res).clone()
    torch.cuda.synchronize()
    assert moe.moe_device_status() == moe.MOE_OK
    direct = quant in ("fp8", "fp8_token")
    a1, total, q, s = moe.moe_rmsnorm(x, gamma, residual=res, quant=quant if direct else None)
    n, v = er.rmsnorm(x.cpu(), gamma.cpu(), None if res is None else res.cpu())
    assert ((a1.cpu().double() - n).abs() <= n.abs() * (2 ** -8 + 2 ** -17) + 1e-39).all()
    assert torch.equal(layer.a1, a1)
    plain = MoELayer(inp.to(cuda_dev), keep_residual=True)
    if residual:
        plain.inp.residual = total
    if direct:
        assert torch.equal(layer.a1q, q) and torch.equal(layer.a1q_scale, s)
        plain.norm_quant, plain.a1q, plain.a1q_scale = True, q, s
    want = plain.forward(plain.inp.logits, a1)
    assert torch.equal(got, want) and torch.equal(layer.residual_out, plain.residual_out)
    if residual:
        with pytest.raises(ValueError, match="residual"):
            plain.forward(plain.inp.logits, a1, residual=res)


def test_input_norm_refuses_a_single_launch(cuda_dev):
    cfg = scaled(CONFIGS["llama1_fused"], name="one", T=2, H=256, I=256, E=4, shared_I=256)
    with pytest.raises(ValueError, match="input_norm"):
        MoELayer(make_inputs(cfg).to(cuda_dev), input_norm=torch.ones(256, dtype=BF, device=cuda_dev))


def test_training_step_captured(cuda_dev):
    """The whole step in a graph, replayed on another routing and other values, against the eager calls bit for bit; two
    captured steps with buffers of their own run one after the other on two streams."""
    T, k, E, H, I = 70, 2, 6, 256, 136
    sets = [_experts(T, k, E, H, I, "swigluoai", BF, seed=s) for s in (1, 2)]
    ids, a1, w13, w2, dy = (t.to(cuda_dev) for t in sets[0])
    ex = [MoEExperts(w13, w2, T, k, "swigluoai", dw_dtype=torch.float32) for _ in range(2)]
    al = [moe.Alignment(T, k, E, cuda_dev) for _ in range(2)]

    def step(i, stream=None):
        moe.moe_align(ids, E, out=al[i], stream=stream)
        return (ex[i].forward(a1, al[i], stream=stream), *ex[i].backward(dy, a1, al[i], stream=stream))

    for i in range(2):
        step(i)
    graphs = []
    for i in range(2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(i, side)
        graphs.append((graph, side))
    for t, v in zip((ids, a1, w13, w2, dy), sets[1]):
        t.copy_(v)
    want = [t.clone() for t in step(0)]
    for e in ex:
        for t in (e.y, e.dw13, e.dw2, e.da1):
            t.fill_(7)
    torch.cuda.synchronize()
    for graph, side in graphs:
        with torch.cuda.stream(side):
            graph.replay()
    torch.cuda.synchronize()
    for e in ex:
        assert all(torch.equal(a, b) for a, b in zip((e.y, e.dw13, e.dw2, e.da1), want))
    assert moe.moe_device_status() == moe.MOE_OK


def test_two_threads_on_two_streams(cuda_dev):
    """Host threads that call at once, each on its stream with buffers of its own, get what one gets alone (the first calls
    of a kernel's several forms among them)."""
    import threading

    T, k, E, H, I = 90, 2, 6, 264, 136
    sets = [[t.to(cuda_dev) for t in _experts(T, k, E, H, I, "silu", BF, seed=s)] for s in (21, 22)]
    gamma = torch.ones(H, dtype=BF, device=cuda_dev)

    def step(ids, a1, w13, w2, dy, stream):
        n, _, q, sc = moe.moe_rmsnorm(a1, gamma, quant="fp8", stream=stream)
        al = moe.Alignment(T, k, E, cuda_dev)
        moe.moe_align(ids, E, out=al, stream=stream)
        ex = MoEExperts(w13, w2, T, k, dw_dtype=torch.float32, stream=stream)
        y = ex.forward(n, al, stream=stream)
        return (n, q, sc, y, *ex.backward(dy, n, al, stream=stream))

    alone = [[t.clone() for t in step(*v, None)] for v in sets]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            torch.cuda.set_device(cuda_dev)
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                for _ in range(30):
                    got[i] = step(*sets[i], side)
            side.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert moe.moe_device_status() == moe.MOE_OK
