"""What MoEExperts and MoELayer.experts_backward hold between calls: gradients that a first call adds to, weights that are
replaced, a forward pass that a backward call has used up."""
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe
from mixture_experts_layer_tokens_gb300.inputs import CONFIGS, make_inputs, scaled
from mixture_experts_layer_tokens_gb300.layer import MoEExperts, MoELayer

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
T, K, E, H, I = 45, 2, 5, 264, 136


def _inputs(seed=0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand((T, E), generator=g).argsort(1)[:, :K].to(torch.int32),
            torch.randn((T, H), generator=g).to(dtype),
            (torch.randn((E, 2 * I, H), generator=g) / H ** 0.5).to(dtype),
            (torch.randn((E, H, I), generator=g) / I ** 0.5).to(dtype),
            torch.randn((T * K, H), generator=g).to(dtype))


def _layer(dev, seed=3):
    cfg = scaled(CONFIGS["tiny"], name="state", T=64, H=256, I=128, E=8, top_k=2)
    layer = MoELayer(make_inputs(cfg, seed=seed).to(dev))
    layer.forward(layer.inp.logits, layer.inp.a1)
    dy = torch.randn((128, 256), generator=torch.Generator().manual_seed(seed)).to(BF).to(dev)
    return layer, dy


def _spoil(dev):
    """What the allocator hands out next holds NaN."""
    torch.cuda.synchronize()
    for size in (1 << 10, 1 << 16, 1 << 19, 1 << 20, 1 << 22, 1 << 24):
        held = [torch.full((size // 4,), float("nan"), device=dev) for _ in range(8)]
        del held


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,wdt", [(BF, None), (BF, F32), (HF, F32)])
def test_first_call_adds_to_zeros(cuda_dev, dtype, wdt):
    ids, a1, w13, w2, dy = (t.to(cuda_dev) for t in _inputs(1, dtype))
    al = moe.moe_align(ids, E)
    ex = MoEExperts(w13, w2, T, K, dw_dtype=wdt)
    ex.forward(a1, al)
    want = [t.clone() for t in ex.backward(dy, a1, al)[:2]]
    _spoil(cuda_dev)
    ex = MoEExperts(w13, w2, T, K, dw_dtype=wdt)
    ex.forward(a1, al)
    # (a group's rows are one run of the sums, added to 0)
    assert all(torch.equal(a, b) for a, b in zip(ex.backward(dy, a1, al, accumulate=True)[:2], want))


@pytest.mark.gpu
@pytest.mark.parametrize("wdt", [None, F32])
def test_first_call_of_a_layer_adds_to_zeros(cuda_dev, wdt):
    layer, dy = _layer(cuda_dev)
    want = [t.clone() for t in layer.experts_backward(dy, layer.inp.a1, dw_dtype=wdt)]
    other, _ = _layer(cuda_dev)
    _spoil(cuda_dev)
    got = other.experts_backward(dy, other.inp.a1, dw_dtype=wdt, accumulate=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("accumulate", [False, True])
def test_zeros_are_set_before_another_stream_adds(cuda_dev, accumulate):
    """An object made on a stream that is busy, and used at once on another."""
    ids, a1, w13, w2, dy = (t.to(cuda_dev) for t in _inputs(7))
    al = moe.moe_align(ids, E)
    ex = MoEExperts(w13, w2, T, K, dw_dtype=F32)
    ex.forward(a1, al)
    want = [t.clone() for t in ex.backward(dy, a1, al)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # (a tenth of a second)
    ex = MoEExperts(w13, w2, T, K, dw_dtype=F32)
    ex.forward(a1, al, stream=side)
    got = ex.backward(dy, a1, al, accumulate=accumulate, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_gradients_made_under_capture(cuda_dev):
    """Zeros set in a graph would be set again by every replay, so there the first call has to write."""
    ids, a1, w13, w2, dy = (t.to(cuda_dev) for t in _inputs(2))
    al = moe.moe_align(ids, E)
    ex = MoEExperts(w13, w2, T, K, dw_dtype=F32)
    ex.forward(a1, al)
    one = [t.clone() for t in ex.backward(dy, a1, al)[:2]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph, held = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph, stream=side):
        held.append(MoEExperts(w13, w2, T, K, dw_dtype=F32, stream=side))
        held[0].forward(a1, al, stream=side)
        with pytest.raises(ValueError, match="accumulate"):
            held[0].backward(dy, a1, al, accumulate=True, stream=side)
        held[0].backward(dy, a1, al, stream=side)
        held[0].forward(a1, al, stream=side)
        held[0].backward(dy, a1, al, accumulate=True, stream=side)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((held[0].dw13, held[0].dw2), one):
            assert torch.equal(got, 2 * w)


@pytest.mark.gpu
def test_layer_uses_the_weights_it_has_now(cuda_dev):
    layer, dy = _layer(cuda_dev)
    layer.experts_backward(dy, layer.inp.a1)
    g = torch.Generator().manual_seed(9)
    layer.inp.w13 = (torch.randn(layer.inp.w13.shape, generator=g) / 16).to(BF).to(cuda_dev)
    layer.inp.w2 = (torch.randn(layer.inp.w2.shape, generator=g) / 11).to(BF).to(cuda_dev)
    layer.forward(layer.inp.logits, layer.inp.a1)
    got = [t.clone() for t in layer.experts_backward(dy, layer.inp.a1)]
    ex = MoEExperts(layer.inp.w13, layer.inp.w2, 64, 2)
    ex.forward(layer.inp.a1, layer.al)
    assert all(torch.equal(a, b) for a, b in zip(got, ex.backward(dy, layer.inp.a1, layer.al)))


@pytest.mark.gpu
def test_backward_needs_a_forward_of_its_own(cuda_dev):
    ids, a1, w13, w2, dy = (t.to(cuda_dev) for t in _inputs(3))
    al = moe.moe_align(ids, E)
    ex = MoEExperts(w13, w2, T, K)
    with pytest.raises(ValueError, match="forward"):
        ex.backward(dy, a1, al)
    ex.hidden(a1, al)
    with pytest.raises(ValueError, match="dout"):  # (refused before anything is used up)
        ex.backward(dy[:, :8], a1, al)
    want = [t.clone() for t in ex.backward(dy, a1, al)]
    with pytest.raises(ValueError):
        ex.forward(a1[:, :8], al)
    with pytest.raises(ValueError, match="forward"):
        ex.backward(dy, a1, al)
    ex.forward(a1, al)
    assert all(torch.equal(a, b) for a, b in zip(ex.backward(dy, a1, al), want))


@pytest.mark.gpu
@pytest.mark.parametrize("first", [0, 1])
def test_parts_of_a_step_in_graphs(cuda_dev, first):
    """A captured forward pass with eager gradients, and the other way round, whichever is captured first: the host does
    not see a replay, and refuses neither."""
    ids, a1, w13, w2, dy = (t.to(cuda_dev) for t in _inputs(4))
    al = moe.moe_align(ids, E)
    ex = MoEExperts(w13, w2, T, K)
    ex.forward(a1, al)
    want = [t.clone() for t in ex.backward(dy, a1, al)]
    side = torch.cuda.Stream()
    calls = (lambda: ex.forward(a1, al, stream=side), lambda: ex.backward(dy, a1, al, stream=side))
    graphs = [torch.cuda.CUDAGraph() for _ in calls]
    for i in (first, 1 - first):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graphs[i], stream=side):
            calls[i]()
    for _ in range(2):
        graphs[0].replay()
        assert all(torch.equal(a, b) for a, b in zip(ex.backward(dy, a1, al), want))
        ex.forward(a1, al)
        graphs[1].replay()
        assert all(torch.equal(a, b) for a, b in zip((ex.dw13, ex.dw2, ex.da1), want))


@pytest.mark.parametrize("dtype,wdt", [(BF, HF), (HF, BF), (BF, torch.float64)])
def test_gradient_types_are_refused_first(dtype, wdt):
    _, _, w13, w2, _ = _inputs(5, dtype)
    with pytest.raises(TypeError, match="dw_dtype"):
        MoEExperts(w13, w2, T, K, dw_dtype=wdt)


@pytest.mark.gpu
def test_a_refused_gradient_type_leaves_the_layer_as_it_was(cuda_dev):
    layer, dy = _layer(cuda_dev)
    with pytest.raises(TypeError):
        layer.experts_backward(dy, layer.inp.a1, dw_dtype=HF)
    assert layer.experts_backward(dy, layer.inp.a1, dw_dtype=F32)[0].dtype is F32


@pytest.mark.gpu
@pytest.mark.parametrize("top_k", [1, 2])
def test_no_tokens(cuda_dev, top_k):
    """Nothing to do but the weights' gradients, which are zeros, or stay."""
    _, _, w13, w2, _ = (t.to(cuda_dev) for t in _inputs(6))
    none = lambda *s: torch.empty((0,) + s, dtype=BF, device=cuda_dev)  # noqa: E731
    al = moe.moe_align(torch.empty((0, top_k), dtype=torch.int32, device=cuda_dev), E)
    ex = MoEExperts(w13, w2, 0, top_k)
    assert ex.forward(none(H), al).shape == (0, H)
    ex.dw2.fill_(7)
    dw13, dw2, da1 = ex.backward(none(H), none(H), al)
    assert bool((dw13 == 0).all()) and bool((dw2 == 0).all()) and da1.shape == (0, H)
    ex.forward(none(H), al)
    dw2.fill_(7)
    assert bool((ex.backward(none(H), none(H), al, accumulate=True)[1] == 7).all())
    assert moe.moe_device_status() == moe.MOE_OK
