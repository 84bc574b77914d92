"""moe_activation and its gradient against their fp64 definitions.

Tolerances: act(g) is within 2^-20 (1 + |g|) and act'(g) within 2^-19 (1 + |g|) (the logistic function within 2^-21,
of 1.702 g too; its share in the slope is weighed by 1 + 2 * 1.702 |g|), the products round by 2^-24 each, and an
output once, by half a step."""
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe
from oracle import experts_ref as er

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]


def _half(ref, dtype):
    fi = torch.finfo(dtype)
    return ref.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps


def _within(got, ref, tol, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    bad = (got - ref).abs() - tol
    assert (bad <= 0).all(), f"{what}: {int((bad > 0).sum())} of {bad.numel()}, worst excess {bad.max():.3e}"


def _inputs(S, I, name, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + S * 3 + I)
    gu = (torch.randn((S, I if name.endswith("no_mul") else 2 * I), generator=g) * 4).to(dtype)
    # the clamps' borders and their neighbours, zeros and large values
    special = torch.tensor([7.0, -7.0, 7.0625, -7.0625, 6.96875, 0.0, -0.0, 100.0, -100.0, -30.0, 14.0, -14.0])
    flat = gu.view(-1)
    at = torch.randint(0, flat.numel(), (min(flat.numel(), 4 * len(special)),), generator=g)
    flat[at] = special.repeat(4)[:len(at)].to(dtype)
    return gu, torch.randn((S, I), generator=g).to(dtype)


def _check_h(h, gu, name, dtype):
    ref, m, g = er.activation(gu, name)
    _within(h, ref, _half(ref, dtype) * 1.01 + 2 ** -20 * (1 + g.abs()) * m.abs(), f"h {name}")


def _check_dgu(dgu, dh, gu, name, dtype):
    ref = er.activation_backward(dh, gu, name)
    _, m, g = er.activation(gu, name)
    d = dh.double().abs()
    tol = 2 ** -19 * (1 + g.abs()) * m.abs() * d
    if not name.endswith("no_mul"):
        tol = torch.cat([tol, 2 ** -20 * (1 + g.abs()) * d], 1)
    _within(dgu, ref, _half(ref, dtype) * 1.01 + tol, f"dgu {name}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", sorted(moe.ACTIVATIONS))
@pytest.mark.parametrize("S,I", [(1, 8), (3, 24), (129, 264), (513, 1032)])
def test_activation(cuda_dev, S, I, name, dtype):
    gu, dh = _inputs(S, I, name, dtype)
    store = torch.full((S + 1, I), 7.0, dtype=dtype, device=cuda_dev)
    h = moe.moe_activation(gu.to(cuda_dev), name, h=store[:S])
    _check_h(h, gu, name, dtype)
    back = torch.full((S + 1, gu.shape[1]), 7.0, dtype=dtype, device=cuda_dev)
    dgu, h2 = moe.moe_activation_backward(dh.to(cuda_dev), gu.to(cuda_dev), name, dgu=back[:S], need_h=True)
    _check_dgu(dgu, dh, gu, name, dtype)
    assert torch.equal(h, h2) and bool((store[S] == 7).all()) and bool((back[S] == 7).all())
    assert moe.moe_activation_backward(dh.to(cuda_dev), gu.to(cuda_dev), name)[1] is None


@pytest.mark.parametrize("name", sorted(moe.ACTIVATIONS))
def test_activation_in_place(cuda_dev, name):
    gu, dh = _inputs(70, 256, name, torch.bfloat16)
    a, b = gu.to(cuda_dev), dh.to(cuda_dev)
    dgu, h = moe.moe_activation_backward(b, a, name, dgu=a, h=b)
    assert dgu is a and h is b
    _check_dgu(dgu, dh, gu, name, torch.bfloat16)
    _check_h(h, gu, name, torch.bfloat16)


@pytest.mark.parametrize("name", sorted(moe.ACTIVATIONS))
def test_activation_far_and_not_a_number(cuda_dev, name):
    """A gate of -inf (a sum that 16 bits could not hold) is 0 with a slope of 0; a NaN stays where it is."""
    no_mul = name.endswith("no_mul")
    for dtype in DTYPES:
        gu = torch.ones((1, 16 if no_mul else 32), dtype=dtype)
        gu[0, 0], gu[0, 1], gu[0, 2] = float("-inf"), torch.finfo(dtype).min, float("nan")
        dh = torch.full((1, 16), 2.0, dtype=dtype)
        h = moe.moe_activation(gu.to(cuda_dev), name).cpu()
        dgu, _ = moe.moe_activation_backward(dh.to(cuda_dev), gu.to(cuda_dev), name)
        dgu = dgu.cpu()
        assert h[0, 0] == 0 and h[0, 1] == 0 and torch.isnan(h[0, 2]) and torch.isfinite(h[0, 3:]).all()
        assert dgu[0, 0] == 0 and dgu[0, 1] == 0 and torch.isnan(dgu[0, 2])
        assert torch.isfinite(dgu[0, 3:16]).all()
        if not no_mul:
            assert dgu[0, 16] == 0 and torch.isnan(dgu[0, 18]) and torch.isfinite(dgu[0, 19:]).all()


def test_activation_slope_by_differences(cuda_dev):
    """The gradient against differences of the operator's own values, in fp16 where a step of 1/8 is exact: the
    difference is off by the third derivative (below 2 for these) times step^2 / 6 and two roundings over the steps."""
    gu = (torch.arange(64) / 8 - 4).to(torch.float16)[None]
    for name in ("silu_no_mul", "gelu_no_mul"):
        at = lambda v: moe.moe_activation(v.to(cuda_dev), name).double().cpu()  # noqa: E731
        slope = moe.moe_activation_backward(torch.ones_like(gu).to(cuda_dev), gu.to(cuda_dev), name)[0].double().cpu()
        diff = (at(gu + 0.125) - at(gu - 0.125)) / 0.25
        tol = 2 * 0.125 ** 2 / 6 + 2 * 4.2 * 2 ** -11 / 0.25 + 1.2 * 2 ** -11
        assert (slope - diff).abs().max() <= tol


def test_activation_captured(cuda_dev):
    gu, dh = _inputs(33, 512, "silu", torch.bfloat16)
    a, b = gu.to(cuda_dev), dh.to(cuda_dev)
    h = moe.moe_activation(a)
    dgu, _ = moe.moe_activation_backward(b, a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        moe.moe_activation(a, h=h, stream=side)
        moe.moe_activation_backward(b, a, dgu=dgu, stream=side)
    gu2, dh2 = _inputs(33, 512, "silu", torch.bfloat16, seed=3)
    a.copy_(gu2)
    b.copy_(dh2)
    graph.replay()
    torch.cuda.synchronize()
    _check_h(h, gu2, "silu", torch.bfloat16)
    _check_dgu(dgu, dh2, gu2, "silu", torch.bfloat16)
    assert moe.moe_activation(a[:0]).shape == (0, 512)
