"""moe_rmsnorm against its fp64 definition.

Tolerances: v is within 2^-24 of itself; the squares, of one sign, are summed in fp32 by at most 32 additions a
thread, 5 steps of shuffles and 31 warps, so their sum is within (2 + 68) 2^-24 and r, with its own operations,
within 38 2^-24; n is within 42 2^-24 < 2^-18 of itself, and so is a group's largest and, after a division, its
scale.  A code stands for n / s, here with the scale that the call gave, before its rounding by half a step: 2^-4
of it, or 2^-10 where the steps are 2^-9."""
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe
from oracle import experts_ref as er

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _inputs(T, H, seed=0, residual=True, scale=1.0):
    g = torch.Generator().manual_seed(seed * 131 + T * 7 + H)
    x = (torch.randn((T, H), generator=g) * scale).to(BF)
    res = (torch.randn((T, H), generator=g) * 2 * scale).to(BF) if residual else None
    return x, res, (torch.rand((H,), generator=g) + 0.5).to(BF)


def _close(got, ref, rel, extra=0.0, what=""):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    bad = (got - ref).abs() - (ref.abs() * rel + extra)
    assert (bad <= 0).all(), f"{what}: {int((bad > 0).sum())} of {bad.numel()}, worst {bad.max():.3e}"


def _check(outs, x, res, w, quant, eps=1e-6):
    out, res_out, q, scale = outs
    n, v = er.rmsnorm(x, w, res, eps)
    if out is not None:
        _close(out, n, 2 ** -8 + 2 ** -17, 1e-39, "out")
    if res_out is not None:
        _close(res_out, v, 2 ** -8 + 2 ** -23, 1e-39, "residual_out")
    if quant is not None:
        _close(scale, er.row_scales(n, 128 if quant == "fp8" else -1), 2 ** -17, 0.0, "scale")
        ratio = n / er.spread(scale.double().cpu(), n.shape[1])
        _close(q.view(torch.float8_e4m3fn).float(), ratio, 2 ** -4 + 2 ** -16, 2 ** -10 * (1 + 2 ** -16), "q")


SIZES = [(1, 8), (1, 7168), (3, 120), (2, 128), (5, 136), (7, 1000), (160, 2048), (33, 4104), (200, 8192), (2, 16384),
         (300, 16384), (4000, 64), (1031, 1032)]


@pytest.mark.parametrize("quant", [None, "fp8", "fp8_token"])
@pytest.mark.parametrize("T,H", SIZES)
def test_rmsnorm(cuda_dev, T, H, quant):
    for residual in (True, False):
        x, res, w = _inputs(T, H, residual=residual)
        d = lambda t: None if t is None else t.to(cuda_dev)  # noqa: E731
        outs = moe.moe_rmsnorm(d(x), d(w), residual=d(res), quant=quant, need_out=quant is None or T % 2 == 0)
        assert (outs[1] is None) == (res is None)
        _check(outs, x, res, w, quant)


def test_rmsnorm_edges(cuda_dev):
    """Rows of zeros (eps alone, and the smallest scale), tiny and large values, one spike; eps 0."""
    x, res, w = _inputs(8, 512, residual=False)
    x[0] = 0
    x[1] *= 1e-20
    x[2] *= 1e15
    x[3] = 0
    x[3, 7] = 100.0
    for quant in ("fp8", "fp8_token"):
        outs = moe.moe_rmsnorm(x.to(cuda_dev), w.to(cuda_dev), quant=quant)
        n, _ = er.rmsnorm(x, w)
        _close(outs[0], n, 2 ** -8 + 2 ** -17, 1e-39, "out")
        _check(outs, x, None, w, quant)
    y = x[2:]
    _check(moe.moe_rmsnorm(y.to(cuda_dev), w.to(cuda_dev), eps=0.0, quant="fp8"), y, None, w, "fp8", eps=0.0)


@pytest.mark.parametrize("T,H", [(6, 256), (400, 7168), (5, 7168)])
def test_rmsnorm_rows_are_their_own(cuda_dev, T, H):
    """A NaN or an infinity changes its row alone, outputs end where they end, and every call gives the same bits."""
    x, res, w = _inputs(T, H)
    args = [t.to(cuda_dev) for t in (x, w, res)]
    store = [torch.full((T + 1, H), 7, dtype=t, device=cuda_dev) for t in (BF, BF, torch.uint8)]
    scale = torch.full((T + 1, (H + 127) // 128), 7.0, device=cuda_dev)
    call = lambda: moe.moe_rmsnorm(args[0], args[1], residual=args[2], quant="fp8", out=store[0][:T],  # noqa: E731
                                   residual_out=store[1][:T], q=store[2][:T], q_scale=scale[:T])
    first = [t.clone() for t in call()]
    assert all(bool((t[T] == 7).all()) for t in store + [scale])
    again = call()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    args[0][T // 2, 3] = float("nan")
    args[0][T - 1, H - 1] = float("inf")
    odd = call()
    keep = torch.ones(T, dtype=torch.bool, device=cuda_dev)
    keep[T // 2] = keep[T - 1] = False
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(first, odd))
    assert torch.isnan(odd[0][T // 2]).all() and torch.isnan(odd[2].view(torch.float8_e4m3fn)[T // 2].float()).all()


@pytest.mark.parametrize("T,H", [(64, 1024), (3000, 1024), (2500, 4096)])
def test_rmsnorm_in_place(cuda_dev, T, H):
    x, res, w = _inputs(T, H)
    a, b, c = x.to(cuda_dev), res.to(cuda_dev), w.to(cuda_dev)
    outs = moe.moe_rmsnorm(a, c, residual=b, out=a, residual_out=b, quant="fp8")
    assert outs[0] is a and outs[1] is b
    _check(outs, x, res, w, "fp8")


def test_rmsnorm_agrees_with_prepare(cuda_dev):
    """With n that bf16 holds exactly, the codes and scales are those of moe_prepare on out."""
    x = torch.zeros((9, 512))
    x[:, ::2] = torch.tensor([1.0, -1.0]).repeat(128)
    x[:, 1::2] = torch.tensor([1.0, 1.0]).repeat(128)
    w = torch.exp2(torch.randint(-6, 7, (512,), generator=torch.Generator().manual_seed(0)).float())
    for quant in ("fp8", "fp8_token"):
        out, _, q, s = moe.moe_rmsnorm(x.to(BF).to(cuda_dev), w.to(BF).to(cuda_dev), eps=0.0, quant=quant)
        pq, ps = moe.moe_prepare(out, None, 1, False, quant)
        assert torch.equal(q, pq) and torch.equal(s.view(-1), ps.view(-1))


def test_rmsnorm_gradient_is_the_finalizes(cuda_dev):
    """dsum and drms of moe_finalize_backward from residual_out are the gradients of the norm."""
    x, res, w = _inputs(17, 1024)
    out, v, _, _ = moe.moe_rmsnorm(x.to(cuda_dev), w.to(cuda_dev), residual=res.to(cuda_dev), eps=1e-5)
    g = torch.Generator().manual_seed(9)
    dout, dres = (torch.randn((17, 1024), generator=g).to(BF) for _ in range(2))
    _, _, dsum, drms = moe.moe_finalize_backward(dout.to(cuda_dev), None, None, 1, residual_out=v, rms_weight=w.to(cuda_dev),
                                                 eps=1e-5, dresidual_out=dres.to(cuda_dev), need_dy=False)
    o, gamma = v.cpu().double().requires_grad_(True), w.double().requires_grad_(True)
    n = o / torch.sqrt((o * o).mean(1, keepdim=True) + 1e-5) * gamma
    do, dg = torch.autograd.grad((n * dout.double()).sum() + (o * dres.double()).sum(), (o, gamma))
    # dsum's parts are sums over a row of 1024: a share of the terms' magnitudes, then half a step
    mag = dout.double().abs() * 4 + dres.double().abs() + 4
    assert ((dsum.cpu().double() - do).abs() <= do.abs() * 2 ** -8 + mag * 2 ** -17).all()
    assert ((drms.cpu().double() - dg).abs() <= 17 * 6 * 4 * 2 ** -20).all()


def test_rmsnorm_captured(cuda_dev):
    """Captured on a side stream and replayed on other values."""
    x, res, w = _inputs(50, 2048)
    a, b, c = x.to(cuda_dev), res.to(cuda_dev), w.to(cuda_dev)
    outs = moe.moe_rmsnorm(a, c, residual=b, quant="fp8_token")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        moe.moe_rmsnorm(a, c, residual=b, quant="fp8_token", out=outs[0], residual_out=outs[1], q=outs[2], q_scale=outs[3],
                        stream=side)
    x2, res2, _ = _inputs(50, 2048, seed=5)
    a.copy_(x2)
    b.copy_(res2)
    graph.replay()
    torch.cuda.synchronize()
    _check(outs, x2, res2, w, "fp8_token")
    assert moe.moe_rmsnorm(a[:0], c)[0].shape == (0, 2048)
