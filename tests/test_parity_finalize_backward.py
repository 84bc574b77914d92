"""moe_finalize_backward against its fp64 definition, element by element.

Tolerances: sums over H in fp32 with at most 32 terms in a thread's chain, 5 shuffle levels and
16 warps, so within 2^-18 of the terms' magnitudes; the few operations of G beside them within
2^-20; dy and dsum are rounded to bf16 once (2^-8 of the value), dweights and drms stay fp32
(drms: a chain over the tokens of a CTA and then over the CTAs)."""
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe
from oracle import router_ref as rr

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _case(T, H, k, rms, dres, weights=True, seed=0):
    g = torch.Generator().manual_seed(T * 13 + H + k + seed)
    bf = lambda *s: torch.randn(s, generator=g).to(BF)  # noqa: E731
    c = dict(dout=bf(T, H), fused_expert_output=bf(T * k, H),
             topk_weights=torch.rand((T, k), generator=g) if weights else None, top_k=k)
    if rms:
        c.update(residual_out=bf(T, H) * 3, rms_weight=(torch.rand(H, generator=g) + 0.5).to(BF))
    if dres:
        c.update(dresidual_out=bf(T, H))
    return c


def _check(dev, T, H, k, rms=True, dres=True, weights=True, need=None):
    c = _case(T, H, k, rms, dres, weights)
    d = {n: v.to(dev) if isinstance(v, torch.Tensor) else v for n, v in c.items()}
    names = ("dy", "dweights", "dsum", "drms")
    kw = {} if need is None else {f"need_{n}": n in need for n in names}
    got = dict(zip(names, moe.moe_finalize_backward(**d, **kw)))
    torch.cuda.synchronize()
    refs, mags = rr.finalize_backward(c["dout"], c["fused_expert_output"], c["topk_weights"], k, c.get("residual_out"),
                                      c.get("rms_weight"), 1e-6, c.get("dresidual_out"))
    for n in names:
        if refs[n] is None or (need is not None and n not in need):
            assert got[n] is None, n
            continue
        v = got[n].cpu().double()
        tol = mags[n] * 2.0 ** -18 + (refs[n].abs() * 2.0 ** -8 if n in ("dy", "dsum") else 0) + 1e-38
        if n == "drms":
            tol = tol + mags[n] * 2.0 ** -24 * (T / 100)
        bad = (v - refs[n]).abs() - tol
        assert (bad <= 0).all(), f"{n}: {int((bad > 0).sum())} beyond, worst excess {bad.max():.3e}"


@pytest.mark.parametrize("T,H,k", [(1, 8, 1), (1, 7168, 8), (3, 264, 2), (130, 2048, 8), (7, 4104, 3), (40, 7168, 4),
                                   (2, 16384, 2), (700, 1024, 2), (5, 12288, 1), (33, 256, 32)])
def test_finalize_backward_shapes(cuda_dev, T, H, k):
    _check(cuda_dev, T, H, k)
    _check(cuda_dev, T, H, k, rms=False, dres=False)


@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("dres", [True, False])
@pytest.mark.parametrize("weights", [True, False])
def test_finalize_backward_variants(cuda_dev, rms, dres, weights):
    _check(cuda_dev, 20, 520, 4, rms, dres, weights)


def test_finalize_backward_parts(cuda_dev):
    for need in (("dy",), ("dweights",), ("dsum",), ("drms",), ("dy", "drms"), ("dweights", "dsum")):
        _check(cuda_dev, 20, 520, 4, need=need)


def test_finalize_backward_in_place_and_without_rows(cuda_dev):
    """dsum over dout or dresidual_out; the expert rows are not needed without dweights."""
    c = {n: v.to(cuda_dev) if isinstance(v, torch.Tensor) else v for n, v in _case(50, 1000, 3, True, True).items()}
    want = moe.moe_finalize_backward(**c)
    for over in ("dout", "dresidual_out"):
        d = dict(c, **{over: c[over].clone()})
        got = moe.moe_finalize_backward(**d, dsum=d[over])
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[2] is d[over]
    got = moe.moe_finalize_backward(**dict(c, fused_expert_output=None), need_dweights=False)
    assert torch.equal(got[0], want[0]) and got[1] is None


def test_finalize_backward_zero_rows_and_empty(cuda_dev):
    """A row of zeros has r = eps^-1/2 and a finite gradient; no tokens give zero drms."""
    c = _case(4, 256, 2, True, False)
    c["residual_out"][1] = 0
    d = {n: v.to(cuda_dev) if isinstance(v, torch.Tensor) else v for n, v in c.items()}
    got = moe.moe_finalize_backward(**d)
    refs, _ = rr.finalize_backward(c["dout"], c["fused_expert_output"], c["topk_weights"], 2, c["residual_out"],
                                   c["rms_weight"])
    assert torch.allclose(got[2].cpu().double(), refs["dsum"], rtol=2.0 ** -7, atol=1e-6 * refs["dsum"].abs().max())
    e = moe.moe_finalize_backward(torch.empty((0, 64), dtype=BF, device=cuda_dev), None,
                                  torch.empty((0, 2), device=cuda_dev), 2,
                                  residual_out=torch.empty((0, 64), dtype=BF, device=cuda_dev),
                                  rms_weight=torch.ones(64, dtype=BF, device=cuda_dev), need_dweights=False,
                                  drms=torch.ones(64, device=cuda_dev))
    assert (e[3] == 0).all()


def test_finalize_backward_graph_and_stream(cuda_dev):
    c = {n: v.to(cuda_dev) if isinstance(v, torch.Tensor) else v for n, v in _case(300, 2048, 4, True, True).items()}
    want = moe.moe_finalize_backward(**c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_finalize_backward(**c, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = dict(zip(("dy", "dweights", "dsum", "drms"), got))
    ws = torch.empty(moe.finalize_backward_workspace_size(300, 2048), dtype=torch.uint8, device=cuda_dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_finalize_backward(**c, **outs, ws=ws)
    for t in outs.values():
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs.values(), want))


def test_finalize_backward_offsets_past_32_bits(cuda_dev):
    """T * top_k * H past 2^31 elements: tokens at both ends."""
    T, H, k = 40_000, 7168, 8
    c = _case(8, H, k, False, False)
    dout = torch.zeros((T, H), dtype=BF, device=cuda_dev)
    y = torch.ones((T * k, H), dtype=BF, device=cuda_dev)
    w = torch.ones((T, k), device=cuda_dev)
    for t, n in ((dout, 4), (w, 4), (y, 4 * k)):
        src = {id(dout): c["dout"], id(w): c["topk_weights"], id(y): c["fused_expert_output"]}[id(t)].to(cuda_dev)
        t[:n], t[-n:] = src[:n], src[n:]
    dy, dw, dsum, _ = moe.moe_finalize_backward(dout, y, w, k)
    refs, mags = rr.finalize_backward(c["dout"], c["fused_expert_output"], c["topk_weights"], k)
    for name, v, n in (("dy", dy, 4 * k), ("dweights", dw, 4), ("dsum", dsum, 4)):
        v = torch.cat([v[:n], v[-n:]]).cpu().double()
        tol = mags[name] * 2.0 ** -18 + (refs[name].abs() * 2.0 ** -8 if name != "dweights" else 0) + 1e-38
        assert ((v - refs[name]).abs() <= tol).all(), name
    assert (dsum[4:-4] == 0).all() and (dw[4:-4] == 0).all()
