"""moe_route_grouped and its gradient against their fp64 definition.

The ids are the ones of exact arithmetic, so they are compared for equality (the cases hold no
two scores that fp64 cannot order).  Weights: expf within 1 ulp, a sum of at most 32 positive
terms (E terms for plain softmax scores, in lanes of E / 32 and 5 levels) and two divisions or
products: within 2^-20.  Gradients: the same errors in each factor, so 2^-19 of the terms'
magnitudes, and half a step of the output's type."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe
from oracle import router_ref as rr

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _check(dev, logits, top_k, bias=None, **kw):
    T = logits.shape[0]
    ids = torch.full((T + 1, top_k), -7, dtype=torch.int32, device=dev)  # a guard row behind the outputs
    w = torch.full((T + 1, top_k), -7.0, device=dev)
    moe.moe_route_grouped(logits.to(dev), top_k, None if bias is None else bias.to(dev), topk_ids=ids[:T],
                          topk_weights=w[:T], **kw)
    torch.cuda.synchronize()
    rid, rw = rr.route_grouped(logits, top_k, bias, **kw)
    got = ids[:T].cpu().numpy()
    bad = int((got != rid).any(1).sum())
    assert bad == 0, f"{bad} of {T} rows differ"
    err = np.abs(w[:T].cpu().double().numpy() - rw) - np.abs(rw) * 2.0 ** -20
    assert (err <= 2.0 ** -140).all(), f"weights: worst excess {err.max():.3e}"
    assert (ids[T] == -7).all() and (w[T] == -7.0).all()


# E, top_k, n_group, topk_group, group_top
LAYOUTS = [(256, 8, 8, 4, 2), (256, 8, 1, 1, 1), (128, 8, 1, 1, 1), (160, 6, 8, 3, 1), (64, 6, 1, 1, 1), (1, 1, 1, 1, 1),
           (2, 2, 1, 1, 1), (2, 1, 2, 1, 1), (33, 5, 3, 2, 2), (32, 32, 4, 4, 2), (1024, 32, 32, 16, 2), (1000, 7, 8, 2, 2),
           (384, 8, 1, 1, 1), (96, 4, 32, 9, 2), (17, 3, 1, 1, 1), (30, 2, 15, 1, 2), (1020, 8, 17, 5, 2),
           (999, 9, 3, 1, 2), (250, 7, 5, 2, 1), (512, 16, 16, 7, 2)]


@pytest.mark.parametrize("E,k,ng,tg,gt", LAYOUTS)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_layouts(cuda_dev, E, k, ng, tg, gt, score):
    g = torch.Generator().manual_seed(E * 31 + k)
    groups = dict(n_group=ng, topk_group=tg, group_top=gt, score=score)
    for T, dt, renorm, scale in ((1, F32, True, 1.0), (9, BF, False, 2.5), (67, F32, True, 2.5), (40, HF, True, 1.0)):
        logits = torch.randn((T, E), generator=g).to(dt)
        bias = torch.randint(-100, 101, (E,), generator=g).float() * 1e-3
        _check(cuda_dev, logits, k, bias, renormalize=renorm, scale=scale, **groups)
        _check(cuda_dev, logits, k, None, renormalize=renorm, scale=scale, **groups)
        _check(cuda_dev, logits, k, torch.zeros(E), renormalize=renorm, scale=scale, **groups)  # an untrained bias


@pytest.mark.parametrize("E,k,ng,tg,gt", [(256, 8, 8, 4, 2), (64, 8, 1, 1, 1), (48, 4, 4, 2, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_order_of_scores_that_fp32_cannot_tell(cuda_dev, E, k, ng, tg, gt, score):
    """Every biased score is 0.7 to within an fp32 rounding of the bias: only fp64 orders them."""
    T = 24
    g = torch.Generator().manual_seed(E)
    row = torch.randn((1, E), generator=g)
    s = torch.from_numpy(rr.scores(row, score))
    bias = (0.7 - s[0]).float()
    logits = row.expand(T, E).clone()
    # other tokens: a few logits a last place apart, the rest far below
    for t in range(1, T):
        at = torch.randperm(E, generator=g)[:k + 2]
        logits[t, at] += torch.randint(-2, 3, (k + 2,), generator=g) * 2.0 ** -23
    _check(cuda_dev, logits, k, bias, score=score, n_group=ng, topk_group=tg, group_top=gt)
    _check(cuda_dev, logits, k, None, score=score, n_group=ng, topk_group=tg, group_top=gt)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
def test_route_masks_and_special_values(cuda_dev, score, renorm, with_bias):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(F32).min
    g = torch.Generator().manual_seed(12)
    E = 12
    l = torch.randn((16, E), generator=g)
    l[0] = -inf                      # a row whose mask leaves nothing
    l[1] = nan
    l[2, 1:] = -inf                  # one expert left
    l[3, ::2] = -inf
    l[4, 3] = inf
    l[5, 2:4] = inf
    l[6] = low                       # masks of the type's lowest value
    l[7, :6] = low
    l[8, 4:8] = nan
    l[9] = 0.0                       # all equal
    l[10, 4:] = -inf                 # one group left
    l[11] = -100.0 - torch.arange(E)  # scores that underflow unless scaled
    l[12] = 40.0 + torch.arange(E) * 0  # sigmoid saturates
    l[13, 5] = -0.0
    bias = torch.randint(-50, 51, (E,), generator=g).float() * 1e-3 if with_bias else None
    for kw in (dict(), dict(n_group=3, topk_group=1, group_top=2), dict(n_group=4, topk_group=2, group_top=1)):
        _check(cuda_dev, l, 3, bias, score=score, renormalize=renorm, **kw)
    if with_bias:  # a bias may mask or force an expert
        bias[2], bias[7], bias[9] = -inf, nan, inf
        for kw in (dict(), dict(n_group=3, topk_group=2, group_top=2)):
            _check(cuda_dev, l, 4, bias, score=score, renormalize=renorm, **kw)


def test_route_many_tokens(cuda_dev):
    g = torch.Generator().manual_seed(77)
    logits = torch.randn((3001, 256), generator=g)
    bias = torch.randint(-100, 101, (256,), generator=g).float() * 1e-3
    _check(cuda_dev, logits, 8, bias, score="sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5)


def test_route_empty(cuda_dev):
    ids, w = moe.moe_route_grouped(torch.empty((0, 8), device=cuda_dev), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    dl = moe.moe_route_grouped_backward(w, torch.empty((0, 8), device=cuda_dev), ids)
    assert dl.shape == (0, 8)


def _check_backward(dev, logits, ids, dw, **kw):
    T, E = logits.shape
    out = torch.full((T + 1, E), 7.0, dtype=logits.dtype, device=dev)
    moe.moe_route_grouped_backward(dw.to(dev), logits.to(dev), ids.to(dev), dlogits=out[:T], **kw)
    torch.cuda.synchronize()
    ref, mag = rr.route_grouped_backward(dw, logits, ids, **kw)
    fi = torch.finfo(logits.dtype)
    err = np.abs(out[:T].cpu().double().numpy() - ref)
    tol = mag * 2.0 ** -19 + np.abs(ref) * fi.eps / 2 + fi.smallest_normal * fi.eps
    # a score below 2^-126 is a subnormal fp32 number, off by up to half of 2^-149, and dweights scale
    # multiplies that (scores of logits of -100 lie there)
    tol = tol + 2.0 ** -150 * np.abs(dw.numpy()).max(initial=0) * kw.get("scale", 1.0)
    assert (err <= tol).all(), f"worst excess {(err - tol).max():.3e}"
    assert (out[T] == 7.0).all()


@pytest.mark.parametrize("E,k", [(256, 8), (128, 8), (1, 1), (2, 2), (33, 5), (1000, 32), (1024, 7), (60, 1), (12, 12)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward(cuda_dev, E, k, score, renorm):
    g = torch.Generator().manual_seed(E + k)
    for T, dt in ((1, F32), (50, F32), (21, BF), (13, HF)):
        logits = (torch.randn((T, E), generator=g) * 2).to(dt)
        ids = torch.rand((T, E), generator=g).argsort(1)[:, :k].to(torch.int32).contiguous()
        dw = torch.randn((T, k), generator=g)
        _check_backward(cuda_dev, logits, ids, dw, score=score, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_masks_and_repeated_ids(cuda_dev, score, renorm):
    inf = float("inf")
    g = torch.Generator().manual_seed(3)
    l = torch.randn((8, 10), generator=g)
    l[0] = -inf
    l[1, :9] = -inf
    l[2, 4] = float("nan")
    l[3, 2] = inf
    l[4] = -100.0 - torch.arange(10)
    ids = torch.rand((8, 10), generator=g).argsort(1)[:, :4].to(torch.int32).contiguous()
    ids[2, 0], ids[3, 1], ids[5], ids[6, 2] = 4, 2, 3, ids[6, 0]  # ids that name an expert twice and four times
    _check_backward(cuda_dev, l, ids, torch.randn((8, 4), generator=g), score=score, renormalize=renorm)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_of_experts_that_the_bias_masks(cuda_dev, score, renorm):
    """Fewer experts than choices are left: the masked ones are chosen with the constant weight 0."""
    g = torch.Generator().manual_seed(8)
    l = torch.randn((20, 12), generator=g)
    bias = torch.full((12,), float("-inf"))
    bias[1], bias[4], bias[7], bias[9] = 0.1, float("nan"), -0.2, float("inf")
    ids, w = moe.moe_route_grouped(l.to(cuda_dev), 6, bias.to(cuda_dev), score=score, renormalize=renorm)
    assert int((w == 0).sum()) == 20 * 3
    dw = torch.randn((20, 6), generator=g)
    dl = moe.moe_route_grouped_backward(dw.to(cuda_dev), l.to(cuda_dev), ids, score=score, renormalize=renorm,
                                        bias=bias.to(cuda_dev))
    ref, mag = rr.route_grouped_backward(dw, l, ids, score, renorm, bias=bias)
    err = np.abs(dl.cpu().double().numpy() - ref)
    assert (err <= mag * 2.0 ** -19 + np.abs(ref) * 2.0 ** -24).all()


def test_route_backward_out_of_range_ids_are_recorded(cuda_dev):
    l = torch.randn((4, 8), device=cuda_dev)
    ids = torch.tensor([[0, 1], [8, 2], [-1, 3], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device=cuda_dev)
    dl = moe.moe_route_grouped_backward(torch.ones((4, 2), device=cuda_dev), l, ids, renormalize=False)
    assert moe.moe_device_status() == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_device_status() == moe.MOE_OK
    ref, _ = rr.route_grouped_backward(torch.ones((4, 2)), l, ids, renormalize=False)
    assert np.allclose(dl.cpu().numpy(), ref, rtol=1e-5, atol=1e-7)


def test_route_graph_and_stream(cuda_dev):
    g = torch.Generator().manual_seed(7)
    l, b = torch.randn((300, 256), generator=g).to(cuda_dev), (torch.rand(256, generator=g) * 0.1).to(cuda_dev)
    kw = dict(bias=b, n_group=8, topk_group=4, group_top=2)
    ids, w = moe.moe_route_grouped(l, 8, **kw)
    dl = moe.moe_route_grouped_backward(w, l, ids)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    i2, w2 = moe.moe_route_grouped(l, 8, stream=side, **kw)
    side.synchronize()
    assert torch.equal(i2, ids) and torch.equal(w2, w)
    graph, d2 = torch.cuda.CUDAGraph(), torch.empty_like(l)
    with torch.cuda.graph(graph):
        moe.moe_route_grouped(l, 8, topk_ids=i2, topk_weights=w2, **kw)
        moe.moe_route_grouped_backward(w2, l, i2, dlogits=d2)
    i2.zero_(), w2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(i2, ids) and torch.equal(w2, w) and torch.equal(d2, dl)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [True, False])
def test_route_peaked_and_repeated_logits(cuda_dev, score, with_bias):
    """Logits over a wide range (most softmax scores tiny) and rows with many equal values."""
    g = torch.Generator().manual_seed(21)
    for dt in (F32, BF):
        wide = (torch.randn((40, 64), generator=g) * 8).to(dt)
        few = torch.randint(-2, 3, (40, 64), generator=g).to(dt)
        for l in (wide, few):
            bias = torch.randint(-9, 10, (64,), generator=g).float() * 1e-2 if with_bias else None
            for kw in (dict(), dict(n_group=8, topk_group=3, group_top=2), dict(n_group=4, topk_group=2, group_top=1)):
                _check(cuda_dev, l, 8, bias, score=score, **kw)
                _check(cuda_dev, l, 12, bias, score=score, **kw)


@pytest.mark.parametrize("k", [5, 8, 12])
def test_route_masked_choices_behind_near_ones(cuda_dev, k):
    """Fewer experts than choices are left, some of them too close for fp32: the masked ones still follow by
    index, whatever their bias."""
    g = torch.Generator().manual_seed(5)
    bias = torch.randint(-100, 101, (36,), generator=g).float() * 1e-3
    l = torch.full((20, 36), float("-inf"))
    for t in range(20):
        at = torch.randperm(36, generator=g)[:6]
        l[t, at] = torch.randn(6, generator=g)
        s = torch.sigmoid(l[t, at].double())
        # two of them with the same biased score to 1e-7
        want = s[0] + bias[at[0]].double() - bias[at[1]].double()
        l[t, at[1]] = torch.log(want / (1 - want)).float() if 0 < want < 1 else l[t, at[1]]
    for kw in (dict(), dict(n_group=4, topk_group=2, group_top=2), dict(n_group=3, topk_group=3, group_top=1)):
        _check(cuda_dev, l, k, bias, **kw)


def test_route_offsets_past_32_bits(cuda_dev):
    """T * E past 2^32 bytes: the first and last rows of a large batch."""
    T, E, k = 9_000_000, 256, 8
    l = torch.randn((64, E), generator=torch.Generator().manual_seed(3)).to(BF)
    big = torch.zeros((T, E), dtype=BF, device=cuda_dev)
    big[:32], big[-32:] = l[:32].to(cuda_dev), l[32:].to(cuda_dev)
    ids, w = moe.moe_route_grouped(big, k, n_group=8, topk_group=4, group_top=2)
    dl = moe.moe_route_grouped_backward(w, big, ids)
    torch.cuda.synchronize()
    rid, rw = rr.route_grouped(l, k, n_group=8, topk_group=4, group_top=2)
    pick = lambda t: torch.cat([t[:32], t[-32:]]).cpu()  # noqa: E731
    assert np.array_equal(pick(ids).numpy(), rid)
    assert np.allclose(pick(w).double().numpy(), rw, rtol=2.0 ** -20, atol=0)
    ref, mag = rr.route_grouped_backward(pick(w), l, pick(ids))
    assert (np.abs(pick(dl).double().numpy() - ref) <= mag * 2.0 ** -19 + np.abs(ref) * 2.0 ** -8 + 1e-38).all()
