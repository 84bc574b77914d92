"""Refusals of the linear, grouped-route and finalize-gradient calls, before any launch: no GPU needed."""
import ctypes

import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe

P = ctypes.c_void_p
FAKE = P(256)  # never dereferenced: every call below fails its host-side checks
BF16, FP16, FP32, FP8 = moe.MOE_DT_BF16, moe.MOE_DT_FP16, moe.MOE_DT_FP32, moe.MOE_DT_FP8_E4M3
BAD, UNSUP, WS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE


def test_linear_refusals(moelib):
    def call(x=FAKE, w=FAKE, b=None, r=None, M=4, N=8, K=64, dt=BF16, act=0, odt=BF16, out=FAKE, pre=None):
        return moelib.moe_linear(x, w, b, r, M, N, K, dt, act, odt, out, pre, None)

    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(K=4), dict(K=68), dict(x=None), dict(w=None), dict(out=None),
               dict(x=P(264)), dict(w=P(258)), dict(b=P(260)), dict(r=P(264)), dict(out=P(2)), dict(pre=P(8)),
               dict(N=(1 << 21) + 1), dict(M=(1 << 30) + 1), dict(K=(1 << 30) + 8)):
        assert call(**kw) == BAD, kw
    for kw in (dict(dt=FP32), dict(dt=FP8), dict(dt=9), dict(odt=FP16), dict(dt=FP16, odt=BF16), dict(odt=FP8),
               dict(act=4), dict(act=-1)):
        assert call(**kw) == UNSUP, kw
    assert call(M=0, x=None, out=None) == moe.MOE_OK


def test_linear_backward_refusals(moelib):
    def call(d=FAKE, ddt=BF16, x=FAKE, w=FAKE, pre=None, M=4, N=8, K=64, dt=BF16, act=0, dx=FAKE, dw=FAKE, db=None,
             ws=FAKE, n=1 << 20):
        return moelib.moe_linear_backward(d, ddt, x, w, pre, M, N, K, dt, act, dx, dw, db, ws, n, None)

    for kw in (dict(M=-1), dict(N=0), dict(K=12), dict(d=None), dict(x=None), dict(w=None), dict(act=1),
               dict(dx=None, dw=None), dict(dx=P(8)), dict(dw=P(8)), dict(db=P(8)), dict(d=P(8)), dict(pre=P(8)),
               dict(ws=P(8))):
        assert call(**kw) == BAD, kw
    for kw in (dict(ddt=FP16), dict(dt=FP32), dict(act=7)):
        assert call(**kw) == UNSUP, kw
    assert call(ws=None) == WS and call(n=16) == WS
    size = moe.linear_backward_workspace_size
    assert size(0, 8, 64) == 0
    assert size(100, 33, 64) >= 100 * 40 * 2 + 2 * 33 * 4
    # bounded partial sums however many rows
    assert size(1 << 24, 8, 8) <= (1 << 24) * 16 + 256 + 1024 * 8 * 4


def _cfg(score=1, n_group=1, topk_group=1, group_top=1, renorm=1, scale=1.0):
    return ctypes.byref(moe.RouteConfig(score, n_group, topk_group, group_top, renorm, scale))


def test_route_grouped_refusals(moelib):
    def call(l=FAKE, dt=FP32, b=None, T=4, E=16, k=2, cfg=None, ids=FAKE, w=FAKE):
        return moelib.moe_route_grouped(l, dt, b, T, E, k, cfg or _cfg(), ids, w, None)

    for kw in (dict(T=-1), dict(T=(1 << 30) + 1), dict(E=0), dict(E=1025), dict(k=0), dict(k=17), dict(k=33, E=64), dict(l=None), dict(ids=None),
               dict(w=None), dict(l=P(4)), dict(b=P(4)), dict(ids=P(4)), dict(w=P(4)), dict(cfg=_cfg(score=2)),
               dict(cfg=_cfg(n_group=0)), dict(cfg=_cfg(n_group=3)), dict(cfg=_cfg(n_group=33), E=66),
               dict(cfg=_cfg(n_group=4, topk_group=0)), dict(cfg=_cfg(n_group=4, topk_group=5)),
               dict(cfg=_cfg(n_group=8, topk_group=2), k=5), dict(cfg=_cfg(group_top=3)), dict(cfg=_cfg(group_top=0)),
               dict(cfg=_cfg(n_group=16, topk_group=4, group_top=2)), dict(cfg=_cfg(scale=float("inf"))),
               dict(cfg=_cfg(scale=float("nan")))):
        assert call(**kw) == BAD, kw
    assert call(dt=FP8) == UNSUP and call(dt=moe.MOE_DT_NVFP4) == UNSUP
    assert moelib.moe_route_grouped(FAKE, FP32, None, 4, 16, 2, None, FAKE, FAKE, None) == BAD
    assert call(T=0, l=None, ids=None, w=None) == moe.MOE_OK


def test_route_grouped_backward_refusals(moelib):
    def call(dw=FAKE, l=FAKE, dt=FP32, b=None, ids=FAKE, T=4, E=16, k=2, cfg=None, dl=FAKE):
        return moelib.moe_route_grouped_backward(dw, l, dt, b, ids, T, E, k, cfg or _cfg(), dl, None)

    for kw in (dict(T=-1), dict(E=0), dict(k=17), dict(dw=None), dict(l=None), dict(ids=None), dict(dl=None),
               dict(dl=P(4)), dict(b=P(4)), dict(cfg=_cfg(score=5))):
        assert call(**kw) == BAD, kw
    assert call(dt=FP8) == UNSUP
    assert call(T=0, dw=None) == moe.MOE_OK


def test_finalize_backward_refusals(moelib):
    def call(d=FAKE, dr=None, o=FAKE, g=FAKE, eps=1e-6, y=FAKE, w=FAKE, T=4, H=64, k=2, dy=FAKE, dw=FAKE, ds=FAKE,
             drms=FAKE, ws=FAKE, n=1 << 20):
        return moelib.moe_finalize_backward(d, dr, o, g, eps, y, w, T, H, k, dy, dw, ds, drms, ws, n, None)

    for kw in (dict(T=-1), dict(T=(1 << 30) + 1), dict(H=0), dict(H=60), dict(k=0), dict(k=33), dict(eps=-1.0), dict(d=None), dict(o=None),
               dict(g=None), dict(y=None), dict(w=None), dict(dy=None, dw=None, ds=None, drms=None), dict(d=P(8)),
               dict(dy=P(8)), dict(drms=P(8)), dict(ws=P(8)), dict(eps=float("nan"))):
        assert call(**kw) == BAD, kw
    assert call(H=16392) == UNSUP
    assert call(ws=None) == WS and call(n=16) == WS
    assert moe.finalize_backward_workspace_size(0, 64) == 0


def test_binding_refusals_without_a_gpu():
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.moe_linear(x, w, activation="relu6")
    with pytest.raises(TypeError):
        moe.moe_linear(x.float(), w)
    with pytest.raises(TypeError):
        moe.moe_linear(x, w, out=torch.zeros((4, 8), dtype=torch.float16))
    with pytest.raises(TypeError):
        moe.moe_linear_backward(torch.zeros((4, 8), dtype=torch.float16), x, w)
    with pytest.raises(ValueError):
        moe.moe_route_grouped(torch.zeros((4, 8)), 2, score="tanh")
    with pytest.raises(TypeError):
        moe.moe_route_grouped(torch.zeros((4, 8), dtype=torch.float64), 2)
    # sizes past 32 bits are refused, not cut off
    meta = lambda *shape, t=torch.bfloat16: torch.empty(shape, dtype=t, device="meta")  # noqa: E731
    for call in (lambda: moe.moe_linear(meta(2 ** 32 + 4, 64), meta(8, 64)),
                 lambda: moe.moe_linear(meta(4, 64), meta(2 ** 32 + 8, 64)),
                 lambda: moe.moe_linear_backward(meta(4, 8), meta(4, 2 ** 32 + 8), meta(8, 2 ** 32 + 8)),
                 lambda: moe.moe_route_grouped(meta(2 ** 32 + 4, 16), 2),
                 lambda: moe.moe_route_grouped(meta(4, 2 ** 32 + 16), 2),
                 lambda: moe.moe_route_grouped(meta(4, 16), 2 ** 32 + 2),
                 lambda: moe.moe_route_grouped(meta(4, 16), -1),
                 lambda: moe.moe_route_grouped_backward(meta(4, 2), meta(2 ** 32 + 4, 16), meta(4, 2)),
                 lambda: moe.moe_finalize_backward(meta(2 ** 32 + 4, 64), None, None, 2),
                 lambda: moe.moe_finalize_backward(meta(4, 64), None, None, 0)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
    # the per-argument check: type, shape, contiguity, device
    ok = torch.zeros((4, 8))
    for t, err in ((ok.double(), TypeError), (ok[:3], ValueError), (torch.zeros((8, 4)).T, ValueError), (ok, ValueError)):
        with pytest.raises(err):
            moe._tensor(t, torch.float32, (4, 8), "t", 0)
    assert moe._tensor(None, torch.float32, (4, 8), "t", 0) is None
