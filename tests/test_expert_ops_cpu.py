"""Refusals of the norm, the grouped products and the activation, before any launch: no GPU needed."""
import ctypes

import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe

P = ctypes.c_void_p
FAKE = P(256)  # never dereferenced: every call below fails its host-side checks
BF16, FP16, FP32, FP8 = moe.MOE_DT_BF16, moe.MOE_DT_FP16, moe.MOE_DT_FP32, moe.MOE_DT_FP8_E4M3
OK, BAD, UNSUP, WS = moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE
SORTED, SLOT, TOKEN = 0, 1, 2


def test_rmsnorm_refusals(moelib):
    fp8, token = moe.QUANT_CONFIGS["fp8"], moe.QUANT_CONFIGS["fp8_token"]

    def call(x=FAKE, r=None, w=FAKE, eps=1e-6, T=4, H=256, qc=None, out=FAKE, ro=None, q=None, sc=None):
        return moelib.moe_rmsnorm(x, r, w, eps, T, H, ctypes.byref(qc) if qc else None, out, ro, q, sc, None)

    odd = P(264)
    for kw in (dict(T=-1), dict(T=(1 << 30) + 1), dict(H=0), dict(H=12), dict(H=16392), dict(H=-8), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(w=None), dict(out=None),
               dict(q=FAKE), dict(sc=FAKE), dict(qc=fp8), dict(qc=fp8, q=FAKE), dict(qc=token, sc=FAKE), dict(x=odd),
               dict(r=odd), dict(w=odd), dict(out=odd), dict(ro=odd), dict(qc=fp8, q=odd, sc=FAKE),
               dict(qc=fp8, q=FAKE, sc=odd)):
        assert call(**kw) == BAD, kw
    for qc in (moe.QUANT_CONFIGS["fp8_tensor"], moe.QuantConfig(FP8, 64, FP8, 128, 128),
               moe.QuantConfig(moe.MOE_DT_NVFP4, 16, BF16, 0, 0)):
        assert call(qc=qc, q=FAKE, sc=FAKE) == UNSUP
    assert call(T=0, x=None, out=None) == OK


def test_grouped_linear_refusals(moelib):
    def call(x=FAKE, xr=SORTED, w=FAKE, o=FAKE, sl=FAKE, S=12, E=4, N=16, K=32, k=2, dt=BF16, out=FAKE, orow=SORTED, ws=FAKE,
             n=1 << 20):
        return moelib.moe_grouped_linear(x, xr, w, o, sl, S, E, N, K, k, dt, out, orow, ws, n, None)

    for kw in (dict(S=-1), dict(S=(1 << 30) + 1), dict(E=0), dict(E=1025), dict(N=0), dict(N=12), dict(K=0), dict(K=20),
               dict(N=(1 << 21) + 8), dict(K=(1 << 21) + 8), dict(k=0), dict(x=None), dict(w=None), dict(o=None),
               dict(out=None), dict(xr=3), dict(xr=-1), dict(orow=TOKEN), dict(orow=-1), dict(sl=None, xr=SLOT),
               dict(sl=None, orow=SLOT), dict(xr=TOKEN, k=5), dict(x=P(264)), dict(w=P(264)), dict(o=P(260)),
               dict(sl=P(260)), dict(out=P(264)), dict(ws=P(264))):
        assert call(**kw) == BAD, kw
    for kw in (dict(dt=FP32), dict(dt=FP8), dict(dt=9)):
        assert call(**kw) == UNSUP, kw
    size = moe.grouped_linear_workspace_size
    assert size(12, 4, 16, 32) == 0 and size(12, 4, 16, 32, "token") >= 12 * 32 * 2 and size(0, 4, 16, 32, "slot") == 0
    assert call(xr=TOKEN, ws=None) == WS and call(xr=SLOT, n=12 * 64 - 1) == WS
    assert call(S=0, x=None, out=None) == OK
    # sums of sizes that fit one by one
    assert call(S=1 << 30, N=1 << 21, E=1024, k=1) == UNSUP


def test_grouped_linear_backward_refusals(moelib):
    def call(d=FAKE, dr=SORTED, x=FAKE, xr=SORTED, w=FAKE, o=FAKE, sl=FAKE, S=12, E=4, N=16, K=32, k=2, dt=BF16, dx=FAKE,
             dxr=SORTED, dw=FAKE, wdt=BF16, acc=0, ws=FAKE, n=1 << 20):
        return moelib.moe_grouped_linear_backward(d, dr, x, xr, w, o, sl, S, E, N, K, k, dt, dx, dxr, dw, wdt, acc, ws, n,
                                                  None)

    for kw in (dict(S=-1), dict(E=0), dict(N=12), dict(K=4), dict(k=0), dict(d=None), dict(x=None), dict(w=None),
               dict(o=None), dict(dx=None, dw=None), dict(dr=3), dict(xr=3), dict(dxr=TOKEN), dict(sl=None, dr=SLOT),
               dict(sl=None, xr=SLOT), dict(sl=None, dxr=SLOT), dict(dr=TOKEN, k=5), dict(d=P(264)), dict(x=P(264)),
               dict(w=P(264)), dict(o=P(260)), dict(sl=P(260)), dict(dx=P(264)), dict(dw=P(264)), dict(ws=P(264))):
        assert call(**kw) == BAD, kw
    for kw in (dict(dt=FP32), dict(wdt=FP16), dict(dt=FP16, wdt=BF16), dict(wdt=FP8)):
        assert call(**kw) == UNSUP, kw
    size = moe.grouped_linear_backward_workspace_size
    assert size(0, 4, 16, 32) == 0 and size(12, 4, 16, 32) >= 4 * 256
    assert size(12, 4, 16, 32, "slot", "token") >= 12 * 16 * 2 + 12 * 32 * 2 + 4 * 256
    assert call(dr=SLOT, ws=None) == WS and call(xr=TOKEN, n=100) == WS and call(ws=None) == WS and call(n=1000) == WS
    assert call(dw=None, dr=SLOT, n=12 * 32 - 1) == WS


def test_activation_refusals(moelib):
    def fwd(gu=FAKE, S=4, I=16, dt=BF16, act=0, h=FAKE):
        return moelib.moe_activation(gu, S, I, dt, act, h, None)

    def bwd(dh=FAKE, gu=FAKE, S=4, I=16, dt=BF16, act=0, dgu=FAKE, h=None):
        return moelib.moe_activation_backward(dh, gu, S, I, dt, act, dgu, h, None)

    for call in (fwd, bwd):
        for kw in (dict(S=-1), dict(S=(1 << 30) + 1), dict(I=0), dict(I=12), dict(I=(1 << 21) + 8), dict(gu=None),
                   dict(gu=P(264)), dict(h=P(264))):
            assert call(**kw) == BAD, kw
        for kw in (dict(dt=FP32), dict(dt=FP8), dict(act=6), dict(act=-1)):
            assert call(**kw) == UNSUP, kw
        assert call(S=0, gu=None) == OK
    assert fwd(h=None) == BAD and bwd(dh=None) == BAD and bwd(dgu=None) == BAD
    assert bwd(dh=P(264)) == BAD and bwd(dgu=P(264)) == BAD
    assert fwd(S=1 << 30, I=1 << 21) == UNSUP


def test_python_refusals():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    o, sl = torch.zeros(5, dtype=torch.int32), torch.zeros(12, dtype=torch.int32)
    with pytest.raises(ValueError, match="quant"):
        moe.moe_rmsnorm(z(4, 16), z(16), quant="fp8_tensor")
    with pytest.raises(ValueError, match="q and q_scale"):
        moe.moe_rmsnorm(z(4, 16), z(16), q=z(4, 16, dt=torch.uint8))
    with pytest.raises(ValueError, match="x:"):
        moe.moe_rmsnorm(z(16), z(16))
    w = z(4, 16, 32)
    for kw, err, what in ((dict(x_rows="token"), ValueError, "sorted_slot"), (dict(out_rows="slot"), ValueError, "sorted_slot"),
                          (dict(sorted_slot=sl, x_rows="columns"), ValueError, "x_rows"),
                          (dict(sorted_slot=sl, out_rows="token"), ValueError, "out_rows"),
                          (dict(sorted_slot=sl, top_k=5, x_rows="token"), ValueError, "top_k"),
                          (dict(top_k=0), ValueError, "top_k"), (dict(top_k=2 ** 32 + 1), ValueError, "top_k")):
        with pytest.raises(err, match=what):
            moe.moe_grouped_linear(z(12, 32), w, o, **kw)
    with pytest.raises(TypeError, match="w:"):
        moe.moe_grouped_linear(z(12, 32), w.float(), o)
    with pytest.raises(ValueError, match="w, the rows"):
        moe.moe_grouped_linear(z(12, 32), w[0], o)
    with pytest.raises(ValueError, match="dw"):
        moe.moe_grouped_linear_backward(z(12, 16), z(12, 32), w, o, accumulate=True)
    with pytest.raises(TypeError, match="dw"):
        moe.moe_grouped_linear_backward(z(12, 16), z(12, 32), w, o, dw=z(4, 16, 32, dt=torch.float16))
    with pytest.raises(TypeError, match="dw"):
        moe.moe_grouped_linear_backward(z(12, 16), z(12, 32), w, o, dw=w.clone(), dw_dtype=torch.float32)
    for size in (moe.grouped_linear_workspace_size, moe.grouped_linear_backward_workspace_size):
        for sizes in ((2 ** 32 + 1, 4, 16, 32), (12, 4, 2 ** 31, 32), (12, 4, 16, -2 ** 32 + 32)):
            with pytest.raises(ValueError, match="2\\^31"):
                size(*sizes)
    with pytest.raises(ValueError, match="activation"):
        moe.moe_activation(z(4, 32), "relu")
    with pytest.raises(TypeError, match="gu"):
        moe.moe_activation(z(4, 32).float())
    with pytest.raises(ValueError, match="gu"):
        moe.moe_activation_backward(z(4, 16), z(4, 33))
