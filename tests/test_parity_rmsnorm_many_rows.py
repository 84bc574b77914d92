"""moe_rmsnorm of 2048 rows and more, whose CTAs take several rows at a time and end with fewer.

Tolerances: as in test_parity_rmsnorm (32 additions a thread at most, and fewer warps a row)."""
import pytest
import torch

from mixture_experts_layer_tokens_gb300 import moe
from test_parity_rmsnorm import BF, _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("quant", [None, "fp8", "fp8_token"])
@pytest.mark.parametrize("T,H", [(2048, 512), (2500, 1032), (3001, 2056), (2047, 2056), (2050, 5000)])
def test_many_rows(cuda_dev, T, H, quant):
    for residual in (True, False):
        x, res, w = _inputs(T, H, residual=residual)
        d = lambda t: None if t is None else t.to(cuda_dev)  # noqa: E731
        for need_out in (True, False) if quant else (True,):
            outs = moe.moe_rmsnorm(d(x), d(w), residual=d(res), quant=quant, need_out=need_out)
            assert (outs[0] is None) == (not need_out) and (outs[1] is None) == (res is None)
            _check(outs, x, res, w, quant)


def test_many_of_the_longest_rows(cuda_dev):
    x, res, w = _inputs(2050, 16384)
    _check(moe.moe_rmsnorm(x.to(cuda_dev), w.to(cuda_dev), residual=res.to(cuda_dev), quant="fp8_token"), x, res, w,
           "fp8_token")
    _check(moe.moe_rmsnorm(x.to(cuda_dev), w.to(cuda_dev), quant="fp8"), x, None, w, "fp8")


@pytest.mark.parametrize("quant", ["fp8", "fp8_token"])
@pytest.mark.parametrize("T,H", [(2500, 1032), (2049, 512)])
def test_many_rows_are_their_own(cuda_dev, T, H, quant):
    """A NaN or an infinity changes its row alone, in a full turn and in the last one; outputs end where they end, and
    every call gives the same bits."""
    x, res, w = (t.to(cuda_dev) for t in _inputs(T, H))
    store = [torch.full((T + 1, H), 7, dtype=t, device=cuda_dev) for t in (BF, BF, torch.uint8)]
    store.append(torch.full((T + 1, (H + 127) // 128) if quant == "fp8" else (T + 1,), 7.0, device=cuda_dev))
    out, total, q, scale = (t[:T] for t in store)
    call = lambda: moe.moe_rmsnorm(x, w, residual=res, quant=quant, out=out, residual_out=total, q=q,  # noqa: E731
                                   q_scale=scale)
    first = [t.clone() for t in call()]
    assert all(torch.equal(a, b) for a, b in zip(first, call()))
    spoilt = [0, T // 2, T - 1]
    x[0, H - 1], x[T // 2, 3], res[T - 1, H // 2] = float("inf"), float("nan"), float("nan")
    odd = call()
    keep = torch.ones(T, dtype=torch.bool, device=cuda_dev)
    keep[spoilt] = False
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(first, odd))
    assert torch.isnan(odd[0][spoilt[1:]]).all() and torch.isnan(odd[0][0, H - 1])
    assert all(bool((t[T] == 7).all()) for t in store)
