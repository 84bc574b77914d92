"""The fp64 definitions of the norm, the grouped products and the activation against autograd, differences and
hand-made cases."""
import pytest
import torch

from oracle import experts_ref as er
from oracle import moe_ref

ACTS = moe_ref.ACTIVATIONS


def test_rmsnorm_by_hand():
    x = torch.tensor([[3.0, -4.0], [0.0, 0.0]])
    n, v = er.rmsnorm(x, torch.tensor([1.0, 2.0]), torch.tensor([[0.0, 0.0], [1.0, 1.0]]), eps=0.0)
    r = (2 / 25) ** 0.5
    assert torch.allclose(n, torch.tensor([[3 * r, -8 * r], [1.0, 2.0]], dtype=torch.float64), rtol=1e-14)
    assert v.tolist() == [[3, -4], [1, 1]]
    s = er.row_scales(torch.tensor([[1.0] * 128 + [-3.0] * 8, [0.0] * 136], dtype=torch.float64), 128)
    assert torch.allclose(s * 448, torch.tensor([[1, 3], [1e-10, 1e-10]], dtype=torch.float64), rtol=1e-14)
    assert er.spread(s, 136).shape == (2, 136) and er.spread(s, 136)[0, 130] == s[0, 1]


@pytest.mark.parametrize("name", ACTS)
def test_activation_is_the_experts(name):
    gu = torch.randn((5, 16), generator=torch.Generator().manual_seed(1)) * 4
    assert torch.allclose(er.activation(gu, name)[0], moe_ref.activation(gu.double(), name), rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("name", ACTS)
def test_activation_gradient(name):
    g = torch.Generator().manual_seed(2)
    gu = torch.randn((6, 16), generator=g, dtype=torch.float64) * 5
    dh = torch.randn((6, 16 if name.endswith("no_mul") else 8), generator=g, dtype=torch.float64)
    want = er.activation_backward(dh, gu, name)
    v = gu.clone().requires_grad_(True)
    got, = torch.autograd.grad(moe_ref.activation(v, name), v, dh)
    assert torch.allclose(got, want, rtol=1e-10, atol=1e-12)
    for i, j in ((0, 0), (3, 5), (5, 15)):  # and differences (away from the clamps' corners)
        if (gu[i, j].abs() - 7).abs() < 1e-3:
            continue
        a, b = gu.clone(), gu.clone()
        a[i, j] += 1e-6
        b[i, j] -= 1e-6
        slope = ((er.activation(a, name)[0] - er.activation(b, name)[0]) * dh).sum() / 2e-6
        assert abs(slope - want[i, j]) < 1e-7 * (1 + abs(want[i, j]))


def test_grouped_products_and_gradients():
    g = torch.Generator().manual_seed(3)
    T, top_k, E, N, K = 5, 2, 4, 3, 6
    slots = torch.randperm(T * top_k, generator=g)
    offsets = torch.tensor([0, 4, 4, 5, 9])  # (the last sorted row belongs to no group)
    x = torch.randn((T, K), generator=g, dtype=torch.float64).requires_grad_(True)
    w = torch.randn((E, N, K), generator=g, dtype=torch.float64).requires_grad_(True)
    dout = torch.randn((T * top_k, N), generator=g, dtype=torch.float64)
    # by slots: the expert of each slot, or none
    out = torch.zeros((T * top_k, N), dtype=torch.float64)
    rows = []
    for e in range(E):
        for p in range(offsets[e], offsets[e + 1]):
            f = int(slots[p])
            rows.append((f, x[f // top_k] @ w[e].T))
    for f, r in rows:
        out = out.index_copy(0, torch.tensor([f]), r[None])
    got, mag = er.grouped_linear(x, w, offsets, slots, top_k, "token", "slot")
    left = int(slots[9])
    assert torch.isnan(got[left]).all() and (mag[left] == 0).all()
    keep = [f for f, _ in rows]
    assert torch.allclose(got[keep], out[keep].detach(), rtol=1e-12)
    dx, dw = torch.autograd.grad((out * dout).sum(), (x, w))
    gx, _, gw, _ = er.grouped_linear_backward(dout, x, w, offsets, slots, top_k, "slot", "token", "slot")
    assert torch.allclose(gw, dw, rtol=1e-12, atol=1e-14) and (gw[1] == 0).all()
    assert torch.allclose(torch.nan_to_num(gx).view(T, top_k, K).sum(1), dx, rtol=1e-12, atol=1e-14)
    # sorted orders are the same rows elsewhere
    sx = x.detach()[slots // top_k]
    assert torch.equal(er.grouped_linear(sx, w, offsets, None, 1)[0][:9], got[slots[:9]])
