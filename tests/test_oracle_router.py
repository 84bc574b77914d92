"""Pins of the fp64 definitions in oracle/router_ref.py: against torch's autograd, finite
differences, brute force and hand-made cases."""
import itertools
import math

import numpy as np
import pytest
import torch

from oracle import moe_ref, router_ref as rr


@pytest.mark.parametrize("activation", ["none", "silu", "gelu", "gelu_tanh"])
def test_linear_and_gradients_against_autograd(activation):
    g = torch.Generator().manual_seed(3)
    x = torch.randn((5, 16), generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn((7, 16), generator=g, dtype=torch.float64, requires_grad=True)
    b = torch.randn((7,), generator=g, dtype=torch.float64, requires_grad=True)
    d = torch.randn((5, 7), generator=g, dtype=torch.float64)
    f = {"none": lambda z: z, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[activation]
    z = x @ w.T + b
    out, zr, _ = rr.linear(x, w, b, None, activation)
    assert torch.allclose(out, f(z), rtol=1e-12, atol=1e-12) and torch.allclose(zr, z)
    want = torch.autograd.grad((f(z) * d).sum(), (x, w, b))
    got, mags, _ = rr.linear_backward(d, x, w, z, activation)
    assert all((m >= g.abs() - 1e-12).all() for m, g in zip(mags, got))
    for a, e in zip(got, want):
        assert torch.allclose(a, e, rtol=1e-10, atol=1e-12)


def test_route_matches_the_plain_router_without_bias_or_groups():
    logits = torch.randn((50, 12), generator=torch.Generator().manual_seed(1))
    ids, w = rr.route_grouped(logits, 3, score="softmax")
    rid, rw = moe_ref.route_softmax_renorm(logits, 3)
    # (that router's weights are rounded to fp32 once: half a step is 2^-24 of the value)
    assert np.array_equal(ids, rid.numpy()) and np.allclose(w, rw.double().numpy(), rtol=2.0 ** -24, atol=0)
    # sigmoid scores keep the logits' order
    assert np.array_equal(rr.route_grouped(logits, 3, score="sigmoid")[0], ids)


def test_route_choice_is_the_best_allowed_subset():
    g = torch.Generator().manual_seed(5)
    logits, bias = torch.randn((20, 12), generator=g), torch.randn(12, generator=g) * 0.3
    s = rr.scores(logits, "sigmoid")
    for group_top in (1, 2):
        ids, _ = rr.route_grouped(logits, 3, bias, "sigmoid", 4, 2, group_top)
        for t in range(20):
            c = s[t] + bias.double().numpy()
            best = max(itertools.combinations(range(4), 2),
                       key=lambda k: sum(np.sort(c[3 * q:3 * q + 3])[-group_top:].sum() for q in k))
            pool = [e for e in range(12) if e // 3 in best]
            top = max(itertools.combinations(pool, 3), key=lambda k: sum(c[e] for e in k))
            assert sorted(ids[t]) == sorted(top)
            assert all(c[a] >= c[b] for a, b in zip(ids[t], ids[t][1:]))


def test_route_hand_made_cases():
    inf, nan = math.inf, math.nan
    # two masked experts of four: chosen last, lower index first, weight 0
    ids, w = rr.route_grouped(torch.tensor([[-inf, 1.0, nan, 2.0]]), 4, score="softmax", scale=2.0)
    assert ids.tolist() == [[3, 1, 0, 2]] and w[0, 2:].tolist() == [0, 0] and math.isclose(w[0].sum(), 2.0)
    # nothing left: all weights 0
    ids, w = rr.route_grouped(torch.full((1, 4), -inf), 2)
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0, 0]]
    # +inf counts as a number: two of them share
    ids, w = rr.route_grouped(torch.tensor([[0.0, inf, inf]]), 2, score="softmax")
    assert ids.tolist() == [[1, 2]] and w.tolist() == [[0.5, 0.5]]
    # a group counts the experts it has: {2.0 masked-partner} against {0.6, 0.6}
    ids, _ = rr.route_grouped(torch.tensor([[3.0, -inf, 0.0, 0.0]]), 1, torch.tensor([0.2, 0, 0, 0]), "sigmoid", 2, 1, 2)
    assert ids.tolist() == [[0]]  # 0.95 + 0.2 against 1.0
    # very negative logits keep their ratio when renormalised
    _, w = rr.route_grouped(torch.tensor([[-200.0, -201.0]]), 2)
    assert math.isclose(w[0, 0] / w[0, 1], math.e, rel_tol=1e-12)
    # equal scores: the lower index; the bias moves the choice and not the weight
    ids, w = rr.route_grouped(torch.zeros((1, 4)), 2, torch.tensor([0.0, 0.0, 0.1, 0.0]), renormalize=False)
    assert ids.tolist() == [[2, 0]] and w.tolist() == [[0.5, 0.5]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(score, renorm):
    g = torch.Generator().manual_seed(9)
    l = torch.randn((4, 6), generator=g, dtype=torch.float64)
    ids = torch.tensor([[0, 3, 5], [1, 2, 4], [5, 1, 0], [2, 2, 3]])  # the last row names an expert twice
    dw = torch.randn((4, 3), generator=g, dtype=torch.float64)

    def f(l):
        s = rr.scores(l, score)
        w = np.take_along_axis(s, ids.numpy(), 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
        return (w * 2.5 * dw.numpy()).sum()

    got, mag = rr.route_grouped_backward(dw, l, ids, score, renorm, 2.5)
    for t, e in itertools.product(range(4), range(6)):
        a, b = l.clone(), l.clone()
        a[t, e] += 1e-5
        b[t, e] -= 1e-5
        assert abs((f(a) - f(b)) / 2e-5 - got[t, e]) < 1e-8
    assert (mag >= np.abs(got) - 1e-15).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_of_masked_choices_against_differences(score, renorm):
    """More choices than experts: what the bias masks is chosen with the constant weight 0."""
    g = torch.Generator().manual_seed(10)
    l = torch.randn((2, 6), generator=g, dtype=torch.float64)
    bias = torch.tensor([0.1, float("-inf"), 0.0, float("nan"), float("-inf"), -0.2])
    dw = torch.randn((2, 5), generator=g, dtype=torch.float64)
    ids, _ = rr.route_grouped(l, 5, bias, score=score, renormalize=renorm)
    assert sorted(ids[0, :3]) == [0, 2, 5] and ids[0, 3:].tolist() == [1, 3]

    def f(l):
        got, w = rr.route_grouped(l, 5, bias, score=score, renormalize=renorm, scale=2.5)
        assert (got == ids).all()
        return (w * dw.numpy()).sum()

    got, mag = rr.route_grouped_backward(dw, l, torch.from_numpy(ids), score, renorm, 2.5, bias)
    for t, e in itertools.product(range(2), range(6)):
        a, b = l.clone(), l.clone()
        a[t, e] += 1e-5
        b[t, e] -= 1e-5
        assert abs((f(a) - f(b)) / 2e-5 - got[t, e]) < 1e-8
    assert (mag >= np.abs(got) - 1e-15).all()


@pytest.mark.parametrize("rms", [True, False])
def test_finalize_gradient_against_autograd(rms):
    g = torch.Generator().manual_seed(4)
    T, H, k = 3, 16, 2
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    y, w, sh = rnd(T * k, H).requires_grad_(True), rnd(T, k).requires_grad_(True), rnd(T, H).requires_grad_(True)
    gamma, d, dr = rnd(H).requires_grad_(True), rnd(T, H), rnd(T, H)
    o = (w[:, :, None] * y.view(T, k, H)).sum(1) + sh
    out = o * (o.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt() * gamma if rms else o
    wants = torch.autograd.grad((out * d).sum() + (o * dr).sum(), (y, w, sh, gamma), allow_unused=True)
    got, mags = rr.finalize_backward(d, y, w, k, o if rms else None, gamma if rms else None, 1e-6, dr)
    for name, want in zip(("dy", "dweights", "dsum", "drms"), wants):
        if want is None:
            assert got[name] is None
            continue
        assert torch.allclose(got[name], want, rtol=1e-10, atol=1e-12), name
        assert (mags[name] >= got[name].abs() - 1e-12).all(), name
