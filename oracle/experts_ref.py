"""Plain fp64 definitions of the RMSNorm in front of the layer, the experts' products over ragged groups of rows and
the activation between them, with the gradients (CPU, slow, no shared code with the GPU path)."""
from __future__ import annotations

import math

import torch


def _f64(t):
    return None if t is None else t.detach().cpu().double()


# ------------------------------------------------------------------ RMSNorm
def rmsnorm(x, weight, residual=None, eps=1e-6):
    """(n, v): the normalised rows and the sums that they are made from."""
    v = _f64(x) if residual is None else _f64(x) + _f64(residual)
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + eps) * _f64(weight), v


def row_scales(n, group):
    """max(amax, 1e-10) / 448 over groups of 128 columns (the last may be shorter), or the row (group -1)."""
    parts = [n] if group < 0 else n.split(group, 1)
    s = torch.stack([p.abs().amax(1).clamp(min=1e-10) / 448 for p in parts], 1)
    return s[:, 0] if group < 0 else s


def spread(scales, H):
    """Scales as one value per column."""
    return scales[:, None].expand(-1, H) if scales.dim() == 1 else scales.repeat_interleave(128, 1)[:, :H]


# ------------------------------------------------------------------ grouped products
def row_index(order, slots, S, top_k):
    """Row of a tensor in the given order for each sorted row."""
    if order == "sorted":
        return torch.arange(S)
    return slots.long() if order == "slot" else slots.long() // top_k


def grouped_linear(x, w, offsets, slots, top_k, x_rows="sorted", out_rows="sorted"):
    """(out, sum of |x||w| per element): dictionaries row of out -> values would be the literal reading; here tensors
    with NaN in the rows that belong to no group."""
    S = len(x) if slots is None else len(slots)
    x, w, o = _f64(x), _f64(w), offsets.tolist()
    rx, ro = row_index(x_rows, slots, S, top_k), row_index(out_rows, slots, S, top_k)
    out = torch.full((S, w.shape[1]), float("nan"), dtype=torch.float64)
    mag = torch.zeros_like(out)
    for e in range(w.shape[0]):
        for p in range(o[e], o[e + 1]):
            out[ro[p]] = w[e] @ x[rx[p]]
            mag[ro[p]] = w[e].abs() @ x[rx[p]].abs()
    return out, mag


def grouped_linear_backward(dout, x, w, offsets, slots, top_k, dout_rows="sorted", x_rows="sorted", dx_rows="sorted"):
    """(dx, its magnitudes, dw, its magnitudes)."""
    S = len(dout) if slots is None else len(slots)
    dout, x, w, o = _f64(dout), _f64(x), _f64(w), offsets.tolist()
    rd, rx, ro = (row_index(r, slots, S, top_k) for r in (dout_rows, x_rows, dx_rows))
    dx = torch.full((S, w.shape[2]), float("nan"), dtype=torch.float64)
    dxm, dw = torch.zeros_like(dx), torch.zeros_like(w)
    dwm = torch.zeros_like(w)
    for e in range(w.shape[0]):
        at = torch.arange(o[e], o[e + 1])
        d, v = dout[rd[at]], x[rx[at]]
        dx[ro[at]], dxm[ro[at]] = d @ w[e], d.abs() @ w[e].abs()
        dw[e], dwm[e] = d.T @ v, d.abs().T @ v.abs()
    return dx, dxm, dw, dwm


# ------------------------------------------------------------------ activation
def _gate(g, name):
    """act(g) and act'(g)."""
    if name.startswith("silu"):
        q = torch.special.expit(g)
        return g * q, q + g * q * (1 - q)
    if name.startswith("gelu") and name != "gelu_tanh":
        phi = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        return g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        q = torch.special.expit(2 * a * (g + 0.044715 * g ** 3))
        return g * q, q + 2 * a * (1 + 3 * 0.044715 * g * g) * g * q * (1 - q)
    assert name == "swigluoai"
    c = torch.clamp(g, max=7.0)
    q = torch.special.expit(1.702 * c)
    return c * q, torch.where(g > 7, 0.0, q + 1.702 * c * q * (1 - q))


def activation(gu, name):
    """(h, what act(g) is multiplied by, g)."""
    gu = _f64(gu)
    if name.endswith("_no_mul"):
        return _gate(gu, name)[0], torch.ones_like(gu), gu
    g, u = gu.chunk(2, 1)
    m = torch.clamp(u, -7.0, 7.0) + 1 if name == "swigluoai" else u
    return _gate(g, name)[0] * m, m, g


def activation_backward(dh, gu, name):
    dh, gu = _f64(dh), _f64(gu)
    _, m, g = activation(gu, name)
    a, slope = _gate(g, name)
    if name.endswith("_no_mul"):
        return dh * slope
    du = dh * a
    if name == "swigluoai":
        du = torch.where(gu.chunk(2, 1)[1].abs() > 7, 0.0, du)
    return torch.cat([dh * slope * m, du], 1)
