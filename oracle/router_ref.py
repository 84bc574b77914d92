"""Plain fp64 definitions of the linear projection, the grouped router and the gradients
around them (CPU, slow, no shared code with the GPU path)."""
from __future__ import annotations

import math

import numpy as np
import torch


def _f64(t):
    return None if t is None else t.detach().cpu().double()


# ------------------------------------------------------------------ linear projection
def act(z: torch.Tensor, name: str) -> torch.Tensor:
    if name == "none":
        return z
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return z * 0.5 * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    raise ValueError(name)


def act_grad(z: torch.Tensor, name: str) -> torch.Tensor:
    if name == "none":
        return torch.ones_like(z)
    if name == "silu":
        q = 1.0 / (1.0 + torch.exp(-z))
        return q + z * q * (1.0 - q)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    raise ValueError(name)


def linear(x, w, bias=None, residual=None, activation="none"):
    """(out, z) of act(x w^T + bias) + residual, and sum |x||w| (+ |bias|) per element."""
    x, w = _f64(x), _f64(w)
    z, mag = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, mag = z + _f64(bias), mag + _f64(bias).abs()
    out = act(z, activation)
    if residual is not None:
        out = out + _f64(residual)
    return out, z, mag


def linear_backward(dout, x, w, preact=None, activation="none"):
    """(dx, dw, dbias), and the sums of absolute values of dz w, dz x, dz and of dout w, dout x, dout (what an
    error of act' multiplies) that bound their errors."""
    dout, x, w = _f64(dout), _f64(x), _f64(w)
    dz = dout if activation == "none" else dout * act_grad(_f64(preact), activation)
    sums = lambda a: (a @ w.abs(), a.T @ x.abs(), a.sum(0))  # noqa: E731
    return (dz @ w, dz.T @ x, dz.sum(0)), sums(dz.abs()), sums(dout.abs())


# ------------------------------------------------------------------ grouped route
def _clean(logits):
    l = logits.detach().cpu().double().numpy().copy()
    l[np.isnan(l)] = -np.inf
    return np.minimum(l, np.finfo(np.float32).max)


def scores(logits, score):
    l = _clean(logits)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    m = l.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(np.isneginf(l), 0.0, np.exp(l - m))
    s = e.sum(1, keepdims=True)
    return np.where(s > 0, e / np.where(s > 0, s, 1), 0.0)


def route_grouped(logits, top_k, bias=None, score="sigmoid", n_group=1, topk_group=1, group_top=1, renormalize=True,
                  scale=1.0):
    """(topk_ids, topk_weights) as numpy arrays, one token at a time by sorting tuples."""
    l, s = _clean(logits), scores(logits, score)
    T, E = l.shape
    b = np.zeros(E) if bias is None else bias.detach().cpu().double().numpy()
    # without a bias the logits' order is the scores', however close these are to 1
    sw = l if bias is None and group_top == 1 else s
    size = E // n_group
    ids, ws = np.zeros((T, top_k), np.int32), np.zeros((T, top_k))
    for t in range(T):
        masked = np.isneginf(l[t]) | np.isnan(b) | np.isneginf(b)
        c = np.where(masked, -np.inf, sw[t] + np.where(masked, 0.0, b))
        group = []
        for g in range(n_group):
            best = sorted((c[e] for e in range(g * size, (g + 1) * size) if not masked[e]), reverse=True)[:group_top]
            group.append(sum(best) if best else -math.inf)
        kept = sorted(range(n_group), key=lambda g: (-group[g], g))[:topk_group]
        pool = [e for e in range(E) if e // size in kept]
        # (masked experts are equal among themselves: by index alone)
        pool.sort(key=lambda e: (-c[e], -l[t, e] if not masked[e] else 0.0, e))
        ids[t] = pool[:top_k]
        w = np.array([0.0 if masked[e] else s[t, e] for e in ids[t]])
        if renormalize:
            live = [e for e in ids[t] if not masked[e]]
            w[:] = 0.0
            if live:  # s_j / sum s, scaled so that nothing underflows
                top = max(l[t, e] for e in live)
                part = {e: (math.exp(l[t, e] - top) if score == "softmax" else
                            math.exp(min(l[t, e], 0.0) - min(top, 0.0)) / (1.0 + math.exp(-abs(l[t, e]))))
                        for e in live}
                total = sum(part.values())
                w = np.array([part.get(e, 0.0) / total for e in ids[t]])
        ws[t] = w * scale
    return ids, ws


def route_grouped_backward(dweights, logits, topk_ids, score="sigmoid", renormalize=True, scale=1.0, bias=None):
    """dlogits [T, E] and a bound on the terms that it is the sum of (numpy); the weight of an expert that the
    bias masks is the constant 0."""
    l, s = _clean(logits), scores(logits, score)
    T, E = l.shape
    dw = dweights.detach().cpu().double().numpy() * scale
    ids = topk_ids.detach().cpu().numpy()
    b = np.zeros(E) if bias is None else bias.detach().cpu().double().numpy()
    gone = np.isnan(b) | np.isneginf(b)
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        ok = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E and not (np.isneginf(l[t, ids[t, j]]) or gone[ids[t, j]])]
        if not ok:
            continue
        e = [ids[t, j] for j in ok]
        d = dw[t, ok]
        if renormalize:
            top = l[t, e].max()
            if score == "softmax":
                p, f = np.exp(l[t, e] - top), np.ones(len(e))
            else:
                p = np.exp(np.minimum(l[t, e], 0) - min(top, 0.0)) / (1 + np.exp(-np.abs(l[t, e])))
                f = 1.0 / (1.0 + np.exp(l[t, e]))
            p = p / p.sum()
            np.add.at(out[t], e, p * f * (d - (p * d).sum()))
            np.add.at(mag[t], e, p * f * (np.abs(d) + (p * np.abs(d)).sum()))
        elif score == "sigmoid":
            v = d * s[t, e] / (1.0 + np.exp(l[t, e]))
            np.add.at(out[t], e, v)
            np.add.at(mag[t], e, np.abs(v))
        else:
            g = np.zeros(E)
            np.add.at(g, e, d)
            ga = np.zeros(E)
            np.add.at(ga, e, np.abs(d))
            out[t] = s[t] * (g - (g * s[t]).sum())
            mag[t] = s[t] * (ga + (ga * s[t]).sum())
    return out, mag


# ------------------------------------------------------------------ finalize, gradient
def finalize_backward(dout, y, topk_weights, top_k, residual_out=None, rms_weight=None, eps=1e-6, dresidual_out=None):
    """dict of dy, dweights, dsum, drms (None where undefined) and of the magnitudes that bound their errors."""
    d = _f64(dout)
    T, H = d.shape
    g, mag, drms, drms_mag = d, d.abs(), None, None
    if rms_weight is not None:
        o, gamma = _f64(residual_out), _f64(rms_weight)
        r = (o.pow(2).mean(1, keepdim=True) + eps).rsqrt()
        drms, drms_mag = (d * o * r).sum(0), (d * o * r).abs().sum(0)
        v = d * gamma
        g = r * (v - o * r * r * (v * o).mean(1, keepdim=True))
        mag = r * (v.abs() + o.abs() * r * r * (v * o).abs().mean(1, keepdim=True))
    if dresidual_out is not None:
        g, mag = g + _f64(dresidual_out), mag + _f64(dresidual_out).abs()
    w = torch.ones((T, top_k), dtype=torch.float64) if topk_weights is None else _f64(topk_weights)
    out = {"dsum": g, "drms": drms, "dy": (w[:, :, None] * g[:, None]).reshape(T * top_k, H), "dweights": None}
    mags = {"dsum": mag, "drms": drms_mag, "dy": (w.abs()[:, :, None] * mag[:, None]).reshape(T * top_k, H)}
    if y is not None and topk_weights is not None:
        yy = _f64(y).view(T, top_k, H)
        out["dweights"] = (yy * g[:, None]).sum(2)
        mags["dweights"] = (yy.abs() * mag[:, None]).sum(2)
    return out, mags
