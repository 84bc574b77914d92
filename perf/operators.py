"""The router's operators and the gradients around them, as timed cases.

Five operators: the linear projection with bias, activation and residual in its epilogue
(``moe_linear``) and its gradients (``moe_linear_backward``), the router with scores, balance bias
and expert groups (``moe_route_grouped``) and its gradient (``moe_route_grouped_backward``), and the
gradient of the finalize (``moe_finalize_backward``).

``run`` makes the library's calls where ``own`` is set; otherwise it computes the same from
elementary torch operations in 32 bits (64 for the routing scores, whose order decides the chosen
experts), rounded once at the end.  ``exact`` restates each operator in 64 bits.
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


# ------------------------------------------------------------------ cases
def _linear(m, n, k, dtype="bf16", act="none", bias=False, residual=False, preact=False, out="same", **kw):
    return dict(kw, op="linear", m=m, n=n, k=k, dtype=dtype, act=act, bias=bias, residual=residual, preact=preact,
                out=out)


def _linear_backward(m, n, k, dtype="bf16", act="none", bias=False, dout="same", **kw):
    return dict(kw, op="linear_backward", m=m, n=n, k=k, dtype=dtype, act=act, bias=bias, dout=dout)


def _route(t, e, top_k, score, n_group=1, topk_group=1, group_top=1, bias=True, renorm=True, scale=1.0, logits="fp32",
           off=0, **kw):
    """off: how many experts each token may not use (logit -inf)."""
    return dict(kw, op="route", t=t, e=e, top_k=top_k, score=score, n_group=n_group, topk_group=topk_group,
                group_top=group_top, bias=bias, renorm=renorm, scale=scale, logits=logits, off=off)


def _route_backward(t, e, top_k, score, renorm=True, scale=1.0, logits="fp32", **kw):
    return dict(kw, op="route_backward", t=t, e=e, top_k=top_k, score=score, renorm=renorm, scale=scale, logits=logits)


def _finalize_backward(t, h, top_k, rms, dres, **kw):
    return dict(kw, op="finalize_backward", t=t, h=h, top_k=top_k, rms=rms, dres=dres)


def listed():
    return [
        # the gate of the DeepSeek-V3-like layer for one decoded token: 3.7 MB of weights, latency
        _linear(1, 256, 7168, out="fp32", name="gate_decode"),
        # the same gate over a prefill chunk, fp32 logits for the router
        _linear(4096, 256, 7168, out="fp32", name="gate_prefill"),
        # a dense down-projection of the Mixtral-like width with everything in the epilogue, saved for training
        _linear(8192, 4096, 14336, act="gelu", bias=True, residual=True, preact=True, name="dense_large"),
        # the gate's training step: fp32 gradients of the logits
        _linear_backward(4096, 256, 7168, dout="fp32", name="gate_backward"),
        # a dense up-projection with SiLU over a ragged batch, Llama-4-Scout-like sizes
        _linear_backward(2050, 8192, 5120, act="silu", bias=True, name="dense_backward"),
        # DeepSeek-V3-like routing (sigmoid, balance bias, 4 of 8 groups by their two best, top 8) of one token
        _route(1, 256, 8, "sigmoid", 8, 4, 2, scale=2.5, name="route_decode"),
        # and of a large prefill
        _route(16384, 256, 8, "sigmoid", 8, 4, 2, scale=2.5, name="route_prefill"),
        # Qwen3-MoE-like: plain softmax scores over 128 experts from bf16 logits, no groups
        _route(4095, 128, 8, "softmax", bias=False, logits="bf16", name="route_softmax"),
        # the gradient of the grouped sigmoid router over a training batch
        _route_backward(16384, 256, 8, "sigmoid", scale=2.5, name="route_backward"),
        # of a softmax router whose weights are not renormalised: every logit of the row has a gradient
        _route_backward(4095, 128, 8, "softmax", renorm=False, logits="bf16", name="route_softmax_backward"),
        # the finalize's gradient for a small batch, with residual stream and RMSNorm
        _finalize_backward(128, 7168, 4, True, True, name="finalize_backward_small"),
        # and for a training batch of the DeepSeek-V3-like layer
        _finalize_backward(4096, 7168, 8, True, True, name="finalize_backward_large"),
    ]


def _logu(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


_MAX_FLOPS = 2 * 8192 * 4096 * 14336


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "route", "route", "route_backward", "finalize_backward"])
    if op in ("linear", "linear_backward"):
        cap = _MAX_FLOPS if op == "linear" else 4 * 2050 * 8192 * 5120
        per = 2 if op == "linear" else 4
        while True:
            m, n, k = _logu(rng, 1, 8192), _logu(rng, 1, 14336), 8 * _logu(rng, 8, 1792)
            if per * m * n * k <= cap:
                break
        dtype, act = rng.choice(["bf16", "bf16", "fp16"]), rng.choice(["none", "none", "silu", "gelu", "gelu_tanh"])
        if op == "linear":
            return _linear(m, n, k, dtype, act, rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.3,
                           rng.choice(["same", "same", "fp32"]))
        return _linear_backward(m, n, k, dtype, act, rng.random() < 0.5, rng.choice(["same", "same", "fp32"]))
    if op == "finalize_backward":
        return _finalize_backward(_logu(rng, 1, 4096), 8 * _logu(rng, 16, 896), rng.randint(1, 8), rng.random() < 0.6,
                                  rng.random() < 0.5)
    t, logits = _logu(rng, 1, 16384), rng.choice(["fp32", "fp32", "bf16", "fp16"])
    score, renorm = rng.choice(["sigmoid", "softmax"]), rng.random() < 0.6
    if op == "route" and rng.random() < 0.5:
        n_group = rng.choice([2, 4, 8, 16])
        size = _logu(rng, 4, 256 // n_group)
        e, topk_group = n_group * size, rng.randint(1, n_group)
        top_k, group_top = rng.randint(1, min(16, size * topk_group)), rng.choice([1, 2])
    else:
        e = _logu(rng, 2, 256)
        n_group, topk_group, group_top, top_k = 1, 1, 1, rng.randint(1, min(16, e))
    scale = rng.choice([1.0, 2.5])
    if op == "route_backward":  # a single renormalised weight is 1 whatever its logit: no gradient to compare
        return _route_backward(t, e, max(2, top_k) if renorm else top_k, score, renorm, scale, logits)
    return _route(t, e, top_k, score, n_group, topk_group, group_top, rng.random() < 0.7, renorm, scale, logits,
                  off=rng.choice([0, 0, min(3, e - 1)]))


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    s = dict(case)
    op = case["op"]
    if op in ("linear", "linear_backward"):
        m, n, k, dt = case["m"], case["n"], case["k"], _T[case["dtype"]]
        s["x"] = normal(m, k, dtype=dt)
        s["w"] = normal(n, k, dtype=dt, std=1 / math.sqrt(k))
    if op == "linear":
        odt = dt if case["out"] == "same" else torch.float32
        s["bias_t"] = normal(n, dtype=dt, std=0.5) if case["bias"] else None
        s["res_t"] = normal(m, n, dtype=odt) if case["residual"] else None
        s["pre_t"] = torch.empty((m, n), dtype=dt, device=DEV) if case["preact"] else None
        s["out_t"] = torch.empty((m, n), dtype=odt, device=DEV)
    elif op == "linear_backward":
        s["dout_t"] = normal(m, n, dtype=dt if case["dout"] == "same" else torch.float32, std=0.1)
        s["pre_t"] = None if case["act"] == "none" else normal(m, n, dtype=dt)
        s["dx_t"], s["dw_t"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
        s["db_t"] = torch.empty(n, dtype=dt, device=DEV) if case["bias"] else None
    elif op in ("route", "route_backward"):
        t, e, top_k = case["t"], case["e"], case["top_k"]
        s["l"] = normal(t, e, dtype=_T[case["logits"]])
        # a balance bias after some training: steps of 1e-3 up and down
        steps = torch.randint(-100, 101, (e,), generator=g, device=DEV)
        if op == "route":
            s["b"] = (steps.float() * 1e-3) if case["bias"] else None
            if case["off"]:
                at = torch.rand((t, e), generator=g, device=DEV).argsort(1)[:, :case["off"]]
                s["l"].scatter_(1, at, float("-inf"))
            s["ids_t"] = torch.empty((t, top_k), dtype=torch.int32, device=DEV)
            s["w_t"] = torch.empty((t, top_k), dtype=torch.float32, device=DEV)
        else:
            s["ids"] = (s["l"].float() + steps.float() * 1e-3).topk(top_k, 1).indices.to(torch.int32)
            s["dw"] = normal(t, top_k)
            s["dl_t"] = torch.empty_like(s["l"])
    else:
        t, h, top_k = case["t"], case["h"], case["top_k"]
        bf = torch.bfloat16
        s["dout_t"], s["y"] = normal(t, h, dtype=bf, std=0.1), normal(t * top_k, h, dtype=bf)
        s["w"] = torch.rand((t, top_k), generator=g, device=DEV) + 0.05
        s["w"] /= s["w"].sum(1, keepdim=True)
        s["dres_t"] = normal(t, h, dtype=bf, std=0.1) if case["dres"] else None
        s["o"] = normal(t, h, dtype=bf, std=1.5) if case["rms"] else None
        s["gamma"] = (torch.rand(h, generator=g, device=DEV) + 0.5).to(bf) if case["rms"] else None
        s["dy_t"], s["dsum_t"] = torch.empty_like(s["y"]), torch.empty_like(s["dout_t"])
        s["dw_t"] = torch.empty((t, top_k), dtype=torch.float32, device=DEV)
        s["drms_t"] = torch.empty(h, dtype=torch.float32, device=DEV) if case["rms"] else None
    return s


# ------------------------------------------------------------------ the library's calls
def _workspace(s, size):
    """The workspace that a program keeps beside its buffers."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(size(), 16), dtype=torch.uint8, device=DEV)
    return s["ws"]


def _own(s):
    from mixture_experts_layer_tokens_gb300 import moe
    op = s["op"]
    if op == "linear":
        out = moe.moe_linear(s["x"], s["w"], bias=s["bias_t"], residual=s["res_t"], activation=s["act"],
                             out=s["out_t"], preact=s["pre_t"])
        return [out, s["pre_t"]]
    if op == "linear_backward":
        ws = _workspace(s, lambda: moe.linear_backward_workspace_size(s["m"], s["n"], s["k"]))
        return list(moe.moe_linear_backward(s["dout_t"], s["x"], s["w"], preact=s["pre_t"], activation=s["act"],
                                            dx=s["dx_t"], dw=s["dw_t"], dbias=s["db_t"], ws=ws))
    if op == "route":
        return list(moe.moe_route_grouped(s["l"], s["top_k"], bias=s["b"], score=s["score"], n_group=s["n_group"],
                                          topk_group=s["topk_group"], group_top=s["group_top"],
                                          renormalize=s["renorm"], scale=s["scale"], topk_ids=s["ids_t"],
                                          topk_weights=s["w_t"]))
    if op == "route_backward":
        return moe.moe_route_grouped_backward(s["dw"], s["l"], s["ids"], score=s["score"], renormalize=s["renorm"],
                                              scale=s["scale"], dlogits=s["dl_t"])
    ws = _workspace(s, lambda: moe.finalize_backward_workspace_size(s["t"], s["h"]))
    return list(moe.moe_finalize_backward(s["dout_t"], s["y"], s["w"], s["top_k"], residual_out=s["o"],
                                          rms_weight=s["gamma"], eps=1e-6, dresidual_out=s["dres_t"], dy=s["dy_t"],
                                          dweights=s["dw_t"], dsum=s["dsum_t"], drms=s["drms_t"], ws=ws))


# ------------------------------------------------------------------ plain forms
def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _dact(z, act):
    if act == "silu":
        q = 1 / (1 + torch.exp(-z))
        return q * (1 + z * (1 - q))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_linear(s):
    z = s["x"].float() @ s["w"].float().T
    if s["bias_t"] is not None:
        z = z + s["bias_t"].float()
    out = _act(z, s["act"])
    if s["res_t"] is not None:
        out = out + s["res_t"].float()
    return [out.to(s["out_t"].dtype), None if s["pre_t"] is None else z.to(s["x"].dtype)]


def _plain_linear_backward(s):
    dz = s["dout_t"].float()
    if s["pre_t"] is not None:
        dz = dz * _dact(s["pre_t"].float(), s["act"])
    dt = s["x"].dtype
    db = None if s["db_t"] is None else dz.sum(0).to(dt)
    return [(dz @ s["w"].float()).to(dt), (dz.T @ s["x"].float()).to(dt), db]


def _plain_route(s):
    l = s["l"].double()
    t, e, groups = s["t"], s["e"], s["n_group"]
    gone = torch.isinf(l)
    if s["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-l))
    else:
        p = torch.exp(l - l.max(1, keepdim=True).values)
        p = p / p.sum(1, keepdim=True)
    c = (p if s["b"] is None else p + s["b"].double()).masked_fill(gone, float("-inf"))
    if groups > 1:
        cg = c.view(t, groups, e // groups)
        best = cg.sort(2, descending=True).values[:, :, :s["group_top"]]
        some = torch.isfinite(best[:, :, :1]).squeeze(2)
        score = best.masked_fill(torch.isinf(best), 0).sum(2).masked_fill(~some, float("-inf"))
        kept = score.sort(dim=1, descending=True, stable=True).indices[:, :s["topk_group"]]
        keep = torch.zeros((t, groups), dtype=torch.bool, device=DEV).scatter_(1, kept, True)
        rank = torch.where(keep.repeat_interleave(e // groups, 1), 1, 0)
    else:
        rank = torch.ones((t, e), dtype=torch.int64, device=DEV)
    # kept groups first, then larger c, then larger logit, then the lower index
    at = l.sort(dim=1, descending=True, stable=True).indices
    at = at.gather(1, c.gather(1, at).sort(dim=1, descending=True, stable=True).indices)
    at = at.gather(1, rank.gather(1, at).sort(dim=1, descending=True, stable=True).indices)[:, :s["top_k"]]
    w = p.gather(1, at)
    if s["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / torch.where(total > 0, total, 1), 0)
    return [at.to(torch.int32), (w * s["scale"]).float()]


def _plain_route_backward(s):
    l, ids, dw = s["l"].float(), s["ids"].long(), s["dw"] * s["scale"]
    if s["score"] == "sigmoid":
        q = 1 / (1 + torch.exp(-l.gather(1, ids)))
        f = 1 / (1 + torch.exp(l.gather(1, ids)))  # 1 - q
        if s["renorm"]:
            p = q / q.sum(1, keepdim=True)
            d = p * f * (dw - (p * dw).sum(1, keepdim=True))
        else:
            d = q * f * dw
        out = torch.zeros_like(l).scatter_(1, ids, d)
    elif s["renorm"]:
        p = torch.exp(l.gather(1, ids) - l.gather(1, ids).max(1, keepdim=True).values)
        p = p / p.sum(1, keepdim=True)
        out = torch.zeros_like(l).scatter_(1, ids, p * (dw - (p * dw).sum(1, keepdim=True)))
    else:
        p = torch.exp(l - l.max(1, keepdim=True).values)
        p = p / p.sum(1, keepdim=True)
        up = torch.zeros_like(l).scatter_(1, ids, dw)
        out = p * (up - (p * up).sum(1, keepdim=True))
    return out.to(s["l"].dtype)


def _plain_finalize_backward(s):
    t, h, k = s["t"], s["h"], s["top_k"]
    d, drms = s["dout_t"].float(), None
    if s["gamma"] is not None:
        o, gamma = s["o"].float(), s["gamma"].float()
        r = 1 / torch.sqrt((o * o).mean(1, keepdim=True) + 1e-6)
        drms = (d * o * r).sum(0)
        v = d * gamma
        d = r * (v - o * r * r * (v * o).mean(1, keepdim=True))
    if s["dres_t"] is not None:
        d = d + s["dres_t"].float()
    y = s["y"].float().view(t, k, h)
    dy = (s["w"][:, :, None] * d[:, None, :]).to(torch.bfloat16).view(t * k, h)
    return [dy, (y * d[:, None, :]).sum(2), d.to(torch.bfloat16), drms]


_PLAIN = {"linear": _plain_linear, "linear_backward": _plain_linear_backward, "route": _plain_route,
          "route_backward": _plain_route_backward, "finalize_backward": _plain_finalize_backward}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = lambda v: None if v is None else v.double()  # noqa: E731
    if op == "linear":
        z = torch.einsum("mk,nk->mn", f64(s["x"]), f64(s["w"]))
        if case["bias"]:
            z += f64(s["bias_t"])
        out = _exact_act(z, case["act"])
        if case["residual"]:
            out = out + f64(s["res_t"])
        return [out, z if case["preact"] else None]
    if op == "linear_backward":
        dz = f64(s["dout_t"])
        if s["pre_t"] is not None:
            z = f64(s["pre_t"]).requires_grad_(True)
            dz, = torch.autograd.grad(_exact_act(z, case["act"]), z, dz)
        return [torch.einsum("mn,nk->mk", dz, f64(s["w"])), torch.einsum("mn,mk->nk", dz, f64(s["x"])),
                torch.einsum("mn->n", dz) if case["bias"] else None]
    if op == "route":
        return [None, _exact_route(s)]
    if op == "route_backward":
        l = f64(s["l"]).requires_grad_(True)
        p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
        w = p.gather(1, s["ids"].long())
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return torch.autograd.grad((w * case["scale"] * f64(s["dw"])).sum(), l)[0]
    return _exact_finalize_backward(s, case)


def _exact_act(z, act):
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":  # (1 + tanh u) / 2 is the logistic function of 2 u
        return z * torch.special.expit(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def _exact_route(s):
    """The weights alone: rounds of one choice each, the best of what is left."""
    l = s["l"].double()
    p = torch.special.expit(l) if s["score"] == "sigmoid" else torch.softmax(l, 1)
    c = p.clone() if s["b"] is None else p + s["b"].double()
    c[torch.isneginf(l)] = -1e300
    t, e, groups = s["t"], s["e"], s["n_group"]
    size, rows = e // groups, torch.arange(s["t"], device=DEV)
    if groups > 1:
        left, score = c.view(t, groups, size).clone(), None
        for i in range(s["group_top"]):
            top, at = left.max(2)
            # a group with fewer usable experts than group_top counts those that it has
            score = top if i == 0 else score + torch.where(top > -1e299, top, 0)
            left.scatter_(2, at[:, :, None], -1e300)
        out = torch.ones((t, groups), dtype=torch.bool, device=DEV)
        for _ in range(s["topk_group"]):
            at = score.argmax(1)
            out[rows, at] = False
            score[rows, at] = -float("inf")
        c = c.view(t, groups, size).masked_fill(out[:, :, None], -float("inf")).view(t, e)
    got = []
    for _ in range(s["top_k"]):
        at = c.argmax(1)
        got.append(p[rows, at])
        c[rows, at] = -float("inf")
    w = torch.stack(got, 1)
    if s["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    return w * s["scale"]


def _exact_finalize_backward(s, case):
    t, h, k = case["t"], case["h"], case["top_k"]
    v = s["dout_t"].double()
    drms = None
    if case["rms"]:
        o = s["o"].double().requires_grad_(True)
        gamma = s["gamma"].double().requires_grad_(True)
        n = o / torch.sqrt(torch.mean(o ** 2, 1, keepdim=True) + 1e-6) * gamma
        v, drms = torch.autograd.grad(n, (o, gamma), v)
    if case["dres"]:
        v = v + s["dres_t"].double()
    y, w = s["y"].view(t, k, h), s["w"].double()
    dy = torch.empty((t * k, h), dtype=torch.float64, device=DEV)
    dw = torch.empty((t, k), dtype=torch.float64, device=DEV)
    for j in range(k):
        dy.view(t, k, h)[:, j] = v * w[:, j, None]
        dw[:, j] = torch.einsum("th,th->t", v, y[:, j].double())
    return [dy, dw, v, drms]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    op = case["op"]
    if op in ("linear", "linear_backward"):
        m, n, k, z = case["m"], case["n"], case["k"], size[case["dtype"]]
        if op == "linear":
            o = z if case["out"] == "same" else 4
            moved = z * (m * k + n * k) + m * n * (o * (1 + case["residual"]) + z * case["preact"]) + z * n * case["bias"]
            return {"bytes": moved, "flops": 2 * m * n * k}
        d = z if case["dout"] == "same" else 4
        moved = 2 * z * (m * k + n * k) + m * n * (d + z * (case["act"] != "none")) + z * n * case["bias"]
        return {"bytes": moved, "flops": 4 * m * n * k}
    if op == "finalize_backward":
        t, h, k = case["t"], case["h"], case["top_k"]
        rows = 2 + 2 * k + case["dres"] + case["rms"]  # dout, dsum, y, dy
        return {"bytes": 2 * t * h * rows + 8 * t * k + 6 * h * case["rms"], "flops": t * h * (3 * k + 8 * case["rms"])}
    t, e, k, z = case["t"], case["e"], case["top_k"], size[case["logits"]]
    if op == "route":
        return {"bytes": t * e * z + 8 * t * k + 4 * e * case["bias"], "flops": 4 * t * e}
    dense = case["score"] == "softmax" and not case["renorm"]
    return {"bytes": t * e * z * (1 + dense) + t * k * (8 + (0 if dense else z)), "flops": t * (10 * k + 4 * e * dense)}
