"""The norm in front of the layer and what trains its experts, as timed cases.

Five operators: RMSNorm with the residual's addition and an 8-bit output (``moe_rmsnorm``), the
experts' products over ragged groups of rows (``moe_grouped_linear``) and their gradients
(``moe_grouped_linear_backward``), and the activation between an expert's two products
(``moe_activation``) with its gradient (``moe_activation_backward``).

``run`` makes the library's calls where ``own`` is set; otherwise it computes the same from
elementary torch operations in 32 bits, rounded once at the end (the groups' products as one batched
product over groups padded to the longest).  ``exact`` restates each operator in 64 bits.
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


# ------------------------------------------------------------------ cases
def _norm(t, h, residual=True, out=True, quant="none", **kw):
    """quant: "fp8" (a scale per 128 columns), "fp8_token" (one per token) or "none"; out: also in bf16."""
    return dict(kw, op="norm", t=t, h=h, residual=residual, out=out, quant=quant)


def _grouped(t, top_k, e, n, k, dtype="bf16", x_rows="sorted", out_rows="sorted", **kw):
    """t tokens choose top_k of e experts each: t * top_k rows over weights [e, n, k]."""
    return dict(kw, op="grouped", t=t, top_k=top_k, e=e, n=n, k=k, dtype=dtype, x_rows=x_rows, out_rows=out_rows)


def _grouped_backward(t, top_k, e, n, k, dtype="bf16", dout_rows="sorted", x_rows="sorted", dx_rows="sorted", dw="same",
                      **kw):
    return dict(kw, op="grouped_backward", t=t, top_k=top_k, e=e, n=n, k=k, dtype=dtype, dout_rows=dout_rows,
                x_rows=x_rows, dx_rows=dx_rows, dw=dw)


def _activation(s, i, act="silu", dtype="bf16", **kw):
    return dict(kw, op="activation", s=s, i=i, act=act, dtype=dtype)


def _activation_backward(s, i, act="silu", dtype="bf16", h=False, **kw):
    """h: the activation's output is made again in the same pass."""
    return dict(kw, op="activation_backward", s=s, i=i, act=act, dtype=dtype, h=h)


def listed():
    return [
        # the norm in front of the DeepSeek-V3-like fp8 layer for one decoded token: latency
        _norm(1, 7168, quant="fp8", name="norm_decode"),
        # the same over a large prefill: residual stream in and out, bf16 for the gate, 8 bits for the experts
        _norm(16384, 7168, quant="fp8", name="norm_prefill"),
        # one token through the gate and up weights of its 8 of 128 Qwen3-MoE-like experts
        _grouped(1, 8, 128, 1536, 2048, x_rows="token", name="grouped_decode"),
        # the down projection of a ragged training batch of the same layer, rows back in slot order
        _grouped(4095, 8, 128, 2048, 768, "fp16", out_rows="slot", name="grouped_down_ragged"),
        # DeepSeek-V3-shaped experts with about 128 rows each: the weights' bytes count
        _grouped(1024, 8, 64, 4096, 7168, x_rows="token", name="grouped_weights"),
        # the gate and up product of the Mixtral-like layer over a long prefill: the tensor cores count
        _grouped(8192, 2, 8, 28672, 4096, x_rows="token", name="grouped_prefill"),
        # gradients of the Qwen3-MoE-like gate and up product, weights' gradients in fp32 for the optimizer
        _grouped_backward(4095, 8, 128, 1536, 2048, x_rows="token", dx_rows="slot", dw="fp32",
                          name="grouped_backward_ragged"),
        # gradients of the Mixtral-like down projection
        _grouped_backward(4096, 2, 8, 4096, 14336, dout_rows="slot", name="grouped_backward_large"),
        # SiLU-and-mul of one decoded token's 8 rows
        _activation(8, 768, name="activation_decode"),
        # and of the Mixtral-like prefill
        _activation(16384, 14336, name="activation_prefill"),
        # the clamped SwiGLU's gradient for a small ragged batch
        _activation_backward(1023, 768, "swigluoai", "fp16", name="activation_backward_small"),
        # the gradient of a Mixtral-like training batch that makes the second product's rows again
        _activation_backward(8192, 14336, h=True, name="activation_backward_large"),
    ]


def _logu(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


_ROWS = ["sorted", "slot", "token"]
_ACTS = ["silu", "gelu", "gelu_tanh", "swigluoai", "silu_no_mul", "gelu_no_mul"]


def draw(rng):
    op = rng.choice(["norm", "grouped", "grouped", "grouped_backward", "grouped_backward", "activation",
                     "activation_backward"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "norm":
        quant = rng.choice(["none", "fp8", "fp8", "fp8_token"])
        return _norm(_logu(rng, 1, 16384), 8 * _logu(rng, 8, 896), rng.random() < 0.7,
                     quant == "none" or rng.random() < 0.6, quant)
    if op in ("activation", "activation_backward"):
        s, i, act = _logu(rng, 1, 16384), 8 * _logu(rng, 8, 1792), rng.choice(_ACTS)
        if op == "activation":
            return _activation(s, i, act, dtype)
        return _activation_backward(min(s, 8192), i, act, dtype, rng.random() < 0.5)
    cap = 2 * 16384 * 28672 * 4096 if op == "grouped" else 4 * 8192 * 4096 * 14336
    while True:
        t, e = _logu(rng, 1, 8192), _logu(rng, 2, 128)
        top_k, n, k = rng.randint(1, min(8, e)), 8 * _logu(rng, 4, 1792), 8 * _logu(rng, 8, 1792)
        if (2 if op == "grouped" else 4) * t * top_k * n * k <= cap and e * n * k <= 1000000000 and t * top_k <= 32768:
            break
    if op == "grouped":
        return _grouped(t, top_k, e, n, k, dtype, rng.choice(_ROWS), rng.choice(_ROWS[:2]))
    return _grouped_backward(t, top_k, e, n, k, dtype, rng.choice(_ROWS), rng.choice(_ROWS), rng.choice(_ROWS[:2]),
                             rng.choice(["same", "same", "fp32"]))


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    s = dict(case)
    op, bf = case["op"], torch.bfloat16
    if op == "norm":
        t, h = case["t"], case["h"]
        s["x"], s["gamma"] = normal(t, h, dtype=bf), (torch.rand(h, generator=g, device=DEV) + 0.5).to(bf)
        s["res"] = normal(t, h, dtype=bf, std=2.0) if case["residual"] else None
        s["res_t"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["out_t"] = torch.empty_like(s["x"]) if case["out"] else None
        if case["quant"] != "none":
            s["q_t"] = torch.empty((t, h), dtype=torch.uint8, device=DEV)
            groups = (t, -(-h // 128)) if case["quant"] == "fp8" else (t,)
            s["scale_t"] = torch.empty(groups, dtype=torch.float32, device=DEV)
        return s
    dt = _T[case["dtype"]]
    if op in ("activation", "activation_backward"):
        rows, i = case["s"], case["i"]
        # sums of a first product after some training: a few of them beyond the clamps
        s["gu"] = normal(rows, i if case["act"].endswith("no_mul") else 2 * i, dtype=dt, std=3.0)
        if op == "activation":
            s["h_t"] = torch.empty((rows, i), dtype=dt, device=DEV)
        else:
            s["dh"], s["dgu_t"] = normal(rows, i, dtype=dt, std=0.1), torch.empty_like(s["gu"])
            s["h_t"] = torch.empty((rows, i), dtype=dt, device=DEV) if case["h"] else None
        return s
    t, top_k, e, n, k = case["t"], case["top_k"], case["e"], case["n"], case["k"]
    rows = t * top_k
    # a router whose experts are not equally liked
    likes = normal(t, e) + normal(e, std=0.5)
    ids = likes.topk(top_k, 1).indices.reshape(-1)
    s["sorted_slot"] = ids.sort(stable=True).indices.to(torch.int32)
    counts = torch.bincount(ids, minlength=e)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["most"] = int(counts.max())
    s["x"] = normal(t if case["x_rows"] == "token" else rows, k, dtype=dt)
    s["w"] = torch.empty((e, n, k), dtype=dt, device=DEV).normal_(0, 1 / math.sqrt(k), generator=g)
    if op == "grouped":
        s["out_t"] = torch.empty((rows, n), dtype=dt, device=DEV)
    else:
        s["dout"] = normal(t if case["dout_rows"] == "token" else rows, n, dtype=dt, std=0.1)
        s["dx_t"] = torch.empty((rows, k), dtype=dt, device=DEV)
        s["dw_t"] = torch.empty((e, n, k), dtype=dt if case["dw"] == "same" else torch.float32, device=DEV)
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
    if op == "norm":
        quant = s["quant"] != "none"
        out, res, q, scale = moe.moe_rmsnorm(
            s["x"], s["gamma"], residual=s["res"], eps=1e-6, quant=s["quant"] if quant else None, out=s["out_t"],
            residual_out=s["res_t"], q=s.get("q_t"), q_scale=s.get("scale_t"), need_out=s["out"])
        return [out, res, q.view(torch.float8_e4m3fn) if quant else None, scale]
    if op == "activation":
        return moe.moe_activation(s["gu"], s["act"], h=s["h_t"])
    if op == "activation_backward":
        return list(moe.moe_activation_backward(s["dh"], s["gu"], s["act"], dgu=s["dgu_t"], h=s["h_t"]))
    rows, n, k, e = s["t"] * s["top_k"], s["n"], s["k"], s["e"]
    if op == "grouped":
        ws = _workspace(s, lambda: moe.grouped_linear_workspace_size(rows, e, n, k, x_rows=s["x_rows"]))
        return moe.moe_grouped_linear(s["x"], s["w"], s["offsets"], s["sorted_slot"], s["top_k"], x_rows=s["x_rows"],
                                      out_rows=s["out_rows"], out=s["out_t"], ws=ws)
    ws = _workspace(s, lambda: moe.grouped_linear_backward_workspace_size(rows, e, n, k, dout_rows=s["dout_rows"],
                                                                          x_rows=s["x_rows"]))
    return list(moe.moe_grouped_linear_backward(s["dout"], s["x"], s["w"], s["offsets"], s["sorted_slot"], s["top_k"],
                                                dout_rows=s["dout_rows"], x_rows=s["x_rows"], dx_rows=s["dx_rows"],
                                                dx=s["dx_t"], dw=s["dw_t"], ws=ws))


# ------------------------------------------------------------------ plain forms
def _plain_norm(s):
    v = s["x"].float()
    if s["res"] is not None:
        v = v + s["res"].float()
    n = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * s["gamma"].float()
    q = scale = None
    if s["quant"] != "none":
        t, h = n.shape
        size = 128 if s["quant"] == "fp8" else h
        # (a last group that is shorter than the others counts as filled up with zeros)
        groups = torch.nn.functional.pad(n, (0, -h % size)).view(t, -1, size)
        scale = groups.abs().amax(2).clamp(min=1e-10) / 448
        q = (groups / scale[:, :, None]).view(t, -1)[:, :h].to(torch.float8_e4m3fn)
        scale = scale if s["quant"] == "fp8" else scale.view(t)
    return [n.to(torch.bfloat16) if s["out"] else None, None if s["res"] is None else v.to(torch.bfloat16), q, scale]


def _gate(g, act):
    if act.startswith("silu"):
        return g / (1 + torch.exp(-g))
    if act.startswith("gelu_tanh"):
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
    if act.startswith("gelu"):
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    g = g.clamp(max=7)
    return g / (1 + torch.exp(-1.702 * g))


def _slope(g, act):
    if act.startswith("silu"):
        q = 1 / (1 + torch.exp(-g))
        return q * (1 + g * (1 - q))
    if act.startswith("gelu_tanh"):
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (g + 0.044715 * g * g * g))
        return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * a * (1 + 3 * 0.044715 * g * g)
    if act.startswith("gelu"):
        return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    c = g.clamp(max=7)
    q = 1 / (1 + torch.exp(-1.702 * c))
    return torch.where(g <= 7, q * (1 + 1.702 * c * (1 - q)), 0)


def _parts(s):
    """Gate and up columns in 32 bits; the up columns as what multiplies, and where they have a slope."""
    v, act = s["gu"].float(), s["act"]
    if act.endswith("no_mul"):
        return v, None, None
    g, u = v[:, :s["i"]], v[:, s["i"]:]
    if act == "swigluoai":
        return g, u.clamp(-7, 7) + 1, (u >= -7) & (u <= 7)
    return g, u, None


def _plain_activation(s):
    g, u, _ = _parts(s)
    h = _gate(g, s["act"])
    return (h if u is None else h * u).to(s["gu"].dtype)


def _plain_activation_backward(s):
    g, u, inside = _parts(s)
    d, a, dt = s["dh"].float(), _gate(g, s["act"]), s["gu"].dtype
    dg = d * _slope(g, s["act"])
    if u is None:
        return [dg.to(dt), a.to(dt) if s["h"] else None]
    du = d * a
    if inside is not None:
        du = torch.where(inside, du, 0)
    return [torch.cat([(dg * u).to(dt), du.to(dt)], 1), (a * u).to(dt) if s["h"] else None]


def _places(s):
    """Of each sorted row: its expert, its place in the expert's group, its slot."""
    rows = torch.arange(s["t"] * s["top_k"], device=DEV)
    expert = torch.searchsorted(s["offsets"][1:].long(), rows, right=True)
    return expert, rows - s["offsets"].long()[expert], s["sorted_slot"].long()


def _padded(s, v, order, expert, place, slot):
    """Rows in the given order -> [experts, rows of the longest group, columns] in 32 bits."""
    v = v.float()
    v = v if order == "sorted" else v[slot] if order == "slot" else v[slot // s["top_k"]]
    out = torch.zeros((s["e"], s["most"], v.shape[1]), device=DEV)
    out[expert, place] = v
    return out


def _unpadded(v, order, expert, place, slot, dtype):
    v = v[expert, place].to(dtype)
    return v if order == "sorted" else torch.empty_like(v).index_copy_(0, slot, v)


def _plain_grouped(s):
    at = _places(s)
    z = torch.bmm(_padded(s, s["x"], s["x_rows"], *at), s["w"].float().transpose(1, 2))
    return _unpadded(z, s["out_rows"], *at, s["x"].dtype)


def _plain_grouped_backward(s):
    at = _places(s)
    d = _padded(s, s["dout"], s["dout_rows"], *at)
    dx = _unpadded(torch.bmm(d, s["w"].float()), s["dx_rows"], *at, s["x"].dtype)
    dw = torch.bmm(d.transpose(1, 2), _padded(s, s["x"], s["x_rows"], *at))
    return [dx, dw.to(s["dw_t"].dtype)]


_PLAIN = {"norm": _plain_norm, "activation": _plain_activation, "activation_backward": _plain_activation_backward,
          "grouped": _plain_grouped, "grouped_backward": _plain_grouped_backward}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "activation":
        return _exact_activation(s["gu"].double(), case["act"])
    if case["op"] == "activation_backward":
        v = s["gu"].double().requires_grad_(True)
        h = _exact_activation(v, case["act"])
        dgu, = torch.autograd.grad(h, v, s["dh"].double())
        return [dgu, h.detach() if case["h"] else None]
    rows, ends = case["t"] * case["top_k"], s["offsets"].tolist()
    slot = s["sorted_slot"].long()
    at = {"sorted": torch.arange(rows, device=DEV), "slot": slot, "token": slot // case["top_k"]}
    forward = case["op"] == "grouped"
    first = torch.zeros((rows, case["n"] if forward else case["k"]), dtype=torch.float64, device=DEV)
    dw = None if forward else torch.zeros((case["e"], case["n"], case["k"]), dtype=torch.float64, device=DEV)
    for i in range(case["e"]):
        a, b = ends[i], ends[i + 1]
        x, w = s["x"][at[case["x_rows"]][a:b]].double(), s["w"][i].double()
        if forward:
            first[at[case["out_rows"]][a:b]] = torch.einsum("pk,nk->pn", x, w)
        else:
            d = s["dout"][at[case["dout_rows"]][a:b]].double()
            first[at[case["dx_rows"]][a:b]] = torch.einsum("pn,nk->pk", d, w)
            dw[i] = torch.einsum("pn,pk->nk", d, x)
    return first if forward else [first, dw]


def _exact_norm(s):
    v = s["x"].double() if s["res"] is None else s["x"].double() + s["res"].double()
    n = v * torch.rsqrt(v.pow(2).sum(1, keepdim=True) / s["h"] + 1e-6) * s["gamma"].double()
    q = scale = None
    if s["quant"] == "fp8":
        parts = [p / p.abs().max(1, keepdim=True).values * 448 for p in n.split(128, 1)]
        q = torch.cat(parts, 1)
        scale = torch.stack([p.abs().max(1).values / 448 for p in n.split(128, 1)], 1)
    elif s["quant"] == "fp8_token":
        scale = n.abs().max(1).values / 448
        q = n / scale[:, None]
    return [n if s["out"] else None, None if s["res"] is None else v, q, scale]


def _exact_activation(v, act):
    if act.endswith("no_mul"):
        g, u = v, 1
    else:
        g, u = v.chunk(2, 1)
    if act == "swigluoai":
        g, u = g.clamp(max=7), u.clamp(-7, 7)
        return (u + 1) * g * torch.special.expit(1.702 * g)
    if act.startswith("silu"):
        return g * torch.special.expit(g) * u
    if act == "gelu_tanh":  # (1 + tanh u) / 2 is the logistic function of 2 u
        return g * torch.special.expit(math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)) * u
    return g * torch.special.ndtr(g) * u


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    op = case["op"]
    if op == "norm":
        t, h = case["t"], case["h"]
        groups = 0 if case["quant"] == "none" else -(-h // 128) if case["quant"] == "fp8" else 1
        moved = 2 * t * h * (1 + 2 * case["residual"] + case["out"]) + 2 * h + t * (h + 4 * groups) * (groups > 0)
        return {"bytes": moved, "flops": t * h * (5 + 2 * (groups > 0))}
    z = size[case["dtype"]]
    if op in ("activation", "activation_backward"):
        s, i, two = case["s"], case["i"], 1 if case["act"].endswith("no_mul") else 2
        if op == "activation":
            return {"bytes": z * s * i * (two + 1), "flops": 6 * s * i}
        return {"bytes": z * s * i * (2 * two + 1 + case["h"]), "flops": 12 * s * i}
    t, top_k, e, n, k = case["t"], case["top_k"], case["e"], case["n"], case["k"]
    rows = t * top_k
    used = e * (1 - (1 - top_k / e) ** t)  # experts that some token chose, on the average of an even router
    x = (t if case["x_rows"] == "token" else rows) * k
    index = 4 * rows + 4 * (e + 1)
    if op == "grouped":
        return {"bytes": int(z * (x + rows * n + used * n * k)) + index, "flops": 2 * rows * n * k}
    d = (t if case["dout_rows"] == "token" else rows) * n
    out = z if case["dw"] == "same" else 4
    return {"bytes": int(z * (x + d + rows * k + used * n * k)) + out * e * n * k + index, "flops": 4 * rows * n * k}
