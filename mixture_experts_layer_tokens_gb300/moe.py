"""Thin ctypes binding of the fused-MoE C ABI (``include/moe.h``).

Every function here checks tensor dtypes/devices, passes ``data_ptr()`` values
and the current torch CUDA stream to the C entry point of the same name, and
turns a non-OK status into :class:`MoeError`.  All arithmetic happens in the
CUDA library; there is no fallback path.  PyTorch only provides device memory
and streams.
"""
from __future__ import annotations

import ctypes
import functools
import os
from operator import index
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, MOE_ERR_TIMEOUT = range(6)
MOE_DT_BF16, MOE_DT_FP8_E4M3, MOE_DT_NVFP4, MOE_DT_FP32, MOE_DT_FP16 = range(5)
MOE_SCORING_SOFTMAX_RENORM, MOE_SCORING_SIGMOID = 0, 1
MOE_BLOCK_M = 128
# moe_activation_t, by the names of the "Fused Experts Kernels" table
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "swigluoai": 3, "silu_no_mul": 4, "gelu_no_mul": 5}

# moe_linear_activation_t and moe_score_t, by name
LINEAR_ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3}
SCORES = {"softmax": 0, "sigmoid": 1}

# moe_rows_t, by name: the order of a tensor's rows in the grouped products
ROWS = {"sorted": 0, "slot": 1, "token": 2}

# (name, argtypes, restype) of every exported entry point
_P, _I, _F, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


class QuantConfig(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int), ("act_group", ctypes.c_int), ("weight", ctypes.c_int),
                ("w_block_n", ctypes.c_int), ("w_block_k", ctypes.c_int)]


QC_BF16 = QuantConfig(MOE_DT_BF16, 0, MOE_DT_BF16, 0, 0)
QC_FP8 = QuantConfig(MOE_DT_FP8_E4M3, 128, MOE_DT_FP8_E4M3, 128, 128)
MOE_GROUP_TOKEN, MOE_GROUP_TENSOR = -1, -2
# quant names: "bf16"; "fp8" (G(128) activations); "fp8_token" ("A"); "fp8_tensor" ("T")
QUANT_CONFIGS = {
    "bf16": QC_BF16,
    "fp8": QC_FP8,
    "fp8_token": QuantConfig(MOE_DT_FP8_E4M3, MOE_GROUP_TOKEN, MOE_DT_FP8_E4M3, 128, 128),
    "fp8_tensor": QuantConfig(MOE_DT_FP8_E4M3, MOE_GROUP_TENSOR, MOE_DT_FP8_E4M3, 128, 128),
}


def _qc(quant: str) -> QuantConfig:
    if quant not in QUANT_CONFIGS:
        raise ValueError(f"unknown quantisation {quant!r}")
    return QUANT_CONFIGS[quant]


def scale_shape(quant: str, T: int, H: int):
    """Shape of a1q_scale for each fp8 format (None for bf16)."""
    return {"bf16": None, "fp8": (T, H // 128), "fp8_token": (T,), "fp8_tensor": (1,)}[quant]
_QCP = ctypes.POINTER(QuantConfig)


class ExpertsProblem(ctypes.Structure):
    """moe_experts_problem: one expert problem of a moe_experts_multi call."""
    _fields_ = [("a1q", ctypes.c_void_p), ("a1q_scale", ctypes.c_void_p), ("w13", ctypes.c_void_p),
                ("w13_scale", ctypes.c_void_p), ("w2", ctypes.c_void_p), ("w2_scale", ctypes.c_void_p),
                ("expert_offsets", ctypes.c_void_p), ("sorted_slot", ctypes.c_void_p), ("tile_map", ctypes.c_void_p),
                ("num_tiles", ctypes.c_void_p), ("T", ctypes.c_int), ("I", ctypes.c_int), ("E", ctypes.c_int),
                ("top_k", ctypes.c_int), ("fused_expert_output", ctypes.c_void_p)]


_EPP = ctypes.POINTER(ExpertsProblem)


class RouteConfig(ctypes.Structure):
    """moe_route_config: how moe_route_grouped scores, groups and weighs the experts."""
    _fields_ = [("score", ctypes.c_int), ("n_group", ctypes.c_int), ("topk_group", ctypes.c_int),
                ("group_top", ctypes.c_int), ("renormalize", ctypes.c_int), ("scale", ctypes.c_float)]


_RCP = ctypes.POINTER(RouteConfig)

SIGNATURES = {
    "moe_route": ([_P, _I, _I, _I, _I, _P, _P, _P], _I),
    "moe_align": ([_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _Z, _P], _I),
    "moe_align_workspace_size": ([_I, _I, _I], _Z),
    "moe_align_noalloc": ([_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P], _I),
    "moe_tile_map_capacity": ([_I, _I, _I], _I),
    "moe_prepare": ([_P, _P, _P, _I, _I, _I, _I, _QCP, _P, _P, _P], _I),
    "moe_experts": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _QCP, _P, _P, _Z, _P], _I),
    "moe_experts_act": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _QCP, _I, _P, _P, _Z, _P], _I),
    "moe_experts_multi": ([_EPP, _I, _I, _QCP, _I, _P, _Z, _P], _I),
    "moe_workspace_size_multi": ([_EPP, _I, _I, _QCP], _Z),
    "moe_workspace_size": ([_I, _I, _I, _I, _I, _QCP], _Z),
    "moe_workspace_intermediate": ([_I, _I, _I, _I, _I, _QCP, _P, _P, _P], _I),
    "moe_workspace_intermediate_nvfp4": ([_I, _I, _I, _I, _I, _P, _P, _P], _I),
    "moe_prepare_nvfp4": ([_P, _P, _I, _I, _I, _I, _P, _P, _P, _P], _I),
    "moe_experts_nvfp4": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P,
                           _Z, _P], _I),
    "moe_workspace_size_nvfp4": ([_I, _I, _I, _I, _I], _Z),
    "moe_layer_fused": ([_P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _P, _Z, _P], _I),
    "moe_layer_fused_workspace_size": ([_I, _I, _I, _I, _I, _I], _Z),
    "moe_finalize": ([_P, _P, _P, _P, _P, _P, _P, _F, _I, _I, _I, _I, _I, _P, _F, _P, _P], _I),
    "moe_prepare_batched_workspace_size": ([_I, _I, _QCP], _Z),
    "moe_prepare_batched": ([_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _QCP, _P, _P, _P, _P, _Z, _P], _I),
    "moe_workspace_size_batched": ([_I, _I, _I, _I, _QCP], _Z),
    "moe_experts_batched": ([_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _QCP, _I, _P, _P, _Z, _P], _I),
    "moe_finalize_batched": ([_P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _F, _I, _I, _I, _I, _I, _P, _F, _P, _P], _I),
    "moe_linear": ([_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P], _I),
    "moe_linear_backward": ([_P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _Z, _P], _I),
    "moe_linear_backward_workspace_size": ([_I, _I, _I], _Z),
    "moe_route_grouped": ([_P, _I, _P, _I, _I, _I, _RCP, _P, _P, _P], _I),
    "moe_route_grouped_backward": ([_P, _P, _I, _P, _P, _I, _I, _I, _RCP, _P, _P], _I),
    "moe_finalize_backward": ([_P, _P, _P, _P, _F, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _Z, _P], _I),
    "moe_finalize_backward_workspace_size": ([_I, _I], _Z),
    "moe_rmsnorm": ([_P, _P, _P, _F, _I, _I, _QCP, _P, _P, _P, _P, _P], _I),
    "moe_grouped_linear": ([_P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _I, _P, _Z, _P], _I),
    "moe_grouped_linear_workspace_size": ([_I, _I, _I, _I, _I], _Z),
    "moe_grouped_linear_backward": ([_P, _I, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _I, _P, _I, _I, _P, _Z,
                                     _P], _I),
    "moe_grouped_linear_backward_workspace_size": ([_I, _I, _I, _I, _I, _I], _Z),
    "moe_activation": ([_P, _I, _I, _I, _I, _P, _P], _I),
    "moe_activation_backward": ([_P, _P, _I, _I, _I, _I, _P, _P, _P], _I),
    "moe_device_status": ([_I], _I),
    "moe_selftest_wait_timeout": ([ctypes.c_uint64, _P], _I),
    "moe_selftest_row_division": ([ctypes.c_longlong, ctypes.c_uint32, _P, _P], _I),
    "moe_status_string": ([_I], ctypes.c_char_p),
}

_lib_handle = None


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} (status {status})")


def lib():
    """Load libmoe.so (built by ``mixture_experts_layer_tokens_gb300.build``).

    Raises if the library is missing: there is no CPU or PyTorch fallback."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m mixture_experts_layer_tokens_gb300.build` (nvcc, sm_103a)")
        h = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            f = getattr(h, name)
            f.argtypes = args
            f.restype = res
        _lib_handle = h
    return _lib_handle


def status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoeError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t: Optional[torch.Tensor], dtype, name: str, cuda: bool = True):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if cuda and not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")


# ------------------------------------------------------------------ entry points
def moe_route(logits: torch.Tensor, top_k: int, scoring: int = MOE_SCORING_SOFTMAX_RENORM,
              topk_ids: Optional[torch.Tensor] = None, topk_weights: Optional[torch.Tensor] = None,
              stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    _need(logits, torch.float32, "logits")
    T, E = logits.shape
    if topk_ids is None:
        topk_ids = torch.empty((T, top_k), dtype=torch.int32, device=logits.device)
    if topk_weights is None:
        topk_weights = torch.empty((T, top_k), dtype=torch.float32, device=logits.device)
    _need(topk_ids, torch.int32, "topk_ids")
    _need(topk_weights, torch.float32, "topk_weights")
    _check("moe_route", lib().moe_route(_ptr(logits), T, E, top_k, scoring, _ptr(topk_ids), _ptr(topk_weights),
                                        _stream(stream)))
    return topk_ids, topk_weights


def align_workspace_size(T: int, top_k: int, E: int) -> int:
    return int(lib().moe_align_workspace_size(T, top_k, E))


def tile_map_capacity(num_slots: int, E: int, block_m: int = MOE_BLOCK_M) -> int:
    return int(lib().moe_tile_map_capacity(num_slots, E, block_m))


class Alignment:
    """Device buffers written by moe_align."""

    def __init__(self, T: int, top_k: int, E: int, device, block_m: int = MOE_BLOCK_M):
        S = T * top_k
        self.T, self.top_k, self.E, self.block_m = T, top_k, E, block_m
        self.expert_offsets = torch.empty(E + 1, dtype=torch.int32, device=device)
        self.sorted_slot = torch.empty(max(S, 1), dtype=torch.int32, device=device)
        self.inv_slot = torch.empty(max(S, 1), dtype=torch.int32, device=device)
        self.tile_map = torch.empty((max(tile_map_capacity(S, E, block_m), 1), 2), dtype=torch.int32, device=device)
        self.num_tiles = torch.zeros(1, dtype=torch.int32, device=device)
        self.ws = torch.empty(max(align_workspace_size(T, top_k, E), 16), dtype=torch.uint8, device=device)


def moe_align(topk_ids: torch.Tensor, E: int, block_m: int = MOE_BLOCK_M, out: Optional[Alignment] = None,
              stream=None) -> Alignment:
    _need(topk_ids, torch.int32, "topk_ids")
    T, k = topk_ids.shape
    al = out if out is not None else Alignment(T, k, E, topk_ids.device, block_m)
    _check("moe_align", lib().moe_align(_ptr(topk_ids), T, k, E, block_m, _ptr(al.expert_offsets),
                                        _ptr(al.sorted_slot), _ptr(al.inv_slot), _ptr(al.tile_map),
                                        _ptr(al.num_tiles), _ptr(al.ws), al.ws.numel(), _stream(stream)))
    return al


ALIGN_NOALLOC_SCRATCH_BYTES = 256 * 1024


def moe_align_noalloc(topk_ids: torch.Tensor, E: int, out: Alignment, block_m: int = MOE_BLOCK_M,
                      stream=None) -> Alignment:
    """moe_align for callers that cannot allocate device memory at call time:
    the library's own fixed scratch array stands in for the workspace (out.ws
    is not used).  Calls that overlap on the GPU race on that array."""
    _need(topk_ids, torch.int32, "topk_ids")
    T, k = topk_ids.shape
    _check("moe_align_noalloc", lib().moe_align_noalloc(
        _ptr(topk_ids), T, k, E, block_m, _ptr(out.expert_offsets), _ptr(out.sorted_slot), _ptr(out.inv_slot),
        _ptr(out.tile_map), _ptr(out.num_tiles), _stream(stream)))
    return out


def moe_prepare(a1: torch.Tensor, topk_weights: Optional[torch.Tensor], top_k: int,
                apply_router_weight_on_input: bool, quant: str, a1q: Optional[torch.Tensor] = None,
                a1q_scale: Optional[torch.Tensor] = None, topk_ids: Optional[torch.Tensor] = None,
                stream=None):
    """quant: "bf16" (no quantisation), "fp8" (E4M3, per-token 128-group scales
    [T, H/128]), "fp8_token" (one scale per token [T]) or "fp8_tensor" (one scale
    [1]).  Passing ``a1q=a1`` with bf16 and no weight is the passthrough (nothing runs)."""
    _need(a1, torch.bfloat16, "a1")
    _need(topk_weights, torch.float32, "topk_weights")
    T, H = a1.shape
    qc = _qc(quant)
    fp8 = quant != "bf16"
    if a1q is None:
        a1q = torch.empty((T, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=a1.device)
    if fp8 and a1q_scale is None:
        a1q_scale = torch.empty(scale_shape(quant, T, H), dtype=torch.float32, device=a1.device)
    _need(a1q, torch.uint8 if fp8 else torch.bfloat16, "a1q")
    _need(a1q_scale, torch.float32, "a1q_scale")
    _check("moe_prepare", lib().moe_prepare(_ptr(a1), _ptr(topk_weights), _ptr(topk_ids), T, H, top_k,
                                            int(bool(apply_router_weight_on_input)), ctypes.byref(qc), _ptr(a1q),
                                            _ptr(a1q_scale), _stream(stream)))
    return a1q, a1q_scale


def workspace_size(T: int, H: int, I: int, E: int, top_k: int, quant: str) -> int:
    return int(lib().moe_workspace_size(T, H, I, E, top_k, ctypes.byref(_qc(quant))))


def experts_intermediate(ws: torch.Tensor, T: int, H: int, I: int, E: int, top_k: int, quant: str):
    """Views into a moe_experts workspace of the intermediate h that the call left
    there (``moe_workspace_intermediate``): h [S, I] (bf16, or uint8 E4M3 codes for the
    fp8 formats) and its fp32 scales -- G(128): [I/128, S] (transposed, row stride
    s_pad), "A"/"T": [S] -- or None for bf16.  S = T * top_k rows in expert order."""
    off, soff, stride = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_int()
    _check("moe_workspace_intermediate", lib().moe_workspace_intermediate(
        T, H, I, E, top_k, ctypes.byref(_qc(quant)), ctypes.byref(off), ctypes.byref(soff), ctypes.byref(stride)))
    S = T * top_k
    fp8 = quant != "bf16"
    esz = 1 if fp8 else 2
    h = ws[off.value:off.value + S * I * esz]
    h = h.view(S, I) if fp8 else h.view(torch.bfloat16).view(S, I)
    if not fp8:
        return h, None
    if quant == "fp8":
        n = (I // 128) * stride.value
        sc = ws[soff.value:soff.value + 4 * n].view(torch.float32).view(I // 128, stride.value)[:, :S]
    else:
        sc = ws[soff.value:soff.value + 4 * S].view(torch.float32)
    return h, sc


def experts_intermediate_nvfp4(ws: torch.Tensor, T: int, H: int, I: int, E: int, top_k: int):
    """Views into a moe_experts_nvfp4 workspace (``moe_workspace_intermediate_nvfp4``):
    the bf16 h [S, I] of the first GEMM and its NVFP4 codes [S, I/2] and scale codes
    [S, I/16] that the second GEMM read."""
    hb, hq, hsf = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check("moe_workspace_intermediate_nvfp4", lib().moe_workspace_intermediate_nvfp4(
        T, H, I, E, top_k, ctypes.byref(hb), ctypes.byref(hq), ctypes.byref(hsf)))
    S = T * top_k
    return (ws[hb.value:hb.value + S * I * 2].view(torch.bfloat16).view(S, I),
            ws[hq.value:hq.value + S * I // 2].view(S, I // 2),
            ws[hsf.value:hsf.value + S * I // 16].view(S, I // 16))


def moe_experts(a1q: torch.Tensor, a1q_scale: Optional[torch.Tensor], w13: torch.Tensor,
                w13_scale: Optional[torch.Tensor], w2: torch.Tensor, w2_scale: Optional[torch.Tensor],
                al: Alignment, quant: str, out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                identity: bool = False, stream=None, activation: str = "silu") -> torch.Tensor:
    """Grouped expert MLPs (``moe_experts_act``; SiLU-and-mul by default, see
    ``ACTIVATIONS``; the *_no_mul activations take w13 [E, I, H]).
    ``identity=True`` (E == 1, top_k == 1) passes a NULL sorted_slot: rows are
    the tokens in order."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    fp8 = quant != "bf16"
    _need(a1q, torch.uint8 if fp8 else torch.bfloat16, "a1q")
    _need(w13, torch.uint8 if fp8 else torch.bfloat16, "w13")
    _need(w2, torch.uint8 if fp8 else torch.bfloat16, "w2")
    for t, n in ((a1q_scale, "a1q_scale"), (w13_scale, "w13_scale"), (w2_scale, "w2_scale")):
        _need(t, torch.float32, n)
    T, H = a1q.shape
    E, rows13, _ = w13.shape
    I = rows13 if activation.endswith("_no_mul") else rows13 // 2
    k = al.top_k
    if out is None:
        out = torch.empty((T * k, H), dtype=torch.bfloat16, device=a1q.device)
    _need(out, torch.bfloat16, "fused_expert_output")
    if ws is None:
        ws = torch.empty(max(workspace_size(T, H, I, E, k, quant), 16), dtype=torch.uint8, device=a1q.device)
    qc = _qc(quant)
    _check("moe_experts_act", lib().moe_experts_act(
        _ptr(a1q), _ptr(a1q_scale), _ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), _ptr(al.expert_offsets),
        None if identity else _ptr(al.sorted_slot), _ptr(al.tile_map), _ptr(al.num_tiles), T, H, I, E, k,
        ctypes.byref(qc), ACTIVATIONS[activation], _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def experts_problem(a1q: torch.Tensor, a1q_scale: Optional[torch.Tensor], w13: torch.Tensor,
                    w13_scale: Optional[torch.Tensor], w2: torch.Tensor, w2_scale: Optional[torch.Tensor],
                    al: Alignment, out: torch.Tensor, identity: bool = False,
                    activation: str = "silu") -> ExpertsProblem:
    """One problem of moe_experts_multi (``identity``: NULL sorted_slot, E == 1, top_k == 1)."""
    T = a1q.shape[0]
    E, rows13, _ = w13.shape
    I = rows13 if activation.endswith("_no_mul") else rows13 // 2
    prob = ExpertsProblem(_ptr(a1q), _ptr(a1q_scale), _ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale),
                          _ptr(al.expert_offsets), None if identity else _ptr(al.sorted_slot), _ptr(al.tile_map),
                          _ptr(al.num_tiles), T, I, E, al.top_k, _ptr(out))
    # the struct holds raw device pointers: keep the tensors alive as long as it is
    prob._tensors = (a1q, a1q_scale, w13, w13_scale, w2, w2_scale, al, out)
    return prob


def workspace_size_multi(problems, H: int, quant: str) -> int:
    arr = (ExpertsProblem * len(problems))(*problems)
    return int(lib().moe_workspace_size_multi(arr, len(problems), H, ctypes.byref(_qc(quant))))


def moe_experts_multi(problems, H: int, quant: str, ws: torch.Tensor, activation: str = "silu", stream=None):
    """Several expert problems (``experts_problem``) in the same GEMM launches."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    arr = (ExpertsProblem * len(problems))(*problems)
    _check("moe_experts_multi", lib().moe_experts_multi(arr, len(problems), H, ctypes.byref(_qc(quant)),
                                                        ACTIVATIONS[activation], _ptr(ws), ws.numel(),
                                                        _stream(stream)))


def _gscale(g, device, name):
    """A global scale as the device fp32 tensor the C ABI takes (a Python number is copied)."""
    if isinstance(g, torch.Tensor):
        _need(g, torch.float32, name)
        return g
    return torch.tensor([float(g)], dtype=torch.float32, device=device)


def moe_prepare_nvfp4(a1: torch.Tensor, topk_weights: Optional[torch.Tensor], top_k: int,
                      apply_router_weight_on_input: bool, a1_gscale, a1q: Optional[torch.Tensor] = None,
                      a1q_sf: Optional[torch.Tensor] = None, stream=None):
    """NVFP4 prepare: a1 [T, H] bf16 -> (a1q [T, H/2] codes, a1q_sf [T, H/16] scale
    codes) with global scale ``a1_gscale`` (number or [1] fp32 device tensor)."""
    _need(a1, torch.bfloat16, "a1")
    _need(topk_weights, torch.float32, "topk_weights")
    T, H = a1.shape
    g = _gscale(a1_gscale, a1.device, "a1_gscale")
    if a1q is None:
        a1q = torch.empty((T, H // 2), dtype=torch.uint8, device=a1.device)
    if a1q_sf is None:
        a1q_sf = torch.empty((T, H // 16), dtype=torch.uint8, device=a1.device)
    _need(a1q, torch.uint8, "a1q")
    _need(a1q_sf, torch.uint8, "a1q_sf")
    _check("moe_prepare_nvfp4", lib().moe_prepare_nvfp4(
        _ptr(a1), _ptr(topk_weights), T, H, top_k, int(bool(apply_router_weight_on_input)), _ptr(g), _ptr(a1q),
        _ptr(a1q_sf), _stream(stream)))
    return a1q, a1q_sf


def workspace_size_nvfp4(T: int, H: int, I: int, E: int, top_k: int) -> int:
    return int(lib().moe_workspace_size_nvfp4(T, H, I, E, top_k))


def moe_experts_nvfp4(a1q: torch.Tensor, a1q_sf: torch.Tensor, a1_gscale, w13: torch.Tensor,
                      w13_sf: torch.Tensor, w13_gscale: torch.Tensor, w2: torch.Tensor, w2_sf: torch.Tensor,
                      w2_gscale: torch.Tensor, h_gscale, al: Alignment, out: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, identity: bool = False, stream=None,
                      activation: str = "silu") -> torch.Tensor:
    """Grouped expert MLPs with NVFP4 operands (``moe_experts_nvfp4``): packed codes
    a1q [T, H/2], w13 [E, 2I, H/2] (*_no_mul: [E, I, H/2]), w2 [E, H, I/2] with
    their scale codes (one per 16 elements) and fp32 global scales."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    for t, n in ((a1q, "a1q"), (a1q_sf, "a1q_sf"), (w13, "w13"), (w13_sf, "w13_sf"), (w2, "w2"), (w2_sf, "w2_sf")):
        _need(t, torch.uint8, n)
    _need(w13_gscale, torch.float32, "w13_gscale")
    _need(w2_gscale, torch.float32, "w2_gscale")
    T, H = a1q.shape[0], a1q.shape[1] * 2
    E, rows13, _ = w13.shape
    I = rows13 if activation.endswith("_no_mul") else rows13 // 2
    k = al.top_k
    ga = _gscale(a1_gscale, a1q.device, "a1_gscale")
    gh = _gscale(h_gscale, a1q.device, "h_gscale")
    if out is None:
        out = torch.empty((T * k, H), dtype=torch.bfloat16, device=a1q.device)
    _need(out, torch.bfloat16, "fused_expert_output")
    if ws is None:
        ws = torch.empty(max(workspace_size_nvfp4(T, H, I, E, k), 16), dtype=torch.uint8, device=a1q.device)
    _check("moe_experts_nvfp4", lib().moe_experts_nvfp4(
        _ptr(a1q), _ptr(a1q_sf), _ptr(ga), _ptr(w13), _ptr(w13_sf), _ptr(w13_gscale), _ptr(w2), _ptr(w2_sf),
        _ptr(w2_gscale), _ptr(gh), _ptr(al.expert_offsets), None if identity else _ptr(al.sorted_slot),
        _ptr(al.tile_map), _ptr(al.num_tiles), T, H, I, E, k, ACTIVATIONS[activation], _ptr(out), _ptr(ws),
        ws.numel(), _stream(stream)))
    return out


def layer_fused_workspace_size(T: int, H: int, I: int, E: int, top_k: int, has_shared: bool) -> int:
    return int(lib().moe_layer_fused_workspace_size(T, H, I, E, top_k, int(bool(has_shared))))


def moe_layer_fused(logits: torch.Tensor, a1: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, top_k: int,
                    scoring: int = MOE_SCORING_SOFTMAX_RENORM, apply_router_weight_on_input: bool = False,
                    shared_w13: Optional[torch.Tensor] = None, shared_w2: Optional[torch.Tensor] = None,
                    residual: Optional[torch.Tensor] = None, rms_weight: Optional[torch.Tensor] = None,
                    eps: float = 1e-6, topk_ids: Optional[torch.Tensor] = None,
                    topk_weights: Optional[torch.Tensor] = None, output: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The whole bf16 layer step in one launch (``moe_layer_fused``): w13 [E, 2I, H],
    w2 [E, H, I]; shared_w13 [2I, H] / shared_w2 [H, I] (or [1, ...]) for a shared expert."""
    _need(logits, torch.float32, "logits")
    for t, n in ((a1, "a1"), (w13, "w13"), (w2, "w2"), (shared_w13, "shared_w13"), (shared_w2, "shared_w2"),
                 (residual, "residual"), (rms_weight, "rms_weight")):
        _need(t, torch.bfloat16, n)
    T, H = a1.shape
    E, rows13, _ = w13.shape
    I = rows13 // 2
    dev = a1.device
    if topk_ids is None:
        topk_ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    if topk_weights is None:
        topk_weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    if output is None:
        output = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    if ws is None:
        ws = torch.empty(max(layer_fused_workspace_size(T, H, I, E, top_k, shared_w13 is not None), 16),
                         dtype=torch.uint8, device=dev)
    _check("moe_layer_fused", lib().moe_layer_fused(
        _ptr(logits), _ptr(a1), T, H, I, E, top_k, scoring, int(bool(apply_router_weight_on_input)), _ptr(w13),
        _ptr(w2), _ptr(shared_w13), _ptr(shared_w2), _ptr(residual), _ptr(rms_weight), eps, _ptr(topk_ids),
        _ptr(topk_weights), _ptr(output), _ptr(ws), ws.numel(), _stream(stream)))
    return output


def moe_finalize(fused_expert_output: torch.Tensor, topk_weights: Optional[torch.Tensor], top_k: int,
                 apply_router_weight_on_input: bool = False, shared: Optional[torch.Tensor] = None,
                 residual: Optional[torch.Tensor] = None, rms_weight: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, out_dtype: int = MOE_DT_BF16, out_global_scale: float = 1.0,
                 output: Optional[torch.Tensor] = None, out_scale: Optional[torch.Tensor] = None,
                 residual_out: Optional[torch.Tensor] = None, topk_ids: Optional[torch.Tensor] = None,
                 stream=None):
    _need(fused_expert_output, torch.bfloat16, "fused_expert_output")
    _need(topk_weights, torch.float32, "topk_weights")
    for t, n in ((shared, "shared"), (residual, "residual"), (rms_weight, "rms_weight"),
                 (residual_out, "residual_out")):
        _need(t, torch.bfloat16, n)
    S, H = fused_expert_output.shape
    T = S // top_k
    dev = fused_expert_output.device
    if output is None:
        if out_dtype == MOE_DT_NVFP4:
            output = torch.empty((T, H // 2), dtype=torch.uint8, device=dev)
        else:
            output = torch.empty((T, H), dtype=torch.float32 if out_dtype == MOE_DT_FP32 else torch.bfloat16,
                                 device=dev)
    if out_dtype == MOE_DT_NVFP4 and out_scale is None:
        out_scale = torch.empty((T, H // 16), dtype=torch.uint8, device=dev)
    _check("moe_finalize", lib().moe_finalize(
        _ptr(output), _ptr(fused_expert_output), _ptr(topk_weights), _ptr(topk_ids), _ptr(shared), _ptr(residual),
        _ptr(rms_weight), float(eps), T, H, top_k, int(bool(apply_router_weight_on_input)), out_dtype,
        _ptr(out_scale), float(out_global_scale), _ptr(residual_out), _stream(stream)))
    return output, out_scale


def moe_device_status(clear: bool = True) -> int:
    return int(lib().moe_device_status(int(clear)))


def moe_selftest_row_division(n: int, seed: int, stream=None) -> int:
    """Run the library's self-test of the requantisation division (see moe.h) on n
    pairs; returns how many results differ from the IEEE division."""
    cnt = torch.zeros(1, dtype=torch.int64, device="cuda")
    _check("moe_selftest_row_division",
           lib().moe_selftest_row_division(int(n), int(seed) & 0xFFFFFFFF, _ptr(cnt), _stream(stream)))
    return int(cnt.item())


def moe_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    """Launch the library's self-test of a device-side wait that runs out (see moe.h):
    afterwards moe_device_status() reports MOE_ERR_TIMEOUT."""
    _check("moe_selftest_wait_timeout", lib().moe_selftest_wait_timeout(int(limit_ns), _stream(stream)))


# ------------------------------------------------------------------ batched activation format
def batched_scale_shape(quant: str, E: int, M: int, H: int):
    """Shape of a1q_b_scale in the batched format (None for bf16)."""
    return {"bf16": None, "fp8": (E, M, H // 128), "fp8_token": (E, M), "fp8_tensor": (1,)}[quant]


def moe_prepare_batched(a1: torch.Tensor, topk_weights: Optional[torch.Tensor], al: "Alignment", E: int,
                        max_tokens: int, apply_router_weight_on_input: bool, quant: str, stream=None):
    """Prepare into the batched format (``moe_prepare_batched``): returns (a1q_b
    [E, max_tokens, H], a1q_b_scale or None, expert_num_tokens [E] int32)."""
    _need(a1, torch.bfloat16, "a1")
    T, H = a1.shape
    fp8 = quant != "bf16"
    qb = torch.empty((E, max_tokens, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=a1.device)
    shp = batched_scale_shape(quant, E, max_tokens, H)
    sb = None if shp is None else torch.empty(shp, dtype=torch.float32, device=a1.device)
    counts = torch.empty((E,), dtype=torch.int32, device=a1.device)
    qc = _qc(quant)
    nws = int(lib().moe_prepare_batched_workspace_size(T, H, ctypes.byref(qc)))
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=a1.device)
    _check("moe_prepare_batched", lib().moe_prepare_batched(
        _ptr(a1), _ptr(topk_weights), _ptr(al.expert_offsets), _ptr(al.sorted_slot), T, H, al.top_k, E, max_tokens,
        int(apply_router_weight_on_input), ctypes.byref(qc), _ptr(qb), _ptr(sb), _ptr(counts), _ptr(ws), ws.numel(),
        _stream(stream)))
    return qb, sb, counts


def workspace_size_batched(E: int, max_tokens: int, H: int, I: int, quant: str) -> int:
    return int(lib().moe_workspace_size_batched(E, max_tokens, H, I, ctypes.byref(_qc(quant))))


def moe_experts_batched(a1q_b: torch.Tensor, a1q_b_scale: Optional[torch.Tensor], w13: torch.Tensor,
                        w13_scale: Optional[torch.Tensor], w2: torch.Tensor, w2_scale: Optional[torch.Tensor],
                        expert_num_tokens: torch.Tensor, quant: str, out: Optional[torch.Tensor] = None,
                        ws: Optional[torch.Tensor] = None, activation: str = "silu", stream=None) -> torch.Tensor:
    """The experts on the batched format (``moe_experts_batched``): out [E, max_tokens, H] bf16."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    E, M, H = a1q_b.shape
    _, rows13, _ = w13.shape
    I = rows13 if activation.endswith("_no_mul") else rows13 // 2
    _need(expert_num_tokens, torch.int32, "expert_num_tokens")
    if out is None:
        out = torch.empty((E, M, H), dtype=torch.bfloat16, device=a1q_b.device)
    if ws is None:
        ws = torch.empty(max(workspace_size_batched(E, M, H, I, quant), 16), dtype=torch.uint8, device=a1q_b.device)
    _check("moe_experts_batched", lib().moe_experts_batched(
        _ptr(a1q_b), _ptr(a1q_b_scale), _ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), _ptr(expert_num_tokens),
        E, M, H, I, ctypes.byref(_qc(quant)), ACTIVATIONS[activation], _ptr(out), _ptr(ws), ws.numel(),
        _stream(stream)))
    return out


def moe_finalize_batched(out_b: torch.Tensor, topk_weights: Optional[torch.Tensor], topk_ids: torch.Tensor,
                         al: "Alignment", apply_router_weight_on_input: bool, shared=None, residual=None,
                         rms_weight=None, eps: float = 1e-6, output: Optional[torch.Tensor] = None,
                         residual_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_finalize reading each slot's row from a batched output [E, max_tokens, H]
    (``moe_finalize_batched``); bf16 output [T, H]."""
    E, M, H = out_b.shape
    T, k = topk_ids.shape
    if output is None:
        output = torch.empty((T, H), dtype=torch.bfloat16, device=out_b.device)
    _check("moe_finalize_batched", lib().moe_finalize_batched(
        _ptr(output), _ptr(out_b), M, _ptr(topk_weights), _ptr(topk_ids), _ptr(al.inv_slot), _ptr(al.expert_offsets),
        _ptr(shared), _ptr(residual), _ptr(rms_weight), eps, T, H, k, int(apply_router_weight_on_input), MOE_DT_BF16,
        None, 1.0, _ptr(residual_out), _stream(stream)))
    return output


# ------------------------------------------------------------------ linear projection
_DT = {torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_FP16, torch.float32: MOE_DT_FP32}


def _tensor(t: Optional[torch.Tensor], dtype, shape, name: str, device: int):
    """A tensor argument as its pointer: dtype, shape, contiguity and device checked."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name}: expected a tensor on the current CUDA device")
    raise ValueError(f"{name}: expected a contiguous tensor")


_INT_MAX = 2 ** 31 - 1  # (ctypes cuts a longer size without a word)


def _launch(stream: Optional[torch.cuda.Stream]):
    """(current device index, raw stream) of a call.  (A call without outputs to allocate costs the host a few
    microseconds, so the raw stream is asked for rather than a torch.cuda.Stream built around it.)"""
    dev = torch.cuda.current_device()
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError("stream: expected a stream of the current CUDA device")
    return dev, stream.cuda_stream


def _empty(shape, dtype, device, stream: Optional[torch.cuda.Stream]):
    """A buffer that the call makes itself: from the pool of the stream that it runs on, so that a workspace
    freed on return is not handed to work on another stream while the kernels still use it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _zeros(shape, dtype, device, stream: Optional[torch.cuda.Stream]):
    """As _empty, but zeros, set on that stream."""
    if stream is None:
        return torch.zeros(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.zeros(shape, dtype=dtype, device=device)


def _capturing(stream: Optional[torch.cuda.Stream]) -> bool:
    """The stream's work goes into a graph, whose replays the host does not see."""
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _linear_args(x: torch.Tensor, w: torch.Tensor, activation: str):
    if activation not in LINEAR_ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"x: expected bfloat16 or float16, got {x.dtype}")
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w: expected [M, K] and [N, K]")
    (M, K), N = x.shape, w.shape[0]
    if M > _INT_MAX or N > _INT_MAX or K > _INT_MAX:
        raise ValueError("x and w: expected sizes up to 2^31 - 1")
    return M, N, K, x.dtype, _DT[x.dtype], LINEAR_ACTIVATIONS[activation]


def moe_linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
               residual: Optional[torch.Tensor] = None, activation: str = "none", out: Optional[torch.Tensor] = None,
               out_dtype: Optional[torch.dtype] = None, preact: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """out = act(x w^T + bias) + residual (``moe_linear``): x [M, K], w [N, K], bias [N] bf16 or fp16; out and
    residual [M, N] in that type or fp32 (``out_dtype``); preact [M, N] receives x w^T + bias for the gradients.
    ``activation``: see ``LINEAR_ACTIVATIONS``."""
    M, N, K, dt, code, act = _linear_args(x, w, activation)
    if out is None:
        out = _empty((M, N), out_dtype or dt, x.device, stream)
    odt = out.dtype
    if odt is not dt and odt is not torch.float32 or out_dtype not in (None, odt):
        raise TypeError(f"out: expected {dt} or float32 as out_dtype says, got {odt}")
    dev, s = _launch(stream)
    _check("moe_linear", lib().moe_linear(
        _tensor(x, dt, (M, K), "x", dev), _tensor(w, dt, (N, K), "w", dev), _tensor(bias, dt, (N,), "bias", dev),
        _tensor(residual, odt, (M, N), "residual", dev), M, N, K, code, act, _DT[odt],
        _tensor(out, odt, (M, N), "out", dev), _tensor(preact, dt, (M, N), "preact", dev), s))
    return out


def linear_backward_workspace_size(M: int, N: int, K: int) -> int:
    if max(abs(M), abs(N), abs(K)) > _INT_MAX:
        raise ValueError("M, N and K: expected sizes up to 2^31 - 1")
    return int(lib().moe_linear_backward_workspace_size(M, N, K))


def moe_linear_backward(dout: torch.Tensor, x: torch.Tensor, w: torch.Tensor, preact: Optional[torch.Tensor] = None,
                        activation: str = "none", dx: Optional[torch.Tensor] = None,
                        dw: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                        ws: Optional[torch.Tensor] = None, need_dx: bool = True, need_dw: bool = True,
                        need_dbias: bool = False, stream=None):
    """Gradients of moe_linear (``moe_linear_backward``) given dout [M, N] (the operands' type or fp32) and the
    forward call's preact (unless ``activation`` is "none"): returns (dx [M, K], dw [N, K], dbias [N]) in the
    operands' type, None where not needed.  The residual's gradient is dout."""
    M, N, K, dt, code, act = _linear_args(x, w, activation)
    if dout.dtype is not dt and dout.dtype is not torch.float32:
        raise TypeError(f"dout: expected {dt} or float32, got {dout.dtype}")
    if dx is None and need_dx:
        dx = _empty((M, K), dt, x.device, stream)
    if dw is None and need_dw:
        dw = _empty((N, K), dt, x.device, stream)
    if dbias is None and need_dbias:
        dbias = _empty((N,), dt, x.device, stream)
    if ws is None:
        ws = _empty((max(linear_backward_workspace_size(M, N, K), 16),), torch.uint8, x.device, stream)
    dev, s = _launch(stream)
    _check("moe_linear_backward", lib().moe_linear_backward(
        _tensor(dout, dout.dtype, (M, N), "dout", dev), _DT[dout.dtype], _tensor(x, dt, (M, K), "x", dev),
        _tensor(w, dt, (N, K), "w", dev), _tensor(preact, dt, (M, N), "preact", dev), M, N, K, code, act,
        _tensor(dx, dt, (M, K), "dx", dev), _tensor(dw, dt, (N, K), "dw", dev), _tensor(dbias, dt, (N,), "dbias", dev),
        _tensor(ws, torch.uint8, ws.shape, "ws", dev), ws.numel(), s))
    return dx, dw, dbias


# ------------------------------------------------------------------ grouped route
# (plain values alone: an object that hashes by its identity, a tensor say, may change under its entry)
@functools.lru_cache(maxsize=1024)
def _route_config(score, n_group, topk_group, group_top, renormalize, scale):
    return ctypes.byref(route_config(score, n_group, topk_group, group_top, renormalize, scale))


def route_config(score: str = "sigmoid", n_group: int = 1, topk_group: int = 1, group_top: int = 1,
                 renormalize: bool = True, scale: float = 1.0) -> RouteConfig:
    if score not in SCORES:
        raise ValueError(f"unknown score {score!r}")
    if not all(-_INT_MAX <= v <= _INT_MAX for v in (n_group, topk_group, group_top)):
        raise ValueError("n_group, topk_group and group_top: expected sizes up to 2^31 - 1")
    return RouteConfig(SCORES[score], n_group, topk_group, group_top, int(bool(renormalize)), scale)


def moe_route_grouped(logits: torch.Tensor, top_k: int, bias: Optional[torch.Tensor] = None, score: str = "sigmoid",
                      n_group: int = 1, topk_group: int = 1, group_top: int = 1, renormalize: bool = True,
                      scale: float = 1.0, topk_ids: Optional[torch.Tensor] = None,
                      topk_weights: Optional[torch.Tensor] = None,
                      stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Router with sigmoid or softmax scores, a balance bias [E] fp32 that steers the choice alone, and expert
    groups (``moe_route_grouped``): logits [T, E] fp32, bf16 or fp16 -> topk_ids [T, top_k] int32 and topk_weights
    [T, top_k] fp32."""
    if logits.dtype not in _DT:
        raise TypeError(f"logits: expected float32, bfloat16 or float16, got {logits.dtype}")
    T, E = logits.shape
    if T > _INT_MAX or E > _INT_MAX or not 1 <= top_k <= _INT_MAX:
        raise ValueError("logits and top_k: expected sizes up to 2^31 - 1")
    cfg = _route_config(score, index(n_group), index(topk_group), index(group_top), bool(renormalize), float(scale))
    if topk_ids is None:
        topk_ids = _empty((T, top_k), torch.int32, logits.device, stream)
    if topk_weights is None:
        topk_weights = _empty((T, top_k), torch.float32, logits.device, stream)
    dev, s = _launch(stream)
    _check("moe_route_grouped", lib().moe_route_grouped(
        _tensor(logits, logits.dtype, (T, E), "logits", dev), _DT[logits.dtype],
        _tensor(bias, torch.float32, (E,), "bias", dev), T, E, top_k, cfg,
        _tensor(topk_ids, torch.int32, (T, top_k), "topk_ids", dev),
        _tensor(topk_weights, torch.float32, (T, top_k), "topk_weights", dev), s))
    return topk_ids, topk_weights


def moe_route_grouped_backward(dweights: torch.Tensor, logits: torch.Tensor, topk_ids: torch.Tensor,
                               score: str = "sigmoid", renormalize: bool = True, scale: float = 1.0,
                               bias: Optional[torch.Tensor] = None, dlogits: Optional[torch.Tensor] = None,
                               stream=None) -> torch.Tensor:
    """Gradient of moe_route_grouped's weights with respect to its logits (``moe_route_grouped_backward``), the
    choice topk_ids held fixed: dweights [T, top_k] fp32 -> dlogits [T, E] in the logits' type.  bias: the forward
    call's, needed where it masks experts."""
    if logits.dtype not in _DT:
        raise TypeError(f"logits: expected float32, bfloat16 or float16, got {logits.dtype}")
    (T, E), (_, top_k) = logits.shape, topk_ids.shape
    if T > _INT_MAX or E > _INT_MAX or top_k > _INT_MAX:
        raise ValueError("logits and topk_ids: expected sizes up to 2^31 - 1")
    cfg = _route_config(score, 1, 1, 1, bool(renormalize), float(scale))
    if dlogits is None:
        dlogits = _empty((T, E), logits.dtype, logits.device, stream)
    dev, s = _launch(stream)
    _check("moe_route_grouped_backward", lib().moe_route_grouped_backward(
        _tensor(dweights, torch.float32, (T, top_k), "dweights", dev),
        _tensor(logits, logits.dtype, (T, E), "logits", dev), _DT[logits.dtype],
        _tensor(bias, torch.float32, (E,), "bias", dev), _tensor(topk_ids, torch.int32, (T, top_k), "topk_ids", dev),
        T, E, top_k, cfg,
        _tensor(dlogits, logits.dtype, (T, E), "dlogits", dev), s))
    return dlogits


# ------------------------------------------------------------------ finalize, gradient
def finalize_backward_workspace_size(T: int, H: int) -> int:
    if max(abs(T), abs(H)) > _INT_MAX:
        raise ValueError("T and H: expected sizes up to 2^31 - 1")
    return int(lib().moe_finalize_backward_workspace_size(T, H))


def moe_finalize_backward(dout: torch.Tensor, fused_expert_output: Optional[torch.Tensor],
                          topk_weights: Optional[torch.Tensor], top_k: int,
                          residual_out: Optional[torch.Tensor] = None, rms_weight: Optional[torch.Tensor] = None,
                          eps: float = 1e-6, dresidual_out: Optional[torch.Tensor] = None,
                          dy: Optional[torch.Tensor] = None, dweights: Optional[torch.Tensor] = None,
                          dsum: Optional[torch.Tensor] = None, drms: Optional[torch.Tensor] = None,
                          ws: Optional[torch.Tensor] = None, need_dy: bool = True, need_dweights: bool = True,
                          need_dsum: bool = True, need_drms: bool = True, stream=None):
    """Gradients of moe_finalize with its bf16 output (``moe_finalize_backward``): given dout [T, H] bf16 (and
    dresidual_out, the gradient of residual_out), the expert rows and weights of the forward call, and with an
    RMSNorm its residual_out and rms_weight, returns (dy [T * top_k, H] bf16, dweights [T, top_k] fp32, dsum [T, H]
    bf16 -- the gradient of the shared row and of the residual --, drms [H] fp32), None where not needed.
    topk_weights None: the weights were applied on the input (no dweights)."""
    T, H = dout.shape
    if T > _INT_MAX or H > _INT_MAX or not 1 <= top_k <= _INT_MAX:
        raise ValueError("dout and top_k: expected sizes up to 2^31 - 1")
    bf, d = torch.bfloat16, dout.device
    if dy is None and need_dy:
        dy = _empty((T * top_k, H), bf, d, stream)
    if dweights is None and need_dweights and topk_weights is not None:
        dweights = _empty((T, top_k), torch.float32, d, stream)
    if dsum is None and need_dsum:
        dsum = _empty((T, H), bf, d, stream)
    if drms is None and need_drms and rms_weight is not None:
        drms = _empty((H,), torch.float32, d, stream)
    if ws is None and drms is not None:
        ws = _empty((max(finalize_backward_workspace_size(T, H), 16),), torch.uint8, d, stream)
    dev, s = _launch(stream)
    _check("moe_finalize_backward", lib().moe_finalize_backward(
        _tensor(dout, bf, (T, H), "dout", dev), _tensor(dresidual_out, bf, (T, H), "dresidual_out", dev),
        _tensor(residual_out, bf, (T, H), "residual_out", dev), _tensor(rms_weight, bf, (H,), "rms_weight", dev), eps,
        _tensor(fused_expert_output, bf, (T * top_k, H), "fused_expert_output", dev),
        _tensor(topk_weights, torch.float32, (T, top_k), "topk_weights", dev), T, H, top_k,
        _tensor(dy, bf, (T * top_k, H), "dy", dev), _tensor(dweights, torch.float32, (T, top_k), "dweights", dev),
        _tensor(dsum, bf, (T, H), "dsum", dev), _tensor(drms, torch.float32, (H,), "drms", dev),
        None if ws is None else _tensor(ws, torch.uint8, ws.shape, "ws", dev), 0 if ws is None else ws.numel(), s))
    return dy, dweights, dsum, drms


# ------------------------------------------------------------------ RMSNorm
_NORM_QUANTS = {q: ctypes.byref(QUANT_CONFIGS[q or "bf16"]) for q in (None, "bf16", "fp8", "fp8_token")}


def moe_rmsnorm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
                quant: Optional[str] = None, out: Optional[torch.Tensor] = None,
                residual_out: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                q_scale: Optional[torch.Tensor] = None, need_out: bool = True, need_residual_out: bool = True,
                stream=None):
    """RMSNorm of x + residual (``moe_rmsnorm``): x and residual [T, H], weight [H] bf16 -> (out [T, H] bf16,
    residual_out [T, H] bf16 -- the sum, made where there is a residual --, q [T, H] E4M3 codes (uint8), q_scale
    fp32), None where not needed.  quant: None or "bf16" (no q), "fp8" (a scale per 128 columns, [T, ceil(H / 128)]) or
    "fp8_token" ([T]), as moe_prepare's.  Gradients: ``moe_finalize_backward(dout, None, None, 1,
    residual_out=..., rms_weight=weight, need_dy=False)`` gives dsum (of x and of the residual) and drms."""
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x: expected [T, H]")
    T, H = shape
    if T > _INT_MAX or H > _INT_MAX:
        raise ValueError("x: expected sizes up to 2^31 - 1")
    if quant not in _NORM_QUANTS:
        raise ValueError(f"quant: expected None, 'bf16', 'fp8' or 'fp8_token', got {quant!r}")
    bf = torch.bfloat16
    if out is None and need_out:
        out = _empty(shape, bf, x.device, stream)
    if residual_out is None and need_residual_out and residual is not None:
        residual_out = _empty(shape, bf, x.device, stream)
    groups = (T, (H + 127) // 128) if quant == "fp8" else (T,)
    if quant == "fp8" or quant == "fp8_token":
        if q is None:
            q = _empty(shape, torch.uint8, x.device, stream)
        if q_scale is None:
            q_scale = _empty(groups, torch.float32, x.device, stream)
    elif q is not None or q_scale is not None:
        raise ValueError("q and q_scale: expected None without a quant")
    dev, s = _launch(stream)
    _check("moe_rmsnorm", lib().moe_rmsnorm(
        _tensor(x, bf, shape, "x", dev), _tensor(residual, bf, shape, "residual", dev),
        _tensor(weight, bf, (H,), "weight", dev), eps, T, H, _NORM_QUANTS[quant],
        _tensor(out, bf, shape, "out", dev), _tensor(residual_out, bf, shape, "residual_out", dev),
        _tensor(q, torch.uint8, shape, "q", dev), _tensor(q_scale, torch.float32, groups, "q_scale", dev), s))
    return out, residual_out, q, q_scale


# ------------------------------------------------------------------ grouped products
def _rows(name: str, order: str, S: int, top_k: int, token: bool = True) -> int:
    """Rows of a tensor in the given order; the order checked."""
    if order not in ROWS or order == "token" and not token:
        raise ValueError(f"{name}: expected 'sorted'{', ' if token else ' or '}'slot'{' or ' if token else ''}"
                         f"{repr('token') if token else ''}, got {order!r}")
    if order != "token":
        return S
    if S % top_k:
        raise ValueError(f"{name}: expected a multiple of top_k rows for the token order")
    return S // top_k


def _grouped_args(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, slots: Optional[torch.Tensor], top_k: int,
                  orders):
    """(S, E, N, K, dtype, dtype code) of a grouped product."""
    if w.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"w: expected bfloat16 or float16, got {w.dtype}")
    if w.dim() != 3 or x.dim() != 2 or offsets.dim() != 1 or (slots is not None and slots.dim() != 1):
        raise ValueError("w, the rows, expert_offsets and sorted_slot: expected [E, N, K], [rows, columns], [E + 1] and [S]")
    if not 1 <= top_k <= _INT_MAX:
        raise ValueError("top_k: expected 1 .. 2^31 - 1")
    if slots is None and any(o != "sorted" for o in orders):
        raise ValueError("sorted_slot: expected for rows in another order than 'sorted'")
    (E, N, K), S = w.shape, x.shape[0] if slots is None else slots.shape[0]
    if max(S, E, N, K) > _INT_MAX:
        raise ValueError("x and w: expected sizes up to 2^31 - 1")
    return S, E, N, K, w.dtype, _DT[w.dtype]


def grouped_linear_workspace_size(S: int, E: int, N: int, K: int, x_rows: str = "sorted") -> int:
    if max(abs(S), abs(E), abs(N), abs(K)) > _INT_MAX:
        raise ValueError("S, E, N and K: expected sizes up to 2^31 - 1")
    return int(lib().moe_grouped_linear_workspace_size(S, E, N, K, ROWS[x_rows]))


def grouped_linear_backward_workspace_size(S: int, E: int, N: int, K: int, dout_rows: str = "sorted",
                                           x_rows: str = "sorted") -> int:
    if max(abs(S), abs(E), abs(N), abs(K)) > _INT_MAX:
        raise ValueError("S, E, N and K: expected sizes up to 2^31 - 1")
    return int(lib().moe_grouped_linear_backward_workspace_size(S, E, N, K, ROWS[dout_rows], ROWS[x_rows]))


def moe_grouped_linear(x: torch.Tensor, w: torch.Tensor, expert_offsets: torch.Tensor,
                       sorted_slot: Optional[torch.Tensor] = None, top_k: int = 1, x_rows: str = "sorted",
                       out_rows: str = "sorted", out: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The experts' product over ragged groups of rows (``moe_grouped_linear``): out_p = x_p w[e]^T for the sorted
    rows p in [expert_offsets[e], expert_offsets[e + 1]); w [E, N, K] bf16 or fp16, expert_offsets [E + 1] and
    sorted_slot [S] int32 as moe_align writes them (sorted_slot may be None where every order is "sorted").
    x_rows, out_rows: the order of a tensor's rows (``ROWS``): "sorted" and "slot" have S rows, "token" (x alone)
    S / top_k.  out [S, N] in the operands' type; rows in front of the first group or behind the last are
    left as they were."""
    S, E, N, K, dt, code = _grouped_args(x, w, expert_offsets, sorted_slot, top_k, (x_rows, out_rows))
    rx, ro = _rows("x_rows", x_rows, S, top_k), _rows("out_rows", out_rows, S, top_k, False)
    if out is None:
        out = _empty((ro, N), dt, x.device, stream)
    if ws is None:
        size = grouped_linear_workspace_size(S, E, N, K, x_rows)
        ws = _empty((size,), torch.uint8, x.device, stream) if size else None
    dev, s = _launch(stream)
    i32 = torch.int32
    _check("moe_grouped_linear", lib().moe_grouped_linear(
        _tensor(x, dt, (rx, K), "x", dev), ROWS[x_rows], _tensor(w, dt, (E, N, K), "w", dev),
        _tensor(expert_offsets, i32, (E + 1,), "expert_offsets", dev), _tensor(sorted_slot, i32, (S,), "sorted_slot", dev),
        S, E, N, K, top_k, code, _tensor(out, dt, (ro, N), "out", dev), ROWS[out_rows],
        None if ws is None else _tensor(ws, torch.uint8, ws.shape, "ws", dev), 0 if ws is None else ws.numel(), s))
    return out


def moe_grouped_linear_backward(dout: torch.Tensor, x: Optional[torch.Tensor], w: torch.Tensor,
                                expert_offsets: torch.Tensor, sorted_slot: Optional[torch.Tensor] = None,
                                top_k: int = 1, dout_rows: str = "sorted", x_rows: str = "sorted",
                                dx_rows: str = "sorted", dx: Optional[torch.Tensor] = None,
                                dw: Optional[torch.Tensor] = None, dw_dtype: Optional[torch.dtype] = None,
                                accumulate: bool = False, ws: Optional[torch.Tensor] = None, need_dx: bool = True,
                                need_dw: bool = True, stream=None):
    """Gradients of moe_grouped_linear (``moe_grouped_linear_backward``) given dout, rows of N columns in
    dout_rows order, and the forward call's x (None without dw): returns (dx [S, K] in dx_rows order, "sorted" or
    "slot", in the operands' type; dw [E, N, K] in that type or fp32 (``dw_dtype``)), None where not needed.
    accumulate: dw (then required) is added to instead of written."""
    S, E, N, K, dt, code = _grouped_args(dout, w, expert_offsets, sorted_slot, top_k, (dout_rows, x_rows, dx_rows))
    rd, rx = _rows("dout_rows", dout_rows, S, top_k), _rows("x_rows", x_rows, S, top_k)
    ro = _rows("dx_rows", dx_rows, S, top_k, False)
    if accumulate and dw is None:
        raise ValueError("dw: expected with accumulate")
    if dx is None and need_dx:
        dx = _empty((ro, K), dt, dout.device, stream)
    if dw is None and need_dw:
        dw = _empty((E, N, K), dw_dtype or dt, dout.device, stream)
    wdt = dt if dw is None else dw.dtype
    if wdt is not dt and wdt is not torch.float32 or dw is not None and dw_dtype not in (None, wdt):
        raise TypeError(f"dw: expected {dt} or float32 as dw_dtype says, got {wdt}")
    if ws is None:
        ws = _empty((max(grouped_linear_backward_workspace_size(S, E, N, K, dout_rows, x_rows), 16),), torch.uint8,
                    dout.device, stream)
    dev, s = _launch(stream)
    i32 = torch.int32
    _check("moe_grouped_linear_backward", lib().moe_grouped_linear_backward(
        _tensor(dout, dt, (rd, N), "dout", dev), ROWS[dout_rows], _tensor(x, dt, (rx, K), "x", dev), ROWS[x_rows],
        _tensor(w, dt, (E, N, K), "w", dev), _tensor(expert_offsets, i32, (E + 1,), "expert_offsets", dev),
        _tensor(sorted_slot, i32, (S,), "sorted_slot", dev), S, E, N, K, top_k, code,
        _tensor(dx, dt, (ro, K), "dx", dev), ROWS[dx_rows], _tensor(dw, wdt, (E, N, K), "dw", dev), _DT[wdt],
        int(bool(accumulate)), None if ws is None else _tensor(ws, torch.uint8, ws.shape, "ws", dev),
        0 if ws is None else ws.numel(), s))
    return dx, dw


# ------------------------------------------------------------------ activation
def _activation_args(gu: torch.Tensor, activation: str):
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    if gu.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"gu: expected bfloat16 or float16, got {gu.dtype}")
    if gu.dim() != 2 or not activation.endswith("_no_mul") and gu.shape[1] % 2:
        raise ValueError("gu: expected [S, 2 I], or [S, I] for the *_no_mul activations")
    (S, cols), dt = gu.shape, gu.dtype
    if S > _INT_MAX or cols > _INT_MAX:
        raise ValueError("gu: expected sizes up to 2^31 - 1")
    return S, cols, cols if activation.endswith("_no_mul") else cols // 2, dt


def moe_activation(gu: torch.Tensor, activation: str = "silu", h: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """The activation between an expert's two products (``moe_activation``, ``ACTIVATIONS``): gu [S, 2 I] = [g | u]
    (*_no_mul: [S, I]) bf16 or fp16 -> h [S, I]."""
    S, cols, I, dt = _activation_args(gu, activation)
    if h is None:
        h = _empty((S, I), dt, gu.device, stream)
    dev, s = _launch(stream)
    _check("moe_activation", lib().moe_activation(
        _tensor(gu, dt, (S, cols), "gu", dev), S, I, _DT[dt], ACTIVATIONS[activation], _tensor(h, dt, (S, I), "h", dev),
        s))
    return h


def moe_activation_backward(dh: torch.Tensor, gu: torch.Tensor, activation: str = "silu",
                            dgu: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                            need_h: bool = False, stream=None):
    """Gradient of moe_activation (``moe_activation_backward``): dh [S, I] -> (dgu, as gu; h, the activation's output
    made again in the same pass, None where not needed)."""
    S, cols, I, dt = _activation_args(gu, activation)
    if dgu is None:
        dgu = _empty((S, cols), dt, gu.device, stream)
    if h is None and need_h:
        h = _empty((S, I), dt, gu.device, stream)
    dev, s = _launch(stream)
    _check("moe_activation_backward", lib().moe_activation_backward(
        _tensor(dh, dt, (S, I), "dh", dev), _tensor(gu, dt, (S, cols), "gu", dev), S, I, _DT[dt], ACTIVATIONS[activation],
        _tensor(dgu, dt, (S, cols), "dgu", dev), _tensor(h, dt, (S, I), "h", dev), s))
    return dgu, h
