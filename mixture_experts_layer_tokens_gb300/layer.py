"""One fused-MoE layer step composed from the C-ABI calls, with every buffer
allocated once up front (PyTorch allocates, the library computes); the gradients of the
finalize alone are made by each MoELayer.router_backward call, and the buffers of the experts'
gradients by the first MoELayer.experts_backward call.

Step: moe_route -> moe_align -> moe_prepare -> moe_experts [-> shared expert via
  moe_experts with one expert and the identity permutation] -> moe_finalize, on the
caller's stream.  The shared expert needs no routing: when it runs as calls of its own
and neither its GEMMs nor the routed experts' split units across CTAs (whose waits
assume every CTA of the launch resident, which two concurrent launches cannot
promise), it runs on a second stream forked at the start of the step and joined
before the finalize, so its GEMMs overlap the routing, quantisation, gather and the
routed experts' GEMMs (which take their units from a counter, so CTAs that start
late because the shared expert still holds their SMs take fewer units).
A layer with a MoERouter makes its logits itself (moe_linear on the hidden states, then
moe_route_grouped in place of moe_route), and its router can be trained beside fixed
experts: moe_finalize_backward, moe_route_grouped_backward, moe_linear_backward.
A layer with input_norm normalises what it is given first (moe_rmsnorm, with the residual's
addition), and an fp8 layer's quantised rows come from the same launch in place of moe_prepare.
The experts of a bf16 layer are trained by MoEExperts: moe_grouped_linear and moe_activation
with their gradients.
NVFP4 layers use moe_prepare_nvfp4 and moe_experts_nvfp4 (the shared expert
stays bf16).  Single-launch layers run the whole step as one moe_layer_fused launch.

The shared expert sees the unweighted bf16 input, as the shared-expert row of
the flashinfer finalize fusion is added unscaled.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import moe
from .inputs import LayerConfig, LayerInputs


class MoERouter:
    """The router with its gate: hidden states -> logits (``moe_linear``) -> choice and weights
    (``moe_route_grouped``), and the gradients back (``moe_route_grouped_backward``,
    ``moe_linear_backward``), every buffer allocated once.

    gate_w [E, H] and gate_bias [E] (None: none) bf16 or fp16; balance_bias [E] fp32 (None: none) steers the
    choice alone.  The logits are fp32.  The other arguments are moe_route_grouped's."""

    def __init__(self, T: int, gate_w: torch.Tensor, top_k: int, gate_bias: Optional[torch.Tensor] = None,
                 balance_bias: Optional[torch.Tensor] = None, score: str = "sigmoid", n_group: int = 1,
                 topk_group: int = 1, group_top: int = 1, renormalize: bool = True, scale: float = 1.0):
        self.gate_w, self.gate_bias, self.balance_bias = gate_w, gate_bias, balance_bias
        (E, H), dev = gate_w.shape, gate_w.device
        self.T, self.E, self.top_k = T, E, top_k
        self.weigh = dict(score=score, renormalize=renormalize, scale=scale)
        self.choose = dict(self.weigh, n_group=n_group, topk_group=topk_group, group_top=group_top)
        self.logits = torch.empty((T, E), dtype=torch.float32, device=dev)
        self.topk_ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
        self.topk_weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
        self._grads = None

    def forward(self, a1: torch.Tensor, topk_ids: Optional[torch.Tensor] = None,
                topk_weights: Optional[torch.Tensor] = None, stream=None):
        """(topk_ids, topk_weights) of the hidden states a1 [T, H]."""
        ids = self.topk_ids if topk_ids is None else topk_ids
        w = self.topk_weights if topk_weights is None else topk_weights
        moe.moe_linear(a1, self.gate_w, self.gate_bias, out=self.logits, stream=stream)
        return moe.moe_route_grouped(self.logits, self.top_k, self.balance_bias, topk_ids=ids, topk_weights=w,
                                     stream=stream, **self.choose)

    def backward(self, dweights: torch.Tensor, a1: torch.Tensor, topk_ids: Optional[torch.Tensor] = None, stream=None):
        """Gradients of the last forward call's weights: (dgate_w, dgate_bias or None, da1, dlogits), the choice
        (topk_ids, when forward wrote another buffer than its own) held fixed.  da1 is what reaches the hidden
        states through the gate alone: the experts' share, and the residual's, are the caller's to add.  Buffers of
        the router, written again by the next call."""
        if self._grads is None:
            (E, H), dt, dev = self.gate_w.shape, self.gate_w.dtype, self.gate_w.device
            # (made by the first call, so from the pool of the stream that it runs on)
            self._dlogits = moe._empty((self.T, E), torch.float32, dev, stream)
            self._grads = dict(
                dx=moe._empty((self.T, H), dt, dev, stream), dw=moe._empty((E, H), dt, dev, stream),
                dbias=None if self.gate_bias is None else moe._empty((E,), dt, dev, stream),
                ws=moe._empty((max(moe.linear_backward_workspace_size(self.T, E, H), 16),), torch.uint8, dev, stream))
        ids = self.topk_ids if topk_ids is None else topk_ids
        moe.moe_route_grouped_backward(dweights, self.logits, ids, bias=self.balance_bias, dlogits=self._dlogits,
                                       stream=stream, **self.weigh)
        da1, dgate_w, dgate_bias = moe.moe_linear_backward(self._dlogits, a1, self.gate_w, stream=stream, **self._grads)
        return dgate_w, dgate_bias, da1, self._dlogits


class MoEExperts:
    """The experts as separate calls that keep what lies between their products, and their gradients: [g | u] =
    x w13^T (``moe_grouped_linear``), h = act(g) u (``moe_activation``), y = h w2^T, and back; every buffer allocated
    once.

    w13 [E, 2I, H] (the *_no_mul activations [E, I, H]) and w2 [E, H, I] bf16 or fp16; T tokens of top_k experts each;
    dw_dtype: the weights' gradients', fp32 or (None) the weights' type.  dw13 and dw2 start as zeros, so that the first
    backward call may add to them; an object that is made under capture has to write them first."""

    def __init__(self, w13: torch.Tensor, w2: torch.Tensor, T: int, top_k: int, activation: str = "silu",
                 dw_dtype: Optional[torch.dtype] = None, stream=None):
        (E, rows13, H), I, S = w13.shape, w2.shape[2], T * top_k
        if tuple(w2.shape) != (E, H, I) or rows13 != (I if activation.endswith("_no_mul") else 2 * I):
            raise ValueError("w13 and w2: expected [E, 2I, H] (*_no_mul: [E, I, H]) and [E, H, I]")
        self.w13, self.w2, self.T, self.top_k, self.activation = w13, w2, T, top_k, activation
        dt, dev = w13.dtype, w13.device
        if dw_dtype not in (None, dt, torch.float32):
            raise TypeError(f"dw_dtype: expected {dt} or float32, got {dw_dtype}")
        empty = lambda shape, dtype=dt: moe._empty(shape, dtype, dev, stream)  # noqa: E731
        self.gu, self.h = empty((S, rows13)), empty((S, I))
        self.y = empty((S, H))
        self.dh, self.drows, self.da1 = empty((S, I)), empty((S, H)), empty((T, H))
        # (zeros set in a graph would be set again by each of its replays)
        self._summed = not (w13.is_cuda and moe._capturing(stream))
        self._kept: Optional[bool] = False  # [g | u] is a hidden call's (None: calls were captured, and replays go unseen)
        grad = moe._zeros if self._summed else moe._empty
        self.dw13, self.dw2 = (grad(shape, dw_dtype or dt, dev, stream) for shape in ((E, rows13, H), (E, H, I)))
        self._zeroed = None  # the zeros are there: for a first backward call on another stream than this one
        if w13.is_cuda and self._summed:
            self._zeroed = torch.cuda.Event()
            self._zeroed.record(stream if stream is not None else torch.cuda.current_stream(dev))
        self.ws = empty((max(moe.grouped_linear_workspace_size(S, E, rows13, H, "token"),
                             moe.grouped_linear_workspace_size(S, E, H, I, "sorted"),
                             moe.grouped_linear_backward_workspace_size(S, E, H, I, "slot", "sorted"),
                             moe.grouped_linear_backward_workspace_size(S, E, rows13, H, "sorted", "token"), 16),),
                        torch.uint8)

    def _slots(self, al: "moe.Alignment") -> torch.Tensor:
        return al.sorted_slot if self.T else al.sorted_slot[:0]  # (an Alignment of no tokens holds room for one slot)

    def hidden(self, a1: torch.Tensor, al: "moe.Alignment", stream=None) -> torch.Tensor:
        """h [S, I] in sorted order, [g | u] kept beside it: the forward pass up to the second product."""
        moe.moe_grouped_linear(a1, self.w13, al.expert_offsets, self._slots(al), self.top_k, x_rows="token", out=self.gu,
                               ws=self.ws, stream=stream)
        h = moe.moe_activation(self.gu, self.activation, h=self.h, stream=stream)
        self._kept = None if self._kept is None or moe._capturing(stream) else True
        return h

    def forward(self, a1: torch.Tensor, al: "moe.Alignment", stream=None) -> torch.Tensor:
        """y [T * top_k, H], the unweighted rows by slots, of the hidden states a1 [T, H]."""
        self.hidden(a1, al, stream)
        return moe.moe_grouped_linear(self.h, self.w2, al.expert_offsets, self._slots(al), self.top_k, out_rows="slot",
                                      out=self.y, ws=self.ws, stream=stream)

    def backward(self, dy: torch.Tensor, a1: torch.Tensor, al: "moe.Alignment", accumulate: bool = False, stream=None):
        """Gradients of the last forward (or hidden) call, given dy [T * top_k, H] by slots: (dw13, dw2, da1).  Once for each
        such call, whose [g | u] it replaces by its gradient: a second call is refused, but not where the object's calls
        were captured, since a replay may have made [g | u] again.
        accumulate: dw13 and dw2 are added to.  da1 [T, H] is what reaches the hidden states through these experts
        alone.  Buffers of this object, written again (or added to) by the next call; a bf16 da1 is summed by
        moe_finalize, an fp16 one is not made (None)."""
        capturing = moe._capturing(stream)
        if capturing:
            self._kept = None
        if self._kept is False:
            raise ValueError("backward: expected a forward (or hidden) call since the last backward call, which used it up")
        if accumulate and not self._summed:
            raise ValueError("accumulate: expected after a call that writes, for gradients made under capture")
        if self._zeroed is not None and not capturing:  # (what is captured cannot wait for what is not)
            (stream if stream is not None else torch.cuda.current_stream()).wait_event(self._zeroed)
            self._zeroed = None
        kw = dict(accumulate=accumulate, ws=self.ws, stream=stream)
        moe.moe_grouped_linear_backward(dy, self.h, self.w2, al.expert_offsets, self._slots(al), self.top_k,
                                        dout_rows="slot", dx=self.dh, dw=self.dw2, **kw)
        # (dgu takes the place of [g | u]'s copy: each value is read before it is written)
        if self._kept:
            self._kept = False
        moe.moe_activation_backward(self.dh, self.gu, self.activation, dgu=self.gu, stream=stream)
        moe.moe_grouped_linear_backward(self.gu, a1, self.w13, al.expert_offsets, self._slots(al), self.top_k,
                                        x_rows="token", dx_rows="slot", dx=self.drows, dw=self.dw13, **kw)
        self._summed = True
        if self.drows.dtype is not torch.bfloat16:
            return self.dw13, self.dw2, None
        moe.moe_finalize(self.drows, None, self.top_k, True, output=self.da1, stream=stream)
        return self.dw13, self.dw2, self.da1


class MoELayer:
    """router: a MoERouter of the same tokens, experts and top_k that takes the place of moe_route (the
    forward call's logits are then not read and may be None).  keep_residual: forward also writes the sum before
    the RMSNorm to residual_out, which router_backward needs.  input_norm: weight [H] bf16 of an RMSNorm (eps
    1e-6) in front of the layer; its gradient is moe_finalize_backward's, from the sum that was normalised."""

    def __init__(self, inp: LayerInputs, stream: Optional[torch.cuda.Stream] = None,
                 router: Optional[MoERouter] = None, keep_residual: bool = False,
                 input_norm: Optional[torch.Tensor] = None):
        cfg = self.cfg = inp.cfg
        assert not cfg.finalize_only
        self.router = router
        if router is not None and ((router.T, router.E, router.top_k) != (cfg.T, cfg.E, cfg.top_k) or
                                   cfg.single_launch):
            raise ValueError("router: expected one of the layer's tokens, experts and top_k, and separate launches")
        if keep_residual and cfg.single_launch:
            raise ValueError("keep_residual: expected separate launches")
        if input_norm is not None and cfg.single_launch:
            raise ValueError("input_norm: expected separate launches")
        self.inp = inp
        dev = inp.logits.device
        T, H, I, E, k = cfg.T, cfg.H, cfg.I, cfg.E, cfg.top_k
        self.input_norm, self.trainer = input_norm, None
        if input_norm is not None:
            self.a1 = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
            self.stream_sum = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        # the norm quantises for the experts, in place of moe_prepare
        self.norm_quant = input_norm is not None and cfg.quant in ("fp8", "fp8_token") and not cfg.weight_on_input
        self.residual_out = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if keep_residual else None
        self.scoring = moe.MOE_SCORING_SIGMOID if cfg.scoring == "sigmoid" else moe.MOE_SCORING_SOFTMAX_RENORM
        self.topk_ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.topk_weights = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.al = moe.Alignment(T, k, E, dev)
        self.nvfp4 = cfg.quant == "nvfp4"
        fp8 = cfg.quant != "bf16" and not self.nvfp4
        # bf16 without weight-on-input: prepare is the passthrough (a1q is a1)
        self.passthrough = cfg.quant == "bf16" and not cfg.weight_on_input
        self.y = torch.empty((T * k, H), dtype=torch.bfloat16, device=dev)
        if self.nvfp4:
            # packed codes and one E4M3 scale code per 16 elements; fp32 global scales on the device
            self.a1q = torch.empty((T, H // 2), dtype=torch.uint8, device=dev)
            self.a1q_scale = torch.empty((T, H // 16), dtype=torch.uint8, device=dev)
            self.g_a = torch.tensor([inp.extra["a1_gscale"]], dtype=torch.float32, device=dev)
            self.g_h = torch.tensor([inp.extra["h_gscale"]], dtype=torch.float32, device=dev)
            self.ws = torch.empty(max(moe.workspace_size_nvfp4(T, H, I, E, k), 16), dtype=torch.uint8, device=dev)
        else:
            self.a1q = None if self.passthrough else torch.empty(
                (T, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev)
            self.a1q_scale = (torch.empty(moe.scale_shape(cfg.quant, T, H), dtype=torch.float32, device=dev)
                              if fp8 else None)
            self.ws = torch.empty(max(moe.workspace_size(T, H, I, E, k, cfg.quant), 16), dtype=torch.uint8,
                                  device=dev)
        self.out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        self.shared = None
        if cfg.shared_I:
            self.shared = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
            ids0 = torch.zeros((T, 1), dtype=torch.int32, device=dev)
            self.al_shared = moe.moe_align(ids0, 1, stream=stream)
            self.ws_shared = torch.empty(max(moe.workspace_size(T, H, cfg.shared_I, 1, 1, "bf16"), 16),
                                         dtype=torch.uint8, device=dev)
            self.side = torch.cuda.Stream(device=dev)
            self.ev_fork = torch.cuda.Event()
            self.ev_join = torch.cuda.Event()
        # the whole step as one launch: a bf16 SiLU layer whose shared expert (if any) has the
        # routed experts' I
        self.single = cfg.single_launch
        if self.single:
            assert cfg.quant == "bf16" and cfg.activation == "silu" and cfg.shared_I in (0, I)
            self.ws_fused = torch.empty(max(moe.layer_fused_workspace_size(T, H, I, E, k, cfg.shared_I > 0), 16),
                                        dtype=torch.uint8, device=dev)
        # a bf16 layer whose shared expert has the routed experts' I and activation runs both
        # in the same GEMM launches (moe_experts_multi)
        self.fused_shared = (cfg.shared_I == I and cfg.quant == "bf16" and cfg.activation == "silu")
        # the shared expert on the second stream: its own calls, neither they (one expert, T
        # rows: split only for T <= 16) nor the routed experts (fp8 never; bf16 and NVFP4
        # at most 16 slots per expert) split units
        routed_splits = cfg.quant in ("bf16", "nvfp4") and T * k <= 16 * E
        self.shared_side = bool(cfg.shared_I) and not self.fused_shared and T > 16 and not routed_splits
        if self.fused_shared:
            a_dummy = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
            self.ws_multi = torch.empty(max(moe.workspace_size_multi(
                [moe.experts_problem(a_dummy, None, inp.w13, None, inp.w2, None, self.al, self.y),
                 moe.experts_problem(a_dummy, None, inp.shared_w13, None, inp.shared_w2, None, self.al_shared,
                                     self.shared, identity=True)], H, "bf16"), 16), dtype=torch.uint8, device=dev)

    def forward(self, logits: Optional[torch.Tensor], a1: torch.Tensor, stream=None,
                residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        """a1 [T, H] bf16: the hidden states; with input_norm what the norm takes.  residual (input_norm alone): the
        residual stream [T, H], added to a1 before the norm; the sum is what the finalize adds in place of the
        inputs' residual.  Without it the finalize adds the inputs' residual as it does without a norm, not a1: where a1
        is itself the residual stream (a first block), it has to be the inputs' residual too."""
        cfg, inp = self.cfg, self.inp
        if residual is not None and self.input_norm is None:
            raise ValueError("residual: expected with input_norm alone")
        if self.single:
            return moe.moe_layer_fused(
                logits, a1, inp.w13, inp.w2, cfg.top_k, self.scoring, cfg.weight_on_input,
                shared_w13=inp.shared_w13[0] if cfg.shared_I else None,
                shared_w2=inp.shared_w2[0] if cfg.shared_I else None, residual=inp.residual,
                rms_weight=inp.rms_weight, eps=1e-6, topk_ids=self.topk_ids, topk_weights=self.topk_weights,
                output=self.out, ws=self.ws_fused, stream=stream)
        main = stream if stream is not None else torch.cuda.current_stream()
        if self.input_norm is not None:
            moe.moe_rmsnorm(a1, self.input_norm, residual=residual, eps=1e-6, quant=cfg.quant if self.norm_quant else None,
                            out=self.a1, residual_out=None if residual is None else self.stream_sum,
                            q=self.a1q if self.norm_quant else None,
                            q_scale=self.a1q_scale if self.norm_quant else None, stream=stream)
            a1 = self.a1
        if self.shared_side:
            self.ev_fork.record(main)
            self.side.wait_event(self.ev_fork)
            moe.moe_experts(a1, None, inp.shared_w13, None, inp.shared_w2, None, self.al_shared, "bf16",
                            out=self.shared, ws=self.ws_shared, identity=True, stream=self.side)
            self.ev_join.record(self.side)
        if self.router is not None:
            self.router.forward(a1, self.topk_ids, self.topk_weights, stream=stream)
        else:
            moe.moe_route(logits, cfg.top_k, self.scoring, self.topk_ids, self.topk_weights, stream=stream)
        moe.moe_align(self.topk_ids, cfg.E, out=self.al, stream=stream)
        if self.passthrough:
            a1q, a1q_scale = a1, None
        elif self.norm_quant:
            a1q, a1q_scale = self.a1q, self.a1q_scale
        elif self.nvfp4:
            a1q, a1q_scale = moe.moe_prepare_nvfp4(a1, self.topk_weights, cfg.top_k, cfg.weight_on_input, self.g_a,
                                                   self.a1q, self.a1q_scale, stream=stream)
        else:
            a1q, a1q_scale = moe.moe_prepare(a1, self.topk_weights, cfg.top_k, cfg.weight_on_input, cfg.quant,
                                             self.a1q, self.a1q_scale, stream=stream)
        shared = self.experts(a1q, a1q_scale, a1, stream, shared_launched=self.shared_side)
        if self.shared_side:
            main.wait_event(self.ev_join)
        moe.moe_finalize(self.y, self.topk_weights, cfg.top_k, cfg.weight_on_input, shared=shared,
                         residual=inp.residual if residual is None else self.stream_sum, rms_weight=inp.rms_weight,
                         output=self.out, residual_out=self.residual_out, stream=stream)
        return self.out

    def router_backward(self, dout: torch.Tensor, a1: torch.Tensor, residual_out: Optional[torch.Tensor] = None,
                        stream=None, dresidual_out: Optional[torch.Tensor] = None, need_dy: bool = False):
        """Gradients that train the router of a layer (whose experts are held fixed, or trained by experts_backward
        from the finalize gradients' dy, made with need_dy): dout [T, H] bf16, the
        gradient of the last forward call's output, and a1, the hidden states that the router saw in it (with input_norm
        the layer's a1, not what forward was given) -> (finalize gradients, router gradients), as
        moe_finalize_backward and MoERouter.backward return them.  residual_out: the sum before the RMSNorm (layers
        with one; None: what a keep_residual layer's forward call wrote).  The router weights of a layer that
        applies them on the input have no gradient here."""
        if self.router is None or self.cfg.weight_on_input:
            raise ValueError("router_backward needs a MoERouter whose weights are applied in the finalize")
        if residual_out is None:
            residual_out = self.residual_out
        if residual_out is None and self.inp.rms_weight is not None:
            raise ValueError("router_backward under an RMSNorm needs residual_out, or a layer with keep_residual")
        fin = moe.moe_finalize_backward(dout, self.y, self.topk_weights, self.cfg.top_k, residual_out=residual_out,
                                        rms_weight=self.inp.rms_weight, dresidual_out=dresidual_out, need_dy=need_dy,
                                        stream=stream)
        return fin, self.router.backward(fin[1], a1, self.topk_ids, stream=stream)

    def experts_backward(self, dy: torch.Tensor, a1: torch.Tensor, dw_dtype: Optional[torch.dtype] = None,
                         accumulate: bool = False, stream=None):
        """Gradients of the routed experts of a bf16 layer, given dy [T * top_k, H] bf16 (moe_finalize_backward's, by
        slots) and the hidden states a1 of the last forward call (with input_norm: the layer's a1): (dw13, dw2, da1),
        as MoEExperts.backward returns them.  [g | u] and h are made again from a1.  dw_dtype: as MoEExperts',
        chosen by the first call.  accumulate: dw13 and dw2 are added to, by the first call to zeros (which has to write
        where it is captured)."""
        if self.cfg.quant != "bf16" or self.cfg.weight_on_input or self.single:
            raise ValueError("experts_backward needs a bf16 layer of separate launches, its weights applied in the finalize")
        if self.trainer is not None and dw_dtype not in (None, self.trainer.dw13.dtype):
            raise ValueError(f"dw_dtype: the first call's was {self.trainer.dw13.dtype}")
        if self.trainer is None:
            self.trainer = MoEExperts(self.inp.w13, self.inp.w2, self.cfg.T, self.cfg.top_k, self.cfg.activation, dw_dtype,
                                      stream)
        # (the weights that the forward call read, not those of the first call here)
        self.trainer.w13, self.trainer.w2 = self.inp.w13, self.inp.w2
        self.trainer.hidden(a1, self.al, stream)
        return self.trainer.backward(dy, a1, self.al, accumulate, stream)

    def experts(self, a1q, a1q_scale, a1, stream=None, shared_launched=False):
        """The routed experts into self.y and the shared expert (if any) into
        self.shared -- one moe_experts_multi call when they can share launches;
        shared_launched: the step has already run the shared expert (second stream).
        Returns the shared-expert rows or None."""
        cfg, inp = self.cfg, self.inp
        if self.shared is not None and self.fused_shared:
            moe.moe_experts_multi(
                [moe.experts_problem(a1q, a1q_scale, inp.w13, inp.w13_scale, inp.w2, inp.w2_scale, self.al, self.y),
                 moe.experts_problem(a1, None, inp.shared_w13, None, inp.shared_w2, None, self.al_shared, self.shared,
                                     identity=True)], cfg.H, "bf16", self.ws_multi, stream=stream)
            return self.shared
        if self.nvfp4:
            moe.moe_experts_nvfp4(a1q, a1q_scale, self.g_a, inp.w13, inp.w13_scale, inp.extra["w13_gscale"], inp.w2,
                                  inp.w2_scale, inp.extra["w2_gscale"], self.g_h, self.al, out=self.y, ws=self.ws,
                                  stream=stream, activation=cfg.activation)
        else:
            moe.moe_experts(a1q, a1q_scale, inp.w13, inp.w13_scale, inp.w2, inp.w2_scale, self.al, cfg.quant,
                            activation=cfg.activation, out=self.y, ws=self.ws, stream=stream)
        if self.shared is None:
            return None
        if shared_launched:
            return self.shared
        return moe.moe_experts(a1, None, inp.shared_w13, None, inp.shared_w2, None, self.al_shared, "bf16",
                               out=self.shared, ws=self.ws_shared, identity=True, stream=stream)


class FinalizeStep:
    """The finalize-only workload: route over k logits, then finalize to bf16
    and to NVFP4."""

    def __init__(self, inp: LayerInputs):
        cfg = self.cfg = inp.cfg
        assert cfg.finalize_only
        self.inp = inp
        dev = inp.logits.device
        T, H, k = cfg.T, cfg.H, cfg.top_k
        self.topk_ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.topk_weights = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        self.out_fp4 = torch.empty((T, H // 2), dtype=torch.uint8, device=dev)
        self.out_sf = torch.empty((T, H // 16), dtype=torch.uint8, device=dev)

    def weights(self, stream=None):
        moe.moe_route(self.inp.logits, self.cfg.top_k, moe.MOE_SCORING_SOFTMAX_RENORM, self.topk_ids,
                      self.topk_weights, stream=stream)
        return self.topk_weights

    def finalize(self, nvfp4: bool, stream=None):
        inp = self.inp
        if nvfp4:
            return moe.moe_finalize(inp.y, self.topk_weights, self.cfg.top_k, False, shared=inp.extra["shared"],
                                    residual=inp.residual, rms_weight=inp.rms_weight, eps=1e-6,
                                    out_dtype=moe.MOE_DT_NVFP4, out_global_scale=1.0, output=self.out_fp4,
                                    out_scale=self.out_sf, topk_ids=inp.topk_ids, stream=stream)
        return moe.moe_finalize(inp.y, self.topk_weights, self.cfg.top_k, False, shared=inp.extra["shared"],
                                residual=inp.residual, rms_weight=inp.rms_weight, eps=1e-6,
                                out_dtype=moe.MOE_DT_BF16, output=self.out, topk_ids=inp.topk_ids, stream=stream)
