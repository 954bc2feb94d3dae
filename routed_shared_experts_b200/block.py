"""The expert half of a decoder block around a layer.

    attention output --moe_linear(w_o) + residual--> residual stream
        --moe_rmsnorm_quantize--> the layer's x (16-bit rows and / or codes)
        --moe_linear(w_r)--> router logits (fp32) --> the layer

``MoEBlock`` owns the buffers between the steps and writes the layer's inputs
(``x``, ``x_scale``, ``logits``, and ``x_r`` for the shared gate of an 8-bit
layer) in place, so a step - captured or not - is three C-ABI calls more than the
layer's own. The layer's output is added to the
residual stream by the next block's norm (``moe_rmsnorm_quantize`` takes the sum
of its two inputs), not by a kernel of its own.
"""
from __future__ import annotations

import torch

from . import capi
from .layer import capture_forward, gate_rows


class MoEBlock:
    """``layer``: a ``MoELayer`` or ``FusedSharedMoELayer``. ``weights``:

    * ``gamma`` [H] (bf16 or fp32): the norm before the layer;
    * ``w_r`` [E,H] bf16 and optional ``logit_bias`` fp32 [E]: the router linear;
    * ``w_o`` [H,A] with the attention output ``attn`` [T,A], bf16, or e4m3 codes
      with ``attn_scale`` fp32 [T] and ``w_o_scale`` fp32 [H] or [1].

    ``attn`` (and ``attn_scale``) and ``residual`` [T,H] bf16 are read, and
    ``residual`` is updated in place, at every ``forward``.
    """

    def __init__(self, layer, weights: dict, attn: torch.Tensor, residual: torch.Tensor,
                 attn_scale: torch.Tensor | None = None, eps: float = 1e-6):
        cfg = layer.cfg
        self.layer, self.w, self.eps = layer, weights, eps
        self.attn, self.attn_scale, self.residual = attn, attn_scale, residual
        self.device = layer.device
        T, H = cfg.T, cfg.H
        inp = layer.inp
        self.quant = None if cfg.dtype == "bf16" else capi.DTYPES["mxfp8" if cfg.dtype in capi.MX_FORMATS else "fp8"]
        if getattr(layer, "quantize_x", False) or getattr(layer, "router_gemm", False):
            raise ValueError("the block quantises x and computes the logits itself")
        # the router reads the 16-bit rows; a bf16 layer reads the same ones, and so does a shared gate
        if self.quant is None:
            self.y = inp["x"]
        else:
            gated = gate_rows(cfg, inp)
            self.y = torch.empty((T, H), dtype=torch.bfloat16, device=self.device) if gated is None else gated
        self.o_dt = capi.MOE_DT_BF16 if attn_scale is None else capi.MOE_DT_FP8_E4M3

    @property
    def out(self):
        return self.layer.out

    def forward(self, stream=None, probes=None):
        """Enqueue one step on ``stream``; returns the layer's output (to be
        added to ``self.residual`` by the next norm)."""
        s = stream or torch.cuda.current_stream(self.device)
        w, inp, res = self.w, self.layer.inp, self.residual
        capi.moe_linear(self.o_dt, self.attn, self.attn_scale, w["w_o"], w.get("w_o_scale"), None,
                        capi.ACTS["none"], res, res, s)
        capi.moe_rmsnorm_quantize(self.quant, res, None, w["gamma"], self.eps, None, self.y,
                                  None if self.quant is None else inp["x"],
                                  None if self.quant is None else inp["x_scale"], s)
        capi.moe_linear(capi.MOE_DT_BF16, self.y, None, w["w_r"], None, w.get("logit_bias"), capi.ACTS["none"], None,
                        inp["logits"], s)
        return self.layer.forward(s, probes)

    def capture(self, stream=None, steps: int = 1) -> torch.cuda.CUDAGraph:
        """The step as a replayable graph (``capture_forward``)."""
        return capture_forward(self, stream, steps)

    @property
    def launches_per_step(self) -> int:
        """Kernels this library launches per forward()."""
        return self.layer.launches_per_step + 3
