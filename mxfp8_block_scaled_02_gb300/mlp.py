"""A gated MLP block on the quantised layers.

    t = x + residual
    out = down( silu(gate) * up ),   [gate | up] = gate_up( rmsnorm(t) )

Four steps, each handing its output to the next already quantised in the
weights' format (MXFP8, MXFP4 or NVFP4): norm with the residual's addition,
merged gate and up projection, gated activation, down projection.  One library
call (ops.gated_mlp) launches them.
"""

from __future__ import annotations

import torch

from . import ops


class GatedMLP:
    """norm_weight bf16 [K]; gate_up PackedWeights [2 F, K] (gate rows first);
    down PackedWeights [K, F] in the same format (process_weights for MXFP8,
    process_weights_fp4 for the 4-bit ones).  x_tensor_scale / h_tensor_scale:
    NVFP4's calibrated scales of the norm's and the activation's output."""

    def __init__(self, norm_weight: torch.Tensor, gate_up: ops.PackedWeights, down: ops.PackedWeights, *,
                 eps: float = 1e-6, x_tensor_scale: torch.Tensor | None = None,
                 h_tensor_scale: torch.Tensor | None = None):
        if gate_up.fmt != down.fmt or gate_up.fmt not in ("e4m3", "mxfp4", "nvfp4"):
            raise ValueError(f"gate_up ({gate_up.fmt}) and down ({down.fmt}) must share one of e4m3, mxfp4, nvfp4")
        if gate_up.batched or down.batched or gate_up.N != 2 * down.K or down.N != gate_up.K:
            raise ValueError(f"gate_up [{gate_up.N}, {gate_up.K}] and down [{down.N}, {down.K}] are not [2 F, K] and [K, F]")
        self.norm_weight, self.gate_up, self.down, self.eps = norm_weight, gate_up, down, eps
        self.x_tensor_scale, self.h_tensor_scale = x_tensor_scale, h_tensor_scale

    def __call__(self, x: torch.Tensor, residual: torch.Tensor | None = None
                 ) -> tuple[torch.Tensor, torch.Tensor | None]:
        """x bf16 [..., K], residual bf16 or fp32 like x -> (bf16 [..., K], x + residual)."""
        return ops.gated_mlp(x, self.norm_weight, self.gate_up, self.down, residual, eps=self.eps,
                             x_tensor_scale=self.x_tensor_scale, h_tensor_scale=self.h_tensor_scale)
