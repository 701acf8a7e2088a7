"""Experts in microscaled 4-bit floating point: the SwiGLU experts of a mixture-of-experts layer with weights and
activations in blocks of 32 four-bit values that share a power-of-two scale (MXFP4, see include/moe.h).

Next to the layer's own int4 weights (dequantised inside the grouped GEMMs, activations in fp16) this form multiplies
4-bit by 4-bit on the tensor cores; routing comes from the layer's router (``Layer.route``).  Every step is one of the
operators in ``ops``.
"""
from __future__ import annotations

from typing import Tuple

import torch

from . import ops

Packed = Tuple[torch.Tensor, torch.Tensor]   # codes [E, N, K/2], scales [E, N, K/32]


class Mx4Experts:
    """E experts FFN_e(x) = W_down,e (silu(W_gate,e x) * (W_up,e x)) on a CUDA device.

    ``gateup``: the rows of W_gate, then those of W_up of each expert (N = 2I, K = H); ``down``: N = H, K = I.
    H and I are multiples of 32."""

    def __init__(self, gateup: Packed, down: Packed):
        self.gateup, self.down = gateup, down
        self.E, n, h2 = gateup[0].shape
        self.H, self.I = 2 * h2, n // 2
        if tuple(down[0].shape) != (self.E, self.H, self.I // 2) or n % 2:
            raise ValueError(f"gateup {tuple(gateup[0].shape)} and down {tuple(down[0].shape)} are not of the same experts")

    @classmethod
    def from_dense(cls, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor) -> "Mx4Experts":
        """Quantise gate and up [E, I, H] and down [E, H, I] (bf16, fp16 or fp32)."""
        return cls(cls.pack(torch.cat((gate, up), dim=1)), cls.pack(down))

    @staticmethod
    def pack(w: torch.Tensor) -> Packed:
        E, n, k = w.shape
        codes, scales = ops.mx4_quantize(w.contiguous().view(E * n, k))
        return codes.view(E, n, k // 2), scales.view(E, n, k // 32)

    def forward(self, x, idx, gates, base=None, out=None, *, stream=None):
        """out [T, H] = base + sum_j gates[:, j] * FFN_{idx[:, j]}(x) for x [T, H] bf16, idx [T, k] int32 (negative: none)
        and gates [T, k] fp32."""
        return ops._run(self._forward, stream, x, idx, gates, base, out)

    def _forward(self, x, idx, gates, base, out):
        d = ops.dispatch_rows(None, idx, self.E)
        codes, scales = ops.mx4_quantize(x, pos=d.pos)
        h = ops.mx4_matmul(codes, scales, *self.gateup, d.offsets)
        codes, scales = ops.mx4_quantize(h, act="swiglu")
        y = ops.mx4_matmul(codes, scales, *self.down, d.offsets)
        return ops.combine_weighted(y, d.pos, gates, base, out)
