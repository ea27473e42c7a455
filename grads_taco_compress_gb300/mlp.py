"""A tensor-parallel gated MLP block trained in FP8, R logical ranks on one GPU.

The layer whose outputs and gradients the compressed AllReduce carries (TACO,
gist.science pt summary, §1: the tensor-parallel layers' intermediate
tensors), with the FP8 block-tensor operators between the two exchanges:

  forward   h = x + residual; n = norm(h) in 8 bits, h kept in 8 bits
            rank r: gate|up = n W_in[r]^T; y = silu(gate) up in 8 bits, gate
            and up kept in 8 bits; part[r] = y W_out[r]^T
            out = AllReduce(part)                        (compressed)
  backward  rank r: dy = dout W_out[r]; dW_out[r] += dout^T y
            dgate|dup from the checkpoints; dW_in[r] += (dgate|dup)^T n
            part[r] = (dgate|dup) W_in[r]
            dn = AllReduce(part); dx, dW_norm from the checkpoint of h

Weights are bf16 masters, quantised with one scale per 128 x 128 tile by
``refresh`` (after every update); weight gradients are running f32 sums. As in
``allreduce``, every step is a libtaco call, but for the addition of the norm
weight's gradient to its running sum.

Several forward passes may be open at a time (micro-batches)::

    out1, h1 = block.forward(x1, r1); saved1 = block.saved
    out2, h2 = block.forward(x2, r2); saved2 = block.saved
    dx1 = block.backward(dout1, dh1, saved1)
    dx2 = block.backward(dout2, dh2, saved2)
"""

from __future__ import annotations

from typing import NamedTuple

import torch

from . import binding as tb
from . import fp8 as F
from .allreduce import EmulatedTwoShotAllReduce


class MlpSaved(NamedTuple):
    """What a forward pass keeps for its backward pass: the norm's output, rstd
    and checkpoint, and each rank's gated output with the checkpoint of gate and
    up. All in 8 bits but rstd; h itself is the caller's alone."""

    y: F.Fp8Tensor
    rstd: torch.Tensor
    checkpoint: F.Fp8Tensor
    gated: tuple


class TensorParallelMlp:
    """Weights, gradients and the launch sequence of one block. ``saved``: the
    MlpSaved of the last forward pass, None once its backward pass has run."""

    def __init__(self, R: int, M: int, h: int, f: int, block: int = 128, eps: float = 1e-6, device="cuda"):
        """R ranks, M tokens, hidden size h, f gated channels in all (f / R a
        rank); block is the AllReduce's Hadamard block."""
        if f % R:
            raise ValueError("f must be a multiple of R")
        self.R, self.M, self.h, self.f, self.eps = R, M, h, f // R, float(eps)
        dev = torch.device(device)

        def weight(*shape):
            return (torch.randn(shape, device=dev) / shape[-1] ** 0.5).to(torch.bfloat16)

        self.w_norm = torch.ones(h, dtype=torch.float32, device=dev)
        self.w_in = [weight(2 * self.f, h) for _ in range(R)]
        self.w_out = [weight(h, self.f) for _ in range(R)]
        self.dw_norm = torch.zeros(h, dtype=torch.float32, device=dev)
        self.dw_in = [torch.zeros((2 * self.f, h), dtype=torch.float32, device=dev) for _ in range(R)]
        self.dw_out = [torch.zeros((h, self.f), dtype=torch.float32, device=dev) for _ in range(R)]
        self.part = torch.empty((R, M, h), dtype=torch.bfloat16, device=dev)
        self.reduce_forward = EmulatedTwoShotAllReduce(R, M, h, block, device=dev)
        self.reduce_backward = EmulatedTwoShotAllReduce(R, M, h, block, device=dev)
        self.saved = None
        self._replaced = False      # a forward pass took the place of a saved state
        self.refresh()

    def refresh(self) -> None:
        """Quantise the weights and their transposes (after an update of the masters)."""
        self._in = [F.taco_fp8_quantize(w, cols=True, tile=F.BLOCK) for w in self.w_in]
        self._out = [F.taco_fp8_quantize(w, cols=True, tile=F.BLOCK) for w in self.w_out]

    def forward(self, x: torch.Tensor, residual: torch.Tensor, out: torch.Tensor | None = None):
        """bf16 x, residual [M, h] -> (the block's output [M, h], in ``out`` or a
        new tensor, and the residual stream x + residual [M, h])."""
        if out is None:
            out = torch.empty((self.M, self.h), dtype=torch.bfloat16, device=self.part.device)
        n = F.taco_rms_norm_fp8(x, self.w_norm, residual, self.eps, checkpoint=True)
        gated = []
        for r in range(self.R):
            y, kept = F.taco_swiglu_fp8(F.taco_matmul_fp8(n.y, self._in[r][0]), checkpoint=True)
            F.taco_matmul_fp8(y, self._out[r][0], out=self.part[r])
            gated.append((y, kept))
        self.reduce_forward(self.part, out=out)
        self._replaced = self.saved is not None
        self.saved = MlpSaved(n.y, n.rstd, n.checkpoint, tuple(gated))
        return out, n.h

    def backward(self, dout: torch.Tensor, dh: torch.Tensor | None = None,
                 saved: MlpSaved | None = None) -> torch.Tensor:
        """dout: gradient of the output, dh: of the residual stream, of the forward
        pass that left ``saved`` (None: the last one, the only one open). Returns
        the gradient of x and of residual; the weights' are added to dw_*."""
        if saved is None:
            if self.saved is None:
                raise ValueError("no forward pass to go back through")
            if self._replaced:
                raise ValueError("more than one forward pass since the last backward: pass the saved state of one")
            saved = self.saved
        dq, dt = F.taco_fp8_quantize(dout, cols=True)
        _, nt = F.taco_fp8_quantize(saved.y, rows=False, cols=True)
        for r, (y, kept) in enumerate(saved.gated):
            _, yt = F.taco_fp8_quantize(y, rows=False, cols=True)
            F.taco_matmul_fp8(dt, yt, out=self.dw_out[r], add=self.dw_out[r])
            dgu = F.taco_swiglu_fp8_backward(F.taco_matmul_fp8(dq, self._out[r][1]), kept)
            gq, gt = F.taco_fp8_quantize(dgu, cols=True)
            F.taco_matmul_fp8(gt, nt, out=self.dw_in[r], add=self.dw_in[r])
            F.taco_matmul_fp8(gq, self._in[r][1], out=self.part[r])
        dn = self.reduce_backward(self.part)
        dx, dw = F.taco_rms_norm_fp8_backward(dn, saved.checkpoint, self.w_norm, saved.rstd, dh=dh)
        self.dw_norm += dw
        if saved is self.saved:
            self.saved, self._replaced = None, False
        return dx
