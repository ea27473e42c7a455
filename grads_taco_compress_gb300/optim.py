"""The optimiser's half of a training step: the norm of all gradients, and an
AdamW step over many tensors at once.

The taco_grad_norm and taco_adamw entry points of include/taco.h, which states
formulas, rounding and errors. States are kept in 32 bits or in 8, as FP8 block
tensors (``fp8``). Steps done, rate and gradient scale can all live on the
device: a step that is captured in a CUDA graph goes on counting when it is
replayed::

    opt = AdamW(block.parameters(), lr=3e-4, bits=8)
    norm = opt.step(block.gradients(), max_norm=1.0)
    block.refresh()

Wrong arguments raise ValueError, a status of the library TacoError.
"""

from __future__ import annotations

import math
from typing import NamedTuple, Sequence

import torch

from .binding import _check
from .fp8 import BLOCK, Fp8Tensor, _binding, _handle


class AdamState(NamedTuple):
    """First moment m and second moment v of a parameter of n elements: f32
    tensors of n elements; or both Fp8Tensors [1, n] (codes on 16 bytes, no gaps
    between scales), v then the square root of the second moment."""

    m: torch.Tensor | Fp8Tensor
    v: torch.Tensor | Fp8Tensor


def taco_adam_state(param: torch.Tensor, bits: int = 32) -> AdamState:
    """The zero state of a parameter, in 32 bits or in 8."""
    if bits not in (8, 32):
        raise ValueError("bits must be 8 or 32")
    if bits == 32:
        return AdamState(*(torch.zeros(param.shape, dtype=torch.float32, device=param.device) for _ in range(2)))
    n = param.numel()

    def zero():
        # zero codes under the scale 1, as taco_fp8_quantize leaves a block of zeros
        return Fp8Tensor(torch.zeros((1, n), dtype=torch.uint8, device=param.device),
                         torch.full((1, -(-n // BLOCK)), 127, dtype=torch.uint8, device=param.device))

    return AdamState(zero(), zero())


def taco_grad_norm(grads: Sequence[torch.Tensor], max_norm: float = math.inf, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """f32 [2]: the norm of all tensors together, and the factor that clips it to
    max_norm (1 where it is not above, NaN where the norm is infinite or NaN),
    which taco_adamw takes as ``grad_scale=r[1:]``. ``workspace``:
    taco_grad_norm_workspace_bytes(len(grads)) bytes."""
    r = _binding().grad_norm(grads, max_norm, out, workspace, _handle(stream))
    if type(r) is int:
        _check(r, "taco_grad_norm")
    return r


def taco_adamw(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], states: Sequence[AdamState],
               counter: torch.Tensor, lr: float | torch.Tensor, betas: tuple[float, float] = (0.9, 0.999),
               eps: float = 1e-8, weight_decay: float | Sequence[float] = 0.01,
               grad_scale: torch.Tensor | None = None, masters: Sequence[torch.Tensor | None] | None = None,
               stream=None) -> None:
    """One AdamW step of all params, in place: contiguous bf16, f16 or f32
    tensors, each with a gradient of its type or f32. ``counter``: int32 [2],
    zero before the first step, whose first entry counts the steps. lr: a number
    or an f32 tensor of one element. weight_decay: a number, or one for each
    parameter. grad_scale: f32 of one element that gradients are multiplied by;
    where it is infinite or NaN, nothing changes. masters: for each parameter an
    f32 tensor with its exact value, or None; a 16-bit parameter without one is
    rounded by thresholds that keep small changes on average."""
    try:
        beta1, beta2 = betas
    except (TypeError, ValueError):
        raise ValueError("betas must be two numbers") from None
    r = _binding().adamw(params, grads, states, counter, lr, beta1, beta2, eps, weight_decay, grad_scale, masters,
                         _handle(stream))
    if type(r) is int:
        _check(r, "taco_adamw")


class AdamW:
    """Parameters with their states: ``taco_adam_state`` of each in ``bits``,
    f32 masters of the 16-bit ones where ``masters`` is set, and the counter.
    ``lr`` may be a device tensor that the program changes between steps."""

    def __init__(self, params: Sequence[torch.Tensor], lr: float | torch.Tensor = 1e-3,
                 betas: tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float | Sequence[float] = 0.01, bits: int = 32, masters: bool = False):
        self.params = list(params)
        if not self.params:
            raise ValueError("no parameters")
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        dev = self.params[0].device
        self.states = [taco_adam_state(p, bits) for p in self.params]
        self.masters = [p.detach().float() if masters and p.dtype != torch.float32 else None for p in self.params]
        self.counter = torch.zeros(2, dtype=torch.int32, device=dev)
        self.norm = torch.zeros(2, dtype=torch.float32, device=dev)

    def step(self, grads: Sequence[torch.Tensor], max_norm: float | None = None, stream=None) -> torch.Tensor | None:
        """One step. With max_norm the gradients are clipped to it as a whole, a
        norm that is infinite or NaN leaves everything as it is, and the norm and
        the factor (f32 [2], written again by the next step) are returned."""
        norm = None
        if max_norm is not None:
            norm = taco_grad_norm(grads, max_norm, out=self.norm, stream=stream)
        taco_adamw(self.params, grads, self.states, self.counter, self.lr, self.betas, self.eps, self.weight_decay,
                   None if norm is None else norm[1:], self.masters, stream=stream)
        return norm
