"""FP8 block tensors and the layer operators that make and read them.

The taco_*_fp8 and taco_fp8_* entry points of include/taco.h, which states
formats, formulas and errors. A block tensor is E4M3 codes plus one E8M0 scale
byte per row and 128 columns, or per 128 x 128 tile for weights. As in
``binding``, torch supplies device memory and streams only, every output can be
preallocated, and the work goes to ``stream`` or to the current one. Codes and
scales that a call allocates share one allocation, and so does a norm's rstd
with its checkpoint, or with h where there is none: holding one holds the other. The
arguments are marshalled by a compiled module (csrc/fp8_binding.cpp): these
calls take a few microseconds on small inputs, and so do their arguments in
Python. Wrong arguments (tensors on different devices among them) raise
ValueError, a status of the library TacoError.

A linear layer y = x W^T in training::

    xq, _ = taco_fp8_quantize(x)                          # or an operator's 8-bit output
    wq, wt = taco_fp8_quantize(w, cols=True, tile=128)    # W and its transpose
    y = taco_matmul_fp8(xq, wq)
    dyq, dyt = taco_fp8_quantize(dy, cols=True)
    dx = taco_matmul_fp8(dyq, wt)
    _, xt = taco_fp8_quantize(xq, rows=False, cols=True)  # the checkpoint, along the tokens
    taco_matmul_fp8(dyt, xt, out=dw, add=dw)              # f32 running gradient
"""

from __future__ import annotations

import importlib.machinery
import importlib.util
from typing import NamedTuple

import torch

from .binding import LIB_PATH, _check, _lib

BLOCK = 128
BINDING_PATH = LIB_PATH.with_name("_fp8_binding.so")


class Fp8Tensor(NamedTuple):
    """Codes u8 [rows, cols] and scales u8 [rows, ceil(cols / 128)], or
    [ceil(rows / 128), ceil(cols / 128)] for one scale per 128 x 128 tile.
    Rows of codes start at multiples of 16 bytes, rows of scales at multiples
    of 4 (``fp8_empty`` allocates them so). The checkpoint of a gated
    activation has a leading dimension of 2: gate, up."""

    codes: torch.Tensor
    scales: torch.Tensor

    def dequantize(self) -> torch.Tensor:
        """The values as fp32 (plain torch operations, for inspection)."""
        s = self.scales.contiguous().view(torch.float8_e8m0fnu).float()
        if s.shape[-2] != self.codes.shape[-2]:
            s = s.repeat_interleave(BLOCK, dim=-2)[..., : self.codes.shape[-2], :]
        s = s.repeat_interleave(BLOCK, dim=-1)[..., : self.codes.shape[-1]]
        return self.codes.contiguous().view(torch.float8_e4m3fn).float() * s


class RmsNormOutput(NamedTuple):
    y: Fp8Tensor
    h: torch.Tensor
    rstd: torch.Tensor
    checkpoint: Fp8Tensor | None


_BINDING = None


def _binding():
    """The compiled binding (raises if it has not been built)."""
    global _BINDING
    if _BINDING is None:
        _lib()
        if not BINDING_PATH.exists():
            raise RuntimeError(f"the compiled binding is not built ({BINDING_PATH} missing): run "
                               "`python -m grads_taco_compress_gb300.build_lib` first")
        loader = importlib.machinery.ExtensionFileLoader("_fp8_binding", str(BINDING_PATH))
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_fp8_binding", loader))
        loader.exec_module(module)
        module.types(Fp8Tensor, RmsNormOutput)
        _BINDING = module
    return _BINDING


def _handle(stream):
    return None if stream is None else int(stream.cuda_stream)


def _up(n: int, m: int) -> int:
    return -(-n // m) * m


def fp8_empty(*shape: int, tile: int = 1, device="cuda") -> Fp8Tensor:
    """An uninitialised FP8 block tensor [rows, cols] or [planes, rows, cols]."""
    *lead, rows, cols = shape
    kb, srows = -(-cols // BLOCK), -(-rows // tile)
    ld, lds = _up(cols, 16), _up(kb, 16)
    codes = torch.empty_strided((*lead, rows, cols), (rows * ld, ld, 1)[-len(shape):], dtype=torch.uint8, device=device)
    scales = torch.empty_strided((*lead, srows, kb), (srows * lds, lds, 1)[-len(shape):], dtype=torch.uint8,
                                 device=device)
    return Fp8Tensor(codes, scales)


def taco_fp8_quantize(x, rows: bool = True, cols: bool = False, tile: int = 1, out: Fp8Tensor | None = None,
                      out_t: Fp8Tensor | None = None, stream=None):
    """x [M, K] (bf16, f16, f32 or an Fp8Tensor) -> (its rows as an Fp8Tensor
    [M, K] or None, its transpose as one [K, M] or None), from one read. tile:
    128 for one scale per 128 x 128 tile (weights). ``out`` and ``out_t`` are
    where the two go; one whose flag is not set is left alone."""
    r = _binding().quantize(x, rows, cols, tile, out, out_t, _handle(stream))
    if type(r) is int:
        _check(r, "taco_fp8_quantize")
    return r


def taco_rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                      eps: float = 1e-6, checkpoint: bool | Fp8Tensor = False, out: Fp8Tensor | None = None,
                      h: torch.Tensor | None = None, rstd: torch.Tensor | None = None,
                      stream=None) -> RmsNormOutput:
    """Root-mean-square norm of h = x + residual, [M, H], with the 8-bit output
    y = h * rstd * weight and, with ``checkpoint`` (True or a preallocated
    Fp8Tensor), h in 8 bits for the backward pass. Returns (y, h, rstd,
    checkpoint); h is x itself where there is no residual. ``h`` may be x or
    residual (in place)."""
    r = _binding().rms_norm(x, weight, residual, eps, checkpoint, out, h, rstd, _handle(stream))
    if type(r) is int:
        _check(r, "taco_rms_norm_fp8")
    return r


def taco_rms_norm_fp8_backward(dy: torch.Tensor, saved, weight: torch.Tensor, rstd: torch.Tensor,
                               dh: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                               dw: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradients (dx [M, H], dw f32 [H]) of taco_rms_norm_fp8 from ``saved``, its
    8-bit checkpoint (an Fp8Tensor) or its h. ``dh`` is the gradient that h
    received elsewhere; ``dx``, the gradient of x and of residual alike, may be
    dy, dh or h (in place). ``workspace``: taco_rms_norm_workspace_bytes bytes."""
    r = _binding().rms_norm_backward(dy, saved, weight, rstd, dh, dx, dw, workspace, _handle(stream))
    if type(r) is int:
        _check(r, "taco_rms_norm_fp8_backward")
    return r


def taco_swiglu_fp8(gate_up: torch.Tensor, checkpoint: bool | Fp8Tensor = False, out: Fp8Tensor | None = None,
                    stream=None):
    """y = silu(gate) * up in 8 bits, from gate_up [M, 2 F] (gate in the first F
    columns). With ``checkpoint`` (True or a preallocated Fp8Tensor [2, M, F])
    gate and up are kept in 8 bits. Returns (y, checkpoint or None)."""
    r = _binding().swiglu(gate_up, checkpoint, out, _handle(stream))
    if type(r) is int:
        _check(r, "taco_swiglu_fp8")
    return r


def taco_swiglu_fp8_backward(dy: torch.Tensor, checkpoint: Fp8Tensor, out: torch.Tensor | None = None,
                             stream=None) -> torch.Tensor:
    """Gradient [M, 2 F] of gate_up from taco_swiglu_fp8's checkpoint."""
    r = _binding().swiglu_backward(dy, checkpoint, out, _handle(stream))
    if type(r) is int:
        _check(r, "taco_swiglu_fp8_backward")
    return r


def taco_matmul_fp8(a: Fp8Tensor, b: Fp8Tensor, out: torch.Tensor | None = None,
                    out_dtype: torch.dtype = torch.bfloat16, add: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """a [M, K] times the transpose of b [N, K] (+ add) -> [M, N], summed in
    fp32 on the block-scaled tensor cores. ``add`` may be ``out`` (in place)."""
    r = _binding().matmul(a, b, out, out_dtype, add, _handle(stream))
    if type(r) is int:
        _check(r, "taco_matmul_fp8")
    return r
