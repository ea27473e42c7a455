"""FP8 block tensors and the layer operators that make and read them.

Argument marshalling of the taco_*_fp8 and taco_fp8_* entry points of
include/taco.h, which states formats, formulas and errors. A block tensor is
E4M3 codes plus one E8M0 scale byte per row and 128 columns, or per 128 x 128
tile for weights. As in ``binding``, torch supplies device memory and streams
only, every output can be preallocated, and the work goes to ``stream`` or to
the current one.

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

import ctypes
from typing import NamedTuple

import torch

from .binding import _check, _lib, _ptr

BLOCK = 128
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


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


class _Fp8Struct(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("ld_codes", ctypes.c_int64),
                ("ld_scales", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("tile_rows", ctypes.c_int32)]


def _up(n: int, m: int) -> int:
    return -(-n // m) * m


def _stream_of(stream, t: torch.Tensor) -> int:
    # torch.cuda.current_stream() without building its Stream object (2.9 us -> 0.1 us a call)
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else int(stream.cuda_stream)


def fp8_empty(*shape: int, tile: int = 1, device="cuda") -> Fp8Tensor:
    """An uninitialised FP8 block tensor [rows, cols] or [planes, rows, cols]."""
    *lead, rows, cols = shape
    kb, srows = -(-cols // BLOCK), -(-rows // tile)
    ld, lds = _up(cols, 16), _up(kb, 16)
    codes = torch.empty_strided((*lead, rows, cols), (rows * ld, ld, 1)[-len(shape):], dtype=torch.uint8, device=device)
    scales = torch.empty_strided((*lead, srows, kb), (srows * lds, lds, 1)[-len(shape):], dtype=torch.uint8,
                                 device=device)
    return Fp8Tensor(codes, scales)


def _new(rows: int, cols: int, tile: int, device) -> tuple[Fp8Tensor, _Fp8Struct]:
    """fp8_empty of a matrix, and its description."""
    kb, srows = -(-cols // BLOCK), rows if tile == 1 else -(-rows // tile)
    ld, lds = (cols + 15) & -16, (kb + 15) & -16
    codes = torch.empty_strided((rows, cols), (ld, 1), dtype=torch.uint8, device=device)
    scales = torch.empty_strided((srows, kb), (lds, 1), dtype=torch.uint8, device=device)
    return Fp8Tensor(codes, scales), _Fp8Struct(codes.data_ptr(), scales.data_ptr(), ld, lds, rows, cols, tile)


def _describe(t: Fp8Tensor, what: str, one_row_tile: int = 1) -> _Fp8Struct:
    """Checks an FP8 block tensor and describes it to the library. The scales
    of a single row have the same shape in both tilings: one_row_tile then."""
    codes, scales = t
    shape, sshape = codes.shape, scales.shape
    if len(shape) != 2 or len(sshape) != 2:
        raise ValueError(f"{what} must be 2-D uint8 codes and scales")
    return _described(codes, scales, shape, sshape, codes.stride(), scales.stride(), what, one_row_tile)


def _described(codes, scales, shape, sshape, strides, sstrides, what, one_row_tile=1) -> _Fp8Struct:
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise ValueError(f"{what} must be uint8 codes and scales")
    if not (codes.is_cuda and scales.is_cuda):
        raise ValueError(f"{what} must be CUDA tensors")
    rows, cols = shape
    srows, kb = sshape
    tile = BLOCK if srows != rows else one_row_tile if rows == 1 else 1
    if srows != -(-rows // tile) or kb != -(-cols // BLOCK):
        raise ValueError(f"{what}: scales {tuple(sshape)} do not fit codes {tuple(shape)}")
    if (cols > 1 and strides[1] != 1) or (kb > 1 and sstrides[1] != 1):
        raise ValueError(f"{what} must have contiguous columns")
    return _Fp8Struct(codes.data_ptr(), scales.data_ptr(), strides[0] if rows > 1 else _up(cols, 16),
                      sstrides[0] if srows > 1 else _up(kb, 4), rows, cols, tile)


def _matrix(t: torch.Tensor, what: str, shape=None, dtype=None) -> int:
    """Checks a plain matrix; its row stride (its width where it has one row)."""
    if not t.is_cuda or t.dtype not in DTYPES or t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D bf16, f16 or f32 CUDA tensor")
    size, strides = t.shape, t.stride()
    if shape is not None and size != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(size)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}")
    if size[1] > 1 and strides[1] != 1:
        raise ValueError(f"{what} must have contiguous columns")
    return strides[0] if size[0] > 1 else max(size[1], 1)


def _vector(t: torch.Tensor, what: str, n: int, dtype=None) -> None:
    if not t.is_cuda or t.dtype not in DTYPES or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor [{n}]")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}")


def _ref(s):
    return None if s is None else ctypes.byref(s)


def taco_fp8_quantize(x, rows: bool = True, cols: bool = False, tile: int = 1, out: Fp8Tensor | None = None,
                      out_t: Fp8Tensor | None = None, stream=None):
    """x [M, K] (bf16, f16, f32 or an Fp8Tensor) -> (its rows as an Fp8Tensor
    [M, K] or None, its transpose as one [K, M] or None), from one read."""
    if tile not in (1, BLOCK):
        raise ValueError(f"tile must be 1 or {BLOCK}")
    source = None
    if isinstance(x, Fp8Tensor):
        source = _describe(x, "x")
        M, K, dev = source.rows, source.cols, x.codes.device
    else:
        ld = _matrix(x, "x")
        (M, K), dev = x.shape, x.device
    a = b = None
    if not rows:
        out = None
    elif out is None:
        out, a = _new(M, K, tile, dev)
    else:
        a = _describe(out, "out", tile)
    if not cols:
        out_t = None
    elif out_t is None:
        out_t, b = _new(K, M, tile, dev)
    else:
        b = _describe(out_t, "out_t", tile)
    if source is not None:
        st = _lib().taco_fp8_requantize(ctypes.byref(source), _ref(a), _ref(b),
                                        _stream_of(stream, x.codes))
    else:
        st = _lib().taco_fp8_quantize(_ptr(x), DTYPES[x.dtype], M, K, ld, _ref(a), _ref(b),
                                      _stream_of(stream, x))
    _check(st, "taco_fp8_quantize")
    return out, out_t


def taco_rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                      eps: float = 1e-6, checkpoint: bool | Fp8Tensor = False, out: Fp8Tensor | None = None,
                      h: torch.Tensor | None = None, rstd: torch.Tensor | None = None,
                      stream=None) -> RmsNormOutput:
    """Root-mean-square norm of h = x + residual, [M, H], with the 8-bit output
    y = h * rstd * weight and, with ``checkpoint`` (True or a preallocated
    Fp8Tensor), h in 8 bits for the backward pass. Returns (y, h, rstd,
    checkpoint); h is x itself where there is no residual. ``h`` may be x or
    residual (in place)."""
    ldx = _matrix(x, "x")
    M, H = x.shape
    if not weight.is_cuda or weight.dtype not in DTYPES or weight.shape != (H,) or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous CUDA tensor [{H}]")
    ldr = ldh = 0
    if residual is not None:
        ldr = _matrix(residual, "residual", x.shape, x.dtype)
        if h is None:
            h, ldh = torch.empty((M, H), dtype=x.dtype, device=x.device), H
        else:
            ldh = _matrix(h, "h", x.shape, x.dtype)
    elif h is not None:
        raise ValueError("h is an output of the residual's addition: pass residual too")
    if out is None:
        out, y = _new(M, H, 1, x.device)
    else:
        y = _describe(out, "out")
    if rstd is None:
        rstd = torch.empty(M, dtype=torch.float32, device=x.device)
    else:
        _vector(rstd, "rstd", M, torch.float32)
    ck = c = None
    if checkpoint is True:
        ck, c = _new(M, H, 1, x.device)
    elif checkpoint:
        ck, c = checkpoint, _describe(checkpoint, "checkpoint")
    st = _lib().taco_rms_norm_fp8(_ptr(x), ldx, _ptr(residual), ldr, _ptr(weight), DTYPES[weight.dtype],
                                  DTYPES[x.dtype], M, H, float(eps), _ptr(h), ldh, _ptr(rstd), ctypes.byref(y),
                                  _ref(c), _stream_of(stream, x))
    _check(st, "taco_rms_norm_fp8")
    return RmsNormOutput(out, x if residual is None else h, rstd, ck)


def taco_rms_norm_fp8_backward(dy: torch.Tensor, saved, weight: torch.Tensor, rstd: torch.Tensor,
                               dh: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                               dw: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradients (dx [M, H], dw f32 [H]) of taco_rms_norm_fp8 from ``saved``, its
    8-bit checkpoint (an Fp8Tensor) or its h. ``dh`` is the gradient that h
    received elsewhere; ``dx``, the gradient of x and of residual alike, may be
    dy or dh (in place)."""
    lddy = _matrix(dy, "dy")
    M, H = dy.shape
    _vector(weight, "weight", H)
    _vector(rstd, "rstd", M, torch.float32)
    c, held, ldh = None, None, 0
    if isinstance(saved, Fp8Tensor):
        c = _describe(saved, "checkpoint")
    else:
        held, ldh = saved, _matrix(saved, "h", dy.shape, dy.dtype)
    lddh = 0 if dh is None else _matrix(dh, "dh", dy.shape, dy.dtype)
    if dx is None:
        dx, lddx = torch.empty((M, H), dtype=dy.dtype, device=dy.device), H
    else:
        lddx = _matrix(dx, "dx", dy.shape, dy.dtype)
    if dw is None:
        dw = torch.empty(H, dtype=torch.float32, device=dy.device)
    else:
        _vector(dw, "dw", H, torch.float32)
    if workspace is None:
        workspace = torch.empty(_lib().taco_rms_norm_workspace_bytes(M, H), dtype=torch.uint8, device=dy.device)
    st = _lib().taco_rms_norm_fp8_backward(
        _ptr(dy), lddy, _ref(c), _ptr(held), ldh, _ptr(weight), DTYPES[weight.dtype], _ptr(rstd), _ptr(dh), lddh,
        DTYPES[dy.dtype], M, H, _ptr(dx), lddx, _ptr(dw), _ptr(workspace), workspace.numel(), _stream_of(stream, dy))
    _check(st, "taco_rms_norm_fp8_backward")
    return dx, dw


def taco_swiglu_fp8(gate_up: torch.Tensor, checkpoint: bool | Fp8Tensor = False, out: Fp8Tensor | None = None,
                    stream=None):
    """y = silu(gate) * up in 8 bits, from gate_up [M, 2 F] (gate in the first F
    columns). With ``checkpoint`` (True or a preallocated Fp8Tensor [2, M, F])
    gate and up are kept in 8 bits. Returns (y, checkpoint or None)."""
    ld = _matrix(gate_up, "gate_up")
    M, F2 = gate_up.shape
    if F2 < 2 or F2 % 2:
        raise ValueError("gate_up must have an even number of columns")
    F = F2 // 2
    if out is None:
        out, y = _new(M, F, 1, gate_up.device)
    else:
        y = _describe(out, "out")
    ck = g = u = None
    if checkpoint:
        ck = fp8_empty(2, M, F, device=gate_up.device) if checkpoint is True else checkpoint
        g, u = _planes(ck)
    p = _ptr(gate_up)
    st = _lib().taco_swiglu_fp8(p, ld, p + F * gate_up.element_size(), ld, DTYPES[gate_up.dtype], M, F,
                                ctypes.byref(y), _ref(g), _ref(u), _stream_of(stream, gate_up))
    _check(st, "taco_swiglu_fp8")
    return out, ck


def _planes(ck: Fp8Tensor) -> tuple[_Fp8Struct, _Fp8Struct]:
    """Checks a gated activation's checkpoint and describes its two planes."""
    codes, scales = ck
    shape, sshape, strides, sstrides = codes.shape, scales.shape, codes.stride(), scales.stride()
    if len(shape) != 3 or len(sshape) != 3 or shape[0] != 2 or sshape[0] != 2:
        raise ValueError("the checkpoint of a gated activation is [2, M, F]: gate, up")
    g = _described(codes, scales, shape[1:], sshape[1:], strides[1:], sstrides[1:], "checkpoint")
    return g, _Fp8Struct(codes.data_ptr() + strides[0], scales.data_ptr() + sstrides[0], g.ld_codes, g.ld_scales,
                         g.rows, g.cols, g.tile_rows)


def taco_swiglu_fp8_backward(dy: torch.Tensor, checkpoint: Fp8Tensor, out: torch.Tensor | None = None,
                             stream=None) -> torch.Tensor:
    """Gradient [M, 2 F] of gate_up from taco_swiglu_fp8's checkpoint."""
    lddy = _matrix(dy, "dy")
    M, F = dy.shape
    g, u = _planes(checkpoint)
    if out is None:
        out, ldo = torch.empty((M, 2 * F), dtype=dy.dtype, device=dy.device), 2 * F
    else:
        ldo = _matrix(out, "out", (M, 2 * F), dy.dtype)
    p = _ptr(out)
    st = _lib().taco_swiglu_fp8_backward(_ptr(dy), lddy, ctypes.byref(g), ctypes.byref(u), DTYPES[dy.dtype], M, F,
                                         p, ldo, p + F * dy.element_size(), ldo, _stream_of(stream, dy))
    _check(st, "taco_swiglu_fp8_backward")
    return out


def taco_matmul_fp8(a: Fp8Tensor, b: Fp8Tensor, out: torch.Tensor | None = None,
                    out_dtype: torch.dtype = torch.bfloat16, add: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """a [M, K] times the transpose of b [N, K] (+ add) -> [M, N], summed in
    fp32 on the block-scaled tensor cores. ``add`` may be ``out`` (in place)."""
    x, w = _describe(a, "a"), _describe(b, "b")
    M, N = x.rows, w.rows
    if out is None:
        out, ldo = torch.empty((M, N), dtype=out_dtype, device=a.codes.device), max(N, 1)
    else:
        ldo = _matrix(out, "out", (M, N))
    ldadd = 0 if add is None else _matrix(add, "add", (M, N), out.dtype)
    st = _lib().taco_matmul_fp8(ctypes.byref(x), ctypes.byref(w), _ptr(add), ldadd, _ptr(out), ldo,
                                DTYPES[out.dtype], _stream_of(stream, out))
    _check(st, "taco_matmul_fp8")
    return out
