"""Plain 64-bit oracle of the FP8 block tensors and the layer operators on them.

Test infrastructure, written from the formulas: E4M3 codes with one
power-of-two scale (E8M0 byte b, 2^(b - 127), 255 = NaN) per row and 128
columns or per 128 x 128 tile; quantisation, the root-mean-square norm, the
gated activation, their gradients, and the matrix product.
"""

from __future__ import annotations

import math

import numpy as np

from .taco_oracle import e4m3_decode, e4m3_encode

BLOCK = 128
NAN_BYTE = 255


def scale_byte(amax) -> np.ndarray:
    """Scale bytes of blocks with largest magnitudes `amax` (NaN or infinite: 255)."""
    amax = np.asarray(amax, dtype=np.float64)
    out = np.full(amax.shape, NAN_BYTE, dtype=np.uint8)
    for i in np.ndindex(amax.shape):
        a = amax[i]
        if not np.isfinite(a):
            continue
        if a == 0:
            out[i] = 127
            continue
        e = -126
        while 448.0 * 2.0 ** e < a:
            e += 1
        out[i] = e + 127
    return out


def block_amax(x, tile: int = 1) -> np.ndarray:
    """Largest magnitudes [ceil(R / tile), ceil(C / 128)]; NaN where a block holds one."""
    R, C = x.shape
    rb, cb = -(-R // tile), -(-C // BLOCK)
    out = np.zeros((rb, cb))
    for r in range(rb):
        rows = np.abs(x[r * tile:(r + 1) * tile])
        for c in range(cb):
            out[r, c] = rows[:, c * BLOCK:(c + 1) * BLOCK].max()
    return out


def spread(scales, R: int, C: int) -> np.ndarray:
    """Scale bytes -> the scale of every element [R, C]."""
    s = np.where(scales == NAN_BYTE, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    tile = 1 if scales.shape[0] == R else BLOCK
    return np.repeat(np.repeat(s, tile, axis=0)[:R], BLOCK, axis=1)[:, :C]


def quantize(x, tile: int = 1):
    """(codes u8 [R, C], scale bytes) of x."""
    x = np.asarray(x, dtype=np.float64)
    scales = scale_byte(block_amax(x, tile))
    with np.errstate(invalid="ignore"):
        codes = e4m3_encode(x / spread(scales, *x.shape))
    return codes, scales


def dequantize(codes, scales) -> np.ndarray:
    return e4m3_decode(codes) * spread(scales, *codes.shape)


def rms_norm(h, weight, eps):
    """(y, rstd) of rows h."""
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * rstd[:, None] * weight, rstd


def rms_norm_backward(dy, h, weight, rstd, dh=None):
    """(dx, dw, scale of dx's terms): the last bounds what rounding can move."""
    xh = h * rstd[:, None]
    g = dy * weight
    c = np.mean(g * xh, axis=1, keepdims=True)
    dx = rstd[:, None] * (g - xh * c)
    terms = rstd[:, None] * (np.abs(g) + np.abs(xh) * np.mean(np.abs(g * xh), axis=1, keepdims=True))
    if dh is not None:
        dx, terms = dx + dh, terms + np.abs(dh)
    return dx, (dy * xh).sum(axis=0), terms


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(gate, up):
    return gate * sigmoid(gate) * up


def swiglu_backward(dy, gate, up):
    s = sigmoid(gate)
    return dy * up * s * (1 + gate * (1 - s)), dy * gate * s


_erfc = np.vectorize(math.erfc, otypes=[np.float64])
GELU_C, GELU_A = math.sqrt(2 / math.pi), 0.044715


def activate(x, kind):
    """The activation `kind` (None: none) of x."""
    if kind == "gelu":
        return x * 0.5 * _erfc(-x / math.sqrt(2))
    if kind == "gelu_tanh":
        return 0.5 * x * (1 + np.tanh(GELU_C * (x + GELU_A * x ** 3)))
    if kind == "silu":
        return x * sigmoid(x)
    return np.where(x < 0, 0.0, x) if kind == "relu" else x


def activation_slope(x, kind):
    """Its derivative (0 at 0 for relu)."""
    if kind == "gelu":
        return 0.5 * _erfc(-x / math.sqrt(2)) + x * np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        t = np.tanh(GELU_C * (x + GELU_A * x ** 3))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * GELU_C * (1 + 3 * GELU_A * x * x)
    if kind == "silu":
        s = sigmoid(x)
        return s + x * s * (1 - s)
    return (x > 0).astype(np.float64) if kind == "relu" else np.ones_like(x)
