"""Plain 64-bit oracle of the AdamW step, of its rounding by thresholds, and of
the gradient norm. Test infrastructure, written from the formulas."""

from __future__ import annotations

import numpy as np

from .taco_oracle import e4m3_decode

#: mantissa bits and smallest normal exponent
FORMATS = {"bf16": (7, -126), "f16": (10, -14), "f32": (23, -126), "e4m3": (3, -6)}

LARGEST = {"bf16": (2 - 2.0 ** -7) * 2.0 ** 127, "f16": 65504.0}


def thresholds(n: int, t: int, start: int = 0) -> np.ndarray:
    """Thresholds in [0, 1) of elements start .. start + n - 1 at step t."""
    i = np.arange(start, start + n, dtype=np.uint64)
    w = (i * np.uint64(0xC13FA9A9) + np.uint64(t) * np.uint64(0x9E3779B1)) % np.uint64(1 << 32)
    return w.astype(np.float64) / 2.0 ** 32


def step_at(x, fmt: str) -> np.ndarray:
    """The format's step at |x|."""
    bits, low = FORMATS[fmt]
    _, e = np.frexp(np.abs(x))
    return 2.0 ** (np.maximum(np.where(x == 0, low, e - 1), low) - bits).astype(np.float64)


def by_threshold(x, u, fmt: str) -> np.ndarray:
    """x rounded towards zero, or up where the part cut off reaches 1 - u; infinite
    where that is beyond a 16-bit format's largest value."""
    s = step_at(x, fmt)
    q = np.floor(np.abs(x) / s + u) * s
    if fmt in LARGEST:
        q = np.where(q > LARGEST[fmt], np.inf, q)
    return np.copysign(q, x)


def root_codes(x, u) -> np.ndarray:
    """The same to E4M3 for a root, which keeps the smallest code where it is not zero."""
    q = by_threshold(x, u, "e4m3")
    return np.where((q == 0) & (x > 0), 2.0 ** -9, q)


def state_values(codes, scales) -> np.ndarray:
    """Codes [n] and scale bytes [ceil(n / 128)] -> values."""
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return e4m3_decode(codes) * np.repeat(s, 128)[: codes.size]


def adamw(x, g, m, v, t, lr, beta1, beta2, eps, decay):
    """(x, m, v, update, denominator) after step t."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    den = np.sqrt(v / (1 - beta2 ** t)) + eps
    update = lr / (1 - beta1 ** t) * m / den
    return x * (1 - lr * decay) - update, m, v, update, den
