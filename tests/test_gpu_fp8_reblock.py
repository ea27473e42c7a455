"""The transpose of FP8 codes into new blocks: exact, whatever the scales of the
rows that meet in a block and whatever the codes. The kernel works in fp16
where the rows' scales lie within 14 binades, no NaN is there and no column's
largest value lies 2^15 below the tile's range, and in fp32 otherwise: the
cases lie on both sides of each limit and at the ends of the scales."""

from __future__ import annotations

import numpy as np
import pytest

import fp8_util as U
from grads_taco_compress_gb300 import fp8 as F
from oracle import fp8_oracle as Q

pytestmark = pytest.mark.gpu

SHAPES = [(1, 5), (3, 17), (128, 128), (130, 300), (257, 1600)]
RANGES = [(127, 127), (110, 123), (110, 124), (110, 125), (100, 140), (0, 3), (0, 14), (0, 15), (1, 1), (5, 60),
          (226, 240), (227, 241), (240, 246), (1, 246)]


def blocks(rng, R, C, low, high):
    """Any codes but NaN, and scale bytes within [low, high] that reach both."""
    codes = rng.integers(0, 256, (R, C)).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x7E
    scales = rng.integers(low, high + 1, (R, -(-C // 128))).astype(np.uint8)
    scales[0], scales[-1] = high, low
    return codes, scales


def check(codes, scales):
    R, C = codes.shape
    b = U.Guarded(C, R, 1)
    F.taco_fp8_quantize(U.held(codes, scales, extra=16), rows=False, cols=True, out_t=b.t)
    U.check_exact(b.get(), Q.dequantize(codes, scales).T)


@pytest.mark.parametrize("low,high", RANGES)
@pytest.mark.parametrize("R,C", SHAPES)
def test_scales(R, C, low, high):
    check(*blocks(np.random.default_rng([R, C, low, high]), R, C, low, high))


@pytest.mark.parametrize("low,high", [(127, 127), (113, 127), (100, 140)])
def test_tiles(low, high):
    rng = np.random.default_rng([low, high])
    codes, _ = blocks(rng, 300, 500, low, high)
    check(codes, rng.integers(low, high + 1, (3, 4)).astype(np.uint8))


@pytest.mark.parametrize("low,high", [(127, 127), (113, 127), (112, 127), (0, 14), (226, 240)])
@pytest.mark.parametrize("kind", ["subnormal", "smallest", "zero columns", "zero rows", "zeros", "top row"])
def test_codes(kind, low, high):
    rng = np.random.default_rng([low, high])
    R, C = 257, 300
    codes, scales = blocks(rng, R, C, low, high)
    if kind == "subnormal":            # columns that need large factors
        codes &= 0x87
    elif kind == "smallest":           # one binade at a time, down to the smallest code alone
        for c in range(C):
            codes[:, c] = np.where(rng.random(R) < 0.5, c % 120, 0)
    elif kind == "zero columns":       # of both signs
        codes[:, ::3] &= 0x80
    elif kind == "zero rows":          # whose scales say nothing
        codes[::2] &= 0x80
        scales[::2] = rng.integers(0, 255, scales[::2].shape)
    elif kind == "zeros":
        codes &= 0x80
    elif kind == "top row":            # one row far above the others
        scales[5] = min(high + 6, 246)
    check(codes, scales)


@pytest.mark.parametrize("where", ["code", "scale", "scale of zeros"])
def test_nan_reaches_its_columns_alone(where):
    codes, scales = blocks(np.random.default_rng(1), 300, 200, 120, 128)
    if where == "code":
        codes[140, 7] = 0xFF
        want = {(7, 1)}
    else:
        scales[140, 0] = 255
        if where == "scale of zeros":
            codes[140, :128] = 0
        want = {(c, 1) for c in range(128)}
    b = U.Guarded(200, 300, 1)
    F.taco_fp8_quantize(U.held(codes, scales, extra=16), rows=False, cols=True, out_t=b.t)
    got = b.get()
    assert set(zip(*np.nonzero(got[1] == 255))) == want
    U.check_exact(got, Q.dequantize(codes, scales).T)
