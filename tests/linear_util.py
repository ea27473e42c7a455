"""Shared by the tests of the FP8 layer's epilogue and its gradient."""

from __future__ import annotations

import numpy as np

from oracle import fp8_oracle as Q

ACTS = [None, "gelu", "gelu_tanh", "silu", "relu"]


def check_interval(got, y, d, tile=1):
    """Codes and scales that are the right rounding of some value within the
    distance d (an array) of y."""
    codes, scales = got
    least = Q.block_amax(np.maximum(np.abs(y) - d, 0), tile)
    # a block that may be all zeros may have any scale up to the largest value's, and 1
    lo = np.where(least == 0, 1, Q.scale_byte(least))
    hi = Q.scale_byte(Q.block_amax(np.abs(y) + d, tile))
    assert (((scales >= lo) & (scales <= hi)) | ((least == 0) & (scales == 127))).all()
    s = Q.spread(scales, *y.shape)
    have = Q.e4m3_decode(codes)
    a, b = Q.e4m3_decode(Q.e4m3_encode((y - d) / s)), Q.e4m3_decode(Q.e4m3_encode((y + d) / s))
    assert ((have >= a) & (have <= b)).all()
