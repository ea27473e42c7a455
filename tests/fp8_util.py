"""Shared by the FP8 block-tensor tests: inputs of every kind, guarded outputs
and comparisons with the 64-bit oracle."""

from __future__ import annotations

import numpy as np
import torch

from grads_taco_compress_gb300 import fp8 as F
from oracle import fp8_oracle as Q

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
#: half a unit in the last place, relative
UNIT = {"bf16": 2.0 ** -9, "f16": 2.0 ** -12, "f32": 2.0 ** -25}
#: twice that: a rounding and what precedes it
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
#: half the smallest subnormal step
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}
GUARD = 0xA5


def values(rng, R, C, dtype, scale=1.0, extremes=True):
    """[R, C] on the GPU: heavy tails, zeros, whole zero blocks, magnitudes over
    many binades; exact in dtype. Returns (tensor, the same in fp64)."""
    x = rng.standard_normal((R, C)) * scale
    x[rng.random((R, C)) < 0.02] *= 50
    x[rng.random((R, C)) < 0.05] = 0
    if extremes and R and C:
        for r in range(0, R, 5):
            x[r] *= 2.0 ** rng.integers(-12, 8)
        x[rng.integers(0, R), : min(C, 128)] = 0.0
    t = torch.from_numpy(x.astype(np.float32)).to(DTYPES[dtype])
    return t.cuda(), t.double().numpy()


def strided(t, pad, offset=0):
    """The same matrix inside a wider one: `pad` more elements per row, starting `offset` in."""
    R, C = t.shape
    big = torch.full((R, C + pad + offset), float("nan"), dtype=t.dtype, device=t.device)
    v = big[:, offset:offset + C]
    v.copy_(t)
    return v


class Guarded:
    """An Fp8Tensor whose surroundings hold a pattern that must survive."""

    def __init__(self, rows, cols, tile=1, extra=0):
        kb, srows = -(-cols // 128), -(-rows // tile)
        self.c = torch.full((rows + 2, -(-cols // 16) * 16 + extra), GUARD, dtype=torch.uint8, device="cuda")
        self.s = torch.full((srows + 2, -(-kb // 4) * 4 + extra), GUARD, dtype=torch.uint8, device="cuda")
        self.rows, self.cols, self.srows, self.kb = rows, cols, srows, kb
        self.t = F.Fp8Tensor(self.c[1:rows + 1, :cols], self.s[1:srows + 1, :kb])

    def get(self):
        c, s = self.c.cpu().numpy().copy(), self.s.cpu().numpy().copy()
        codes, scales = c[1:self.rows + 1, :self.cols].copy(), s[1:self.srows + 1, :self.kb].copy()
        c[1:self.rows + 1, :self.cols] = GUARD
        s[1:self.srows + 1, :self.kb] = GUARD
        assert (c == GUARD).all() and (s == GUARD).all(), "written outside the tensor"
        return codes, scales


def held(codes, scales, extra=0):
    """numpy codes and scales as an Fp8Tensor, its padding filled with NaN codes and NaN scales."""
    kb = scales.shape[1]
    c = torch.full((codes.shape[0], -(-codes.shape[1] // 16) * 16 + extra), 0x7F, dtype=torch.uint8, device="cuda")
    s = torch.full((scales.shape[0], -(-kb // 4) * 4 + extra), 255, dtype=torch.uint8, device="cuda")
    c[:, :codes.shape[1]] = torch.from_numpy(codes)
    s[:, :kb] = torch.from_numpy(scales)
    return F.Fp8Tensor(c[:, :codes.shape[1]], s[:, :kb])


def check_exact(got, x64, tile=1):
    """Codes and scales equal to the oracle's for inputs that are exact."""
    codes, scales = got
    oc, os_ = Q.quantize(x64, tile)
    np.testing.assert_array_equal(scales, os_)
    fine = np.isfinite(Q.spread(os_, *x64.shape))
    g, w = Q.e4m3_decode(codes), Q.e4m3_decode(oc)
    np.testing.assert_array_equal(g[fine], w[fine])


def check_near(got, y64, delta):
    """Codes and scales that are the right rounding of some value within the
    relative `delta` (scalar or per element) of y64."""
    codes, scales = got
    d = np.broadcast_to(np.asarray(delta, dtype=np.float64), y64.shape)
    lo_s = Q.scale_byte(Q.block_amax(np.abs(y64) * (1 - d)))
    hi_s = Q.scale_byte(Q.block_amax(np.abs(y64) * (1 + d)))
    finite = hi_s != 255
    assert (scales[~finite] == 255).all()
    assert ((scales >= lo_s) & (scales <= hi_s))[finite].all()
    s = Q.spread(scales, *y64.shape)
    ok = np.isfinite(s)
    with np.errstate(invalid="ignore"):
        mag = Q.e4m3_decode(codes)
        a, b = Q.e4m3_decode(Q.e4m3_encode(y64 * (1 - d) / s)), Q.e4m3_decode(Q.e4m3_encode(y64 * (1 + d) / s))
    lo, hi = np.minimum(a, b), np.maximum(a, b)
    assert ((mag >= lo) & (mag <= hi))[ok].all()


def check_rounded(out, want, slack, dtype):
    """`out` is `want`, off by at most `slack` before it was rounded to dtype
    (a value beyond the type's largest rounds to infinity)."""
    got = out.double().cpu().numpy() if isinstance(out, torch.Tensor) else out
    top = torch.finfo(DTYPES[dtype]).max * (1 + UNIT[dtype])
    tol = ROUND[dtype] * np.abs(want) + slack + TINY[dtype]
    inf = np.isinf(got)
    assert (np.abs(want)[inf] + tol[inf] >= top).all() and (np.sign(got) == np.sign(want))[inf].all()
    assert (np.abs(want)[~inf] - tol[~inf] <= top).all()
    err = np.abs(got - np.where(inf, 0, want))[~inf]
    assert (err <= tol[~inf]).all(), (err / tol[~inf]).max()
