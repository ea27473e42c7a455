"""The FP8 block-scaled matrix product against the 64-bit oracle.

Tolerance: every product of two codes is exact. The tensor cores add 32 of
them at a time into fp32, each addition off by at most one unit in the last
place of the terms it aligns, so an element is off by at most
(K / 32 + 32) 2^-23 of the sum of its products' magnitudes, and by the one
rounding to the output's type.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_util as U
from grads_taco_compress_gb300 import fp8 as F
from grads_taco_compress_gb300 import binding as tb
from oracle import fp8_oracle as Q

pytestmark = pytest.mark.gpu


def operand(rng, R, K, tile):
    """Random codes of every finite value and scales over many binades, on the GPU and in fp64."""
    codes = rng.integers(0, 127, (R, K)).astype(np.uint8) | (rng.integers(0, 2, (R, K)) << 7).astype(np.uint8)
    scales = rng.integers(117, 137, (-(-R // tile), -(-K // 128))).astype(np.uint8)
    return U.held(codes, scales, extra=int(rng.integers(0, 3)) * 16), Q.dequantize(codes, scales)


def check(out, a64, b64, K, dtype, add64=None):
    want = a64 @ b64.T
    size = np.abs(a64) @ np.abs(b64).T
    if add64 is not None:
        want, size = want + add64, size + np.abs(add64)
    bound = U.ROUND[dtype] * np.abs(want) + (K / 32 + 32) * 2.0 ** -23 * size + U.TINY[dtype]
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.isfinite(out.double().cpu().numpy()).all()
    assert (err <= bound).all(), (err / bound).max()


SHAPES = [(1, 1, 1), (1, 128, 128), (3, 5, 7), (16, 130, 129), (128, 128, 512), (129, 127, 640), (200, 300, 1000),
          (33, 1600, 1600), (512, 1024, 2100), (8, 4096, 4096), (1000, 72, 16), (257, 513, 12800), (64, 257, 8190),
          (300, 8, 260), (5, 9000, 384)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tiles", [(1, 128), (1, 1), (128, 128), (128, 1)])
def test_matmul(M, N, K, dtype, tiles):
    rng = np.random.default_rng([M, N, K])
    a, a64 = operand(rng, M, K, tiles[0])
    b, b64 = operand(rng, N, K, tiles[1])
    if dtype == "f16":   # keep the sums inside the type's range
        a = F.Fp8Tensor(a.codes, a.scales - 14)
        b = F.Fp8Tensor(b.codes, b.scales - 14)
        a64, b64 = a64 * 2.0 ** -14, b64 * 2.0 ** -14
        a, b = [U.held(t.codes.cpu().numpy(), t.scales.cpu().numpy()) for t in (a, b)]
    out = torch.full((M + 2, N), float("nan"), dtype=U.DTYPES[dtype], device="cuda")
    F.taco_matmul_fp8(a, b, out=out[1:M + 1])
    assert torch.isnan(out[0]).all() and torch.isnan(out[M + 1]).all()
    check(out[1:M + 1], a64, b64, K, dtype)
    assert tb.taco_get_fault() == 0


@pytest.mark.parametrize("M,N,K", [(7, 300, 640), (300, 260, 384), (130, 1029, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 1), (16, 8)])
def test_matmul_add_and_strides(M, N, K, dtype, pad, offset):
    rng = np.random.default_rng([M, N, K, pad])
    a, a64 = operand(rng, M, K, 1)
    b, b64 = operand(rng, N, K, 1)
    c, c64 = U.values(rng, M, N, dtype, 1e4)
    cv = U.strided(c, pad, offset)
    wide = torch.full((M, N + pad + offset), float("nan"), dtype=c.dtype, device="cuda")
    out = wide[:, offset:offset + N]
    F.taco_matmul_fp8(a, b, out=out, add=cv)
    check(out, a64, b64, K, dtype, c64)
    assert torch.isnan(wide[:, :offset]).all() and torch.isnan(wide[:, offset + N:]).all()
    F.taco_matmul_fp8(a, b, out=cv, add=cv)     # in place
    assert torch.equal(cv, out)


@pytest.mark.parametrize("M,N,K", [(300, 260, 640), (4, 512, 1024)])
def test_matmul_carries_blocks_that_are_not_finite(M, N, K):
    rng = np.random.default_rng(1)
    a, a64 = operand(rng, M, K, 1)
    b, b64 = operand(rng, N, K, 1)
    want = F.taco_matmul_fp8(a, b, out_dtype=torch.float32)
    a.scales[2, 1] = 255
    b.scales[200, 0] = 255
    got = F.taco_matmul_fp8(a, b, out_dtype=torch.float32)
    assert torch.isnan(got[2]).all() and torch.isnan(got[:, 200]).all()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[2], keep[:, 200] = False, False
    assert torch.equal(got[keep], want[keep])


def test_matmul_zero_rows():
    a = F.fp8_empty(0, 256)
    b, _ = F.taco_fp8_quantize(torch.randn(64, 256, device="cuda"))
    assert F.taco_matmul_fp8(a, b).shape == (0, 64)
    assert F.taco_matmul_fp8(b, a).shape == (64, 0)


@pytest.mark.parametrize("M,N,K", [(4, 4096, 4096), (300, 260, 5000), (2048, 1600, 1600)])
def test_matmul_repeats_bit_for_bit(M, N, K):
    rng = np.random.default_rng(2)
    a, _ = operand(rng, M, K, 1)
    b, _ = operand(rng, N, K, 128)
    first = F.taco_matmul_fp8(a, b, out_dtype=torch.float32)
    for _ in range(20):
        assert torch.equal(F.taco_matmul_fp8(a, b, out_dtype=torch.float32), first)


@pytest.mark.parametrize("K", [4096, 16384])
def test_matmul_long_sums_keep_32_bits(K):
    """Sums of positive products, where every rounding toward zero adds up."""
    rng = np.random.default_rng(K)
    a64 = rng.random((256, K)) + 0.5
    b64 = rng.random((256, K)) + 0.5
    qa, qb = Q.quantize(a64), Q.quantize(b64)
    out = F.taco_matmul_fp8(U.held(*qa), U.held(*qb), out_dtype=torch.float32).double().cpu().numpy()
    want = Q.dequantize(*qa) @ Q.dequantize(*qb).T
    assert (np.abs(out - want) <= (K / 32 + 32) * 2.0 ** -23 * want).all()
