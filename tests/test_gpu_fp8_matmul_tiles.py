"""The FP8 product where a pair of CTAs takes several output tiles, against the
64-bit oracle: 256-wide tiles (bf16, f16) with their overlapping accumulators,
128-wide ones (f32) summed in segments, more than one band of row tiles, odd
and even numbers of blocks along K. Tolerances as in test_gpu_fp8_matmul."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_util as U
from grads_taco_compress_gb300 import binding as tb
from grads_taco_compress_gb300 import fp8 as F
from oracle.taco_oracle import e4m3_decode
from test_gpu_fp8_matmul import check, operand

pytestmark = pytest.mark.gpu


def guarded(M, N, dtype, pad, offset):
    """An output [M, N] inside a wider, taller matrix of NaN."""
    big = torch.full((M + 2, N + pad + offset), float("nan"), dtype=U.DTYPES[dtype], device="cuda")
    return big, big[1:M + 1, offset:offset + N]


def check_guard(big, out, M, N, offset):
    around = big.clone()
    around[1:M + 1, offset:offset + N] = float("nan")
    assert torch.isnan(around).all()


def check16(out, a64, b64, K, dtype, add64):
    """As ``check``, with the type's own rounding to infinity, in `add` too."""
    size = np.abs(a64) @ np.abs(b64).T + np.abs(add64)
    U.check_rounded(out, a64 @ b64.T + add64, (K / 32 + 32) * 2.0 ** -23 * size, dtype)


def scaled(rng, R, K, tile, dtype):
    t, v = operand(rng, R, K, tile)
    if dtype == "f16":   # keep the sums inside the type's range
        t, v = U.held(t.codes.cpu().numpy(), (t.scales - 14).cpu().numpy()), v * 2.0 ** -14
    return t, v


# 9 row tiles of 256 (more than a band of 8) by 11 or 22 column tiles of 256 over
# at most 76 pairs: up to 3 tiles a pair
@pytest.mark.parametrize("M,N,K", [(2100, 2600, 384), (2100, 5400, 1160), (2304, 2560, 128), (2100, 5400, 1700)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tiles", [(1, 128), (128, 1)])
def test_wide_tiles(M, N, K, dtype, tiles):
    rng = np.random.default_rng([M, N, K])
    a, a64 = scaled(rng, M, K, tiles[0], dtype)
    b, b64 = scaled(rng, N, K, tiles[1], dtype)
    big, out = guarded(M, N, dtype, 8, 0)
    F.taco_matmul_fp8(a, b, out=out)
    check(out, a64, b64, K, dtype)
    check_guard(big, out, M, N, 0)
    assert tb.taco_get_fault() == 0


@pytest.mark.parametrize("M,N,K", [(2100, 5399, 1160), (2500, 2601, 384)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (5, 3), (13, 8)])
def test_wide_tiles_add_and_strides(M, N, K, dtype, pad, offset):
    rng = np.random.default_rng([M, N, K, pad])
    a, a64 = scaled(rng, M, K, 1, dtype)
    b, b64 = scaled(rng, N, K, 1, dtype)
    c, c64 = U.values(rng, M, N, dtype, 100.0)
    cv = U.strided(c, pad, offset)
    big, out = guarded(M, N, dtype, pad, offset)
    F.taco_matmul_fp8(a, b, out=out, add=cv)
    check16(out, a64, b64, K, dtype, c64)
    check_guard(big, out, M, N, offset)
    F.taco_matmul_fp8(a, b, out=cv, add=cv)     # in place
    assert torch.equal(cv, out)
    assert tb.taco_get_fault() == 0


# 10 row tiles of 256 by 11 or 41 column tiles of 128; 1, 3 and 2 segments of 1024
@pytest.mark.parametrize("M,N,K", [(2500, 1300, 2100), (2500, 5200, 640), (2100, 5199, 2048)])
@pytest.mark.parametrize("pad,offset,add", [(0, 0, False), (0, 0, True), (4, 0, True), (3, 1, True), (3, 1, False)])
def test_f32_tiles(M, N, K, pad, offset, add):
    rng = np.random.default_rng([M, N, K, pad])
    a, a64 = operand(rng, M, K, 1)
    b, b64 = operand(rng, N, K, 1)
    big, out = guarded(M, N, "f32", pad, offset)
    if add:
        c, c64 = U.values(rng, M, N, "f32", 1e4)
        cv = U.strided(c, pad, offset)
        F.taco_matmul_fp8(a, b, out=out, add=cv)
        check(out, a64, b64, K, "f32", c64)
        F.taco_matmul_fp8(a, b, out=cv, add=cv)     # in place
        assert torch.equal(cv, out)
    else:
        F.taco_matmul_fp8(a, b, out=out)
        check(out, a64, b64, K, "f32")
    check_guard(big, out, M, N, offset)
    assert tb.taco_get_fault() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_tiles_repeat_bit_for_bit(dtype):
    rng = np.random.default_rng(4)
    a, _ = operand(rng, 2100, 1160, 1)
    b, _ = operand(rng, 5400, 1160, 128)
    first = F.taco_matmul_fp8(a, b, out_dtype=U.DTYPES[dtype])
    for _ in range(20):
        assert torch.equal(F.taco_matmul_fp8(a, b, out_dtype=U.DTYPES[dtype]), first)


def positive(gen, R, K, spread):
    """Positive codes of every bit pattern from 2^-6 up, block scales over `spread` binades; the values in fp64."""
    t = F.fp8_empty(R, K)
    t.codes.copy_(torch.randint(0x08, 0x7F, (R, K), generator=gen, device="cuda", dtype=torch.uint8))
    t.scales.copy_(torch.randint(127 - spread, 128, t.scales.shape, generator=gen, device="cuda", dtype=torch.uint8))
    table = torch.from_numpy(e4m3_decode(np.arange(256, dtype=np.uint8))).cuda()
    v = table[t.codes.long()].view(R, K // 128, 128) * torch.exp2(t.scales.double() - 127)[..., None]
    return t, v.view(R, K)


# pairs of CTAs (100 tiles, no split of K would fit beside them) and K split over a cluster of 8
@pytest.mark.parametrize("M,N,K", [(1280, 1280, 16384), (64, 256, 131072)])
@pytest.mark.parametrize("spread", [0, 10])
def test_long_sums_are_formed_in_segments(M, N, K, spread):
    """f32 sums of positive terms that use every bit: an MMA's 32 columns lose up
    to two units in the last place of the sum so far (the tensor cores cut, and
    do not round, in each of two steps of 16 columns), 64 in a segment of 1024
    columns; the additions of segments and splits lose half a unit each of a sum
    that grows evenly, a quarter of their number in all. One sum over 16384 columns loses 16 times what
    a segment does: 300 to 450 units in the mean on these values (measured on
    16-bit outputs, which are summed so)."""
    gen = torch.Generator(device="cuda").manual_seed(K)
    a, a64 = positive(gen, M, K, spread)
    b, b64 = positive(gen, N, K, spread)
    out = F.taco_matmul_fp8(a, b, out_dtype=torch.float32).double()
    want = a64 @ b64.t()
    additions = 16 + (8 if M <= 64 else 0)   # segments of a CTA, splits
    units = ((out - want).abs() / want).max().item() * 2.0 ** 23
    assert units <= 64 + additions / 4
    assert tb.taco_get_fault() == 0
