"""The FP8 product with a layer's epilogue against the 64-bit oracle.

Tolerance: pre is off by what the product is (tests/test_gpu_fp8_matmul.py:
(K / 32 + 32) 2^-23 of the sum of its products' magnitudes) and the rounding of
the bias's addition. No activation is steeper than 1.13. Its own error is at
most 2^-20 |x|: the error function's formula is off by 1.5e-7 / 2, the logistic
and the exponentials by some 2^-22 of a factor that is at most 1. The residual's
addition rounds once more; then comes the rounding to the output's type.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_util as U
import grads_taco_compress_gb300 as taco
from grads_taco_compress_gb300 import binding as tb
from grads_taco_compress_gb300 import fp8 as F
from linear_util import ACTS, check_interval
from oracle import fp8_oracle as Q

pytestmark = pytest.mark.gpu


def operands(rng, M, N, K, tile=128, scale=1.0):
    """x and w on the GPU and in fp64; products of a few units."""
    x = rng.standard_normal((M, K)) * scale
    x[rng.random((M, K)) < 0.01] *= 20
    w = rng.standard_normal((N, K)) * K ** -0.5
    out = []
    for v, t in ((x, 1), (w, tile)):
        q = Q.quantize(v, t)
        out += [U.held(*q, extra=16 * int(rng.integers(0, 3))), Q.dequantize(*q)]
    return out


def reference(x64, w64, bias64, act, residual64, K):
    """(pre, its tolerance, y, its tolerance before the last rounding)"""
    pre = x64 @ w64.T + bias64
    dp = (K / 32 + 32) * 2.0 ** -23 * (np.abs(x64) @ np.abs(w64).T) + 2.0 ** -24 * np.abs(pre)
    y = Q.activate(pre, act)
    dy = 1.13 * dp + (2.0 ** -20 * (np.abs(pre) + dp) if act else 0)
    if residual64 is not None:
        y = y + residual64
        dy = dy + 2.0 ** -24 * np.abs(y)
    return pre, dp, y, dy


SHAPES = [(1, 1, 1), (1, 128, 128), (3, 5, 7), (16, 130, 129), (17, 200, 256), (64, 257, 640), (65, 100, 4200),
          (128, 128, 512), (129, 127, 640), (200, 300, 1000), (300, 1029, 384), (512, 1600, 400), (1000, 72, 16),
          (257, 513, 2600)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kind", ["fp8", "bf16", "f16", "f32"])
def test_linear(M, N, K, act, kind):
    rng = np.random.default_rng([M, N, K])
    x, x64, w, w64 = operands(rng, M, N, K, tile=(1, 128)[N % 2])
    btype = ("f32", "bf16", "f16")[(M + N) % 3]
    bias, bias64 = U.values(rng, 1, N, btype, extremes=False)
    kept = U.Guarded(M, N, extra=32)
    args = dict(bias=bias[0], activation=act, checkpoint=kept.t)
    if kind == "fp8":
        y = U.Guarded(M, N, extra=16)
        got, ck = taco.taco_linear_fp8(x, w, out=y.t, **args)
        pre, dp, want, dy = reference(x64, w64, bias64, act, None, K)
        check_interval(y.get(), want, dy)
    else:
        res, res64 = U.values(rng, M, N, kind, extremes=False)
        out = torch.full((M + 2, N), float("nan"), dtype=U.DTYPES[kind], device="cuda")
        got, ck = taco.taco_linear_fp8(x, w, residual=res, out=out[1:M + 1], **args)
        pre, dp, want, dy = reference(x64, w64, bias64, act, res64, K)
        assert torch.isnan(out[0]).all() and torch.isnan(out[M + 1]).all()
        U.check_rounded(out[1:M + 1], want, dy, kind)
    check_interval(kept.get(), pre, dp)
    assert ck.codes is kept.t.codes and ck.scales is kept.t.scales and tb.taco_get_fault() == 0


@pytest.mark.parametrize("M,N,K", [(7, 300, 640), (300, 260, 384), (130, 1029, 256), (700, 520, 1100)])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 1), (16, 8)])
def test_strides_and_in_place(M, N, K, kind, pad, offset):
    rng = np.random.default_rng([M, N, K, pad])
    x, x64, w, w64 = operands(rng, M, N, K)
    bias, bias64 = U.values(rng, 1, N, "f32", extremes=False)
    c, c64 = U.values(rng, M, N, kind, extremes=False)
    cv = U.strided(c, pad, offset)
    wide = torch.full((M, N + pad + offset), float("nan"), dtype=c.dtype, device="cuda")
    out = wide[:, offset:offset + N]
    y, kept = taco.taco_linear_fp8(x, w, bias[0], "gelu_tanh", residual=cv, out=out)
    assert y is out and kept is None
    _, _, want, dy = reference(x64, w64, bias64, "gelu_tanh", c64, K)
    U.check_rounded(out, want, dy, kind)
    assert torch.isnan(wide[:, :offset]).all() and torch.isnan(wide[:, offset + N:]).all()
    taco.taco_linear_fp8(x, w, bias[0], "gelu_tanh", residual=cv, out=cv)     # in place
    assert torch.equal(cv, out)


@pytest.mark.parametrize("M,N,K", [(5, 700, 640), (40, 256, 5000), (300, 513, 900), (2600, 5000, 256), (1100, 2100, 130)])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_nothing_added_is_the_product(M, N, K, kind):
    """The same sums as taco_matmul_fp8's, bit for bit; a pair takes several tiles."""
    rng = np.random.default_rng([M, N])
    x, _, w, _ = operands(rng, M, N, K)
    y, kept = taco.taco_linear_fp8(x, w, out_dtype=U.DTYPES[kind], checkpoint=True)
    assert torch.equal(y, taco.taco_matmul_fp8(x, w, out_dtype=U.DTYPES[kind]))
    q, _ = taco.taco_linear_fp8(x, w, out_dtype=torch.float8_e4m3fn)
    if kind == "f32" and K <= 1024:   # one segment: the sums that the 8-bit output has too
        e, _ = taco.taco_fp8_quantize(y)
        for t in (q, kept):
            assert torch.equal(t.codes, e.codes) and torch.equal(t.scales, e.scales)
    assert torch.equal(q.codes, kept.codes) or kind == "f32"


@pytest.mark.parametrize("M,N,K", [(2600, 5000, 256), (5000, 1100, 128), (1500, 300, 3000)])
def test_many_tiles(M, N, K):
    rng = np.random.default_rng([M, N])
    x, x64, w, w64 = operands(rng, M, N, K)
    bias, bias64 = U.values(rng, 1, N, "bf16", extremes=False)
    y, kept = taco.taco_linear_fp8(x, w, bias[0], "silu", out_dtype=torch.float8_e4m3fn, checkpoint=True)
    pre, dp, want, dy = reference(x64, w64, bias64, "silu", None, K)
    for t, v, d in ((y, want, dy), (kept, pre, dp)):
        check_interval((t.codes.cpu().numpy(), t.scales.cpu().numpy()), v, d)
    for kind in ("bf16", "f32"):
        y, _ = taco.taco_linear_fp8(x, w, bias[0], "silu", out_dtype=U.DTYPES[kind])
        U.check_rounded(y, want, dy, kind)
    assert tb.taco_get_fault() == 0


@pytest.mark.parametrize("M,N,K", [(300, 260, 640), (4, 512, 1024)])
@pytest.mark.parametrize("act", ACTS)
def test_what_is_not_finite_reaches_what_depends_on_it(M, N, K, act):
    rng = np.random.default_rng(1)
    x, _, w, _ = operands(rng, M, N, K)
    bias = torch.zeros(N, device="cuda")
    plain, _ = taco.taco_linear_fp8(x, w, bias, act, out_dtype=torch.float32)
    fine, keep = taco.taco_linear_fp8(x, w, bias, act, out_dtype=torch.float8_e4m3fn, checkpoint=True)
    x.scales[2, 1] = 255
    w.scales[1, 0] = 255        # rows 128 .. 255 of w
    bias[7] = float("nan")
    bias[256] = float("inf")
    got, _ = taco.taco_linear_fp8(x, w, bias, act, out_dtype=torch.float32)
    assert torch.isnan(got[2]).all() and torch.isnan(got[:, 128:256]).all() and torch.isnan(got[:, 7]).all()
    assert not torch.isfinite(got[:, 256]).any()
    rest = torch.ones_like(got, dtype=torch.bool)
    rest[2], rest[:, 128:256], rest[:, 7], rest[:, 256] = False, False, False, False
    assert torch.equal(got[rest], plain[rest])
    y, kept = taco.taco_linear_fp8(x, w, bias, act, out_dtype=torch.float8_e4m3fn, checkpoint=True)
    for t, was in ((y, fine), (kept, keep)):
        assert (t.scales[:, :3] == 255).all() and (t.scales[2] == 255).all()
        if N > 384:
            others = [r for r in range(M) if r != 2]
            assert torch.equal(t.scales[others, 3], was.scales[others, 3])
            assert torch.equal(t.codes[others, 384:], was.codes[others, 384:])


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_activations_at_their_ends(kind):
    """Pre-activations up to 2^60 through the bias alone."""
    x, _ = taco.taco_fp8_quantize(torch.zeros(2, 128, device="cuda"))
    w, _ = taco.taco_fp8_quantize(torch.zeros(512, 128, device="cuda"))
    b = torch.cat([torch.linspace(-40, 40, 256), torch.tensor([2.0 ** 60, -2.0 ** 60, 1e-30, -1e-30] * 64)]).cuda()
    for act in ACTS:
        want = Q.activate(b.double().cpu().numpy(), act)
        dtype = torch.float8_e4m3fn if kind == "fp8" else torch.float32
        y, _ = taco.taco_linear_fp8(x, w, b, act, out_dtype=dtype)
        if kind == "fp8":
            check_interval((y.codes.cpu().numpy(), y.scales.cpu().numpy()), np.stack([want] * 2),
                           np.stack([np.abs(b.double().cpu().numpy()) * 2.0 ** -20] * 2))
        else:
            got = y[0].double().cpu().numpy()
            assert np.isfinite(got).all()
            assert (np.abs(got - want) <= 2.0 ** -20 * np.abs(b.double().cpu().numpy())).all()


def test_zero_rows():
    x = F.fp8_empty(0, 256)
    w, _ = taco.taco_fp8_quantize(torch.randn(64, 256, device="cuda"))
    bias = torch.zeros(64, device="cuda")
    y, kept = taco.taco_linear_fp8(x, w, bias, "gelu", checkpoint=True)
    assert y.shape == (0, 64) and kept.codes.shape == (0, 64)
    assert taco.taco_linear_fp8(x, w, out_dtype=torch.float8_e4m3fn)[0].codes.shape == (0, 64)
    assert taco.taco_linear_fp8(w, x, bias[:0])[0].shape == (64, 0)


@pytest.mark.parametrize("M,N,K", [(4, 4096, 4096), (300, 260, 5000), (2048, 1600, 1600)])
def test_repeats_bit_for_bit_on_any_stream_and_in_a_graph(M, N, K):
    rng = np.random.default_rng(2)
    x, _, w, _ = operands(rng, M, N, K)
    bias = torch.randn(N, device="cuda").bfloat16()
    first, keep = taco.taco_linear_fp8(x, w, bias, "gelu", out_dtype=torch.float8_e4m3fn, checkpoint=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(10):
        y, kept = taco.taco_linear_fp8(x, w, bias, "gelu", out_dtype=torch.float8_e4m3fn, checkpoint=True,
                                       stream=side if k % 2 else None)
        torch.cuda.synchronize()
        for a, b in ((y, first), (kept, keep)):
            assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    out, ck = F.fp8_empty(M, N), F.fp8_empty(M, N)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        taco.taco_linear_fp8(x, w, bias, "gelu", out=out, checkpoint=ck)
    bias.zero_()
    graph.replay()
    want, wk = taco.taco_linear_fp8(x, w, bias, "gelu", out_dtype=torch.float8_e4m3fn, checkpoint=True)
    for a, b in ((out, want), (ck, wk)):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
