"""FP8 block tensors on the GPU: quantisation, RMS norm, gated activation and
their gradients against the 64-bit oracle.

Tolerances. Quantising an exact input has one right answer. Where the value is
computed first, a code has to be the right rounding of some value within
`delta` of the exact one: a row sum of fp32 terms is added in at most 64 serial
steps, 5 shuffles and 16 warps (85 roundings of 2^-24, 5.1e-6, halved by the
square root), so rstd and y stay within 1e-5; exp(-g) is off by at most 2 units
in the last place plus the rounding of its argument, 2e-7 |g|.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_util as U
from grads_taco_compress_gb300 import fp8 as F
from oracle import fp8_oracle as Q

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ quantise
SHAPES = [(1, 1), (1, 128), (3, 7), (2, 8), (5, 127), (4, 129), (130, 300), (257, 1600), (64, 4096), (1000, 136)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("which", ["rows", "cols", "both"])
@pytest.mark.parametrize("tile", [1, 128])
def test_quantize(R, C, dtype, which, tile):
    rng = np.random.default_rng([R, C, tile])
    x, x64 = U.values(rng, R, C, dtype)
    rows, cols = which != "cols", which != "rows"
    a, b = U.Guarded(R, C, tile), U.Guarded(C, R, tile)
    F.taco_fp8_quantize(x, rows=rows, cols=cols, tile=tile, out=a.t, out_t=b.t)
    got_a, got_b = a.get(), b.get()
    if rows:
        U.check_exact(got_a, x64, tile)
    else:
        assert (got_a[0] == U.GUARD).all()
    if cols:
        U.check_exact(got_b, x64.T, tile)
    else:
        assert (got_b[0] == U.GUARD).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (16, 8), (1, 1)])
def test_quantize_strided(dtype, pad, offset):
    rng = np.random.default_rng([pad, offset])
    x, x64 = U.values(rng, 70, 264, dtype)
    v = U.strided(x, pad, offset)
    a, b = U.Guarded(70, 264, extra=32), U.Guarded(264, 70, extra=16)
    F.taco_fp8_quantize(v, cols=True, out=a.t, out_t=b.t)
    U.check_exact(a.get(), x64)
    U.check_exact(b.get(), x64.T)


@pytest.mark.parametrize("R,C", [(1, 5), (130, 300), (500, 1600)])
@pytest.mark.parametrize("tile_in", [1, 128])
@pytest.mark.parametrize("tile", [1, 128])
def test_requantize(R, C, tile_in, tile):
    rng = np.random.default_rng([R, C, 7])
    x64 = U.values(rng, R, C, "f32")[1]
    codes, scales = Q.quantize(x64, tile_in)
    held = U.held(codes, scales, extra=16)
    if R == 1 and tile_in == 128:
        tile_in = 1
    a, b = U.Guarded(R, C, tile), U.Guarded(C, R, tile)
    F.taco_fp8_quantize(held, cols=True, tile=tile, out=a.t, out_t=b.t)
    d = Q.dequantize(codes, scales)
    U.check_exact(a.get(), d, tile)
    U.check_exact(b.get(), d.T, tile)


@pytest.mark.parametrize("cols", [False, True])
@pytest.mark.parametrize("tile", [1, 128])
def test_quantize_blocks_at_the_ends_of_the_range(cols, tile):
    big = float(torch.finfo(torch.float32).max)
    rows = [0.0, 1e-45, -1e-45, 2.0 ** -126, 2.0 ** -118, 448 * 2.0 ** -126, 449 * 2.0 ** -126, 1e-30, 448.0, 448.00003,
            447.99997, 449.0, 1e30, big, -big]
    rng = np.random.default_rng(0)
    x = np.zeros((128 * len(rows), 256), dtype=np.float32)
    for i, v in enumerate(rows):
        f = (rng.random((128, 256)) * 2 - 1).astype(np.float32)
        x[128 * i:128 * i + 128] = f * np.float32(v)
        x[128 * i:128 * i + 128, ::100] = np.float32(v)
    t = torch.from_numpy(x).cuda()
    a, b = U.Guarded(*x.shape, tile), U.Guarded(x.shape[1], x.shape[0], tile)
    F.taco_fp8_quantize(t, cols=cols, tile=tile, out=a.t, out_t=b.t)
    U.check_exact(a.get(), x.astype(np.float64), tile)
    if cols:
        U.check_exact(b.get(), x.T.astype(np.float64), tile)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_marks_blocks_that_are_not_finite(bad, dtype):
    rng = np.random.default_rng(3)
    x, x64 = U.values(rng, 200, 384, dtype, extremes=False)
    x[5, 130], x64[5, 130] = bad, bad
    x[199, 0], x64[199, 0] = bad, bad
    a, b = U.Guarded(200, 384), U.Guarded(384, 200)
    F.taco_fp8_quantize(x, cols=True, out=a.t, out_t=b.t)
    (ca, sa), (cb, sb) = a.get(), b.get()
    assert sorted(zip(*np.nonzero(sa == 255))) == [(5, 1), (199, 0)]
    assert sorted(zip(*np.nonzero(sb == 255))) == [(0, 1), (130, 0)]
    U.check_exact((ca, sa), np.where(np.isfinite(x64), x64, np.nan))
    assert torch.isnan(a.t.dequantize()[5, 128:256]).all()


def test_empty():
    x = torch.empty(0, 256, device="cuda")
    q, t = F.taco_fp8_quantize(x, cols=True)
    assert q.codes.shape == (0, 256) and t.codes.shape == (256, 0)
    w = torch.ones(256, device="cuda")
    r = F.taco_rms_norm_fp8(x, w, x.clone(), checkpoint=True)
    assert r.y.codes.shape == (0, 256)
    dw = torch.full((256,), 7.0, device="cuda")
    dx, dw = F.taco_rms_norm_fp8_backward(x, r.checkpoint, w, r.rstd, dw=dw)
    assert dx.shape == (0, 256) and (dw == 0).all()
    y, c = F.taco_swiglu_fp8(x, checkpoint=True)
    assert y.codes.shape == (0, 128)
    assert F.taco_swiglu_fp8_backward(torch.empty(0, 128, device="cuda"), c).shape == (0, 256)


# ---------------------------------------------------------------------- norm
NORM = [(1, 1), (1, 4096), (3, 7), (5, 128), (2, 1000), (37, 1600), (129, 3584), (4, 8192), (3, 12345), (2, 20000),
        (2, 32768), (700, 264)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,H", NORM)
@pytest.mark.parametrize("residual,checkpoint", [(False, False), (True, True), (True, False)])
def test_norm(M, H, dtype, residual, checkpoint):
    rng = np.random.default_rng([M, H])
    x, x64 = U.values(rng, M, H, dtype)
    w, w64 = U.values(rng, 1, H, dtype, 0.5, extremes=False)
    r, r64 = U.values(rng, M, H, dtype) if residual else (None, None)
    out, ck = U.Guarded(M, H), U.Guarded(M, H)
    got = F.taco_rms_norm_fp8(x, w[0], r, 1e-5, checkpoint=ck.t if checkpoint else False, out=out.t)
    h64 = x64
    if residual:
        # both addends are exact in fp32 and so is their rounding once
        h64 = (x.float() + r.float()).to(x.dtype).double().cpu().numpy()
        np.testing.assert_array_equal(got.h.double().cpu().numpy(), h64)
    y64, rstd64 = Q.rms_norm(h64, w64[0], np.float64(np.float32(1e-5)))
    np.testing.assert_allclose(got.rstd.double().cpu().numpy(), rstd64, rtol=5e-6)
    U.check_near(out.get(), y64, 1e-5)
    if checkpoint:
        U.check_exact(ck.get(), h64)
    else:
        assert got.checkpoint is None


def test_norm_strided_in_place_and_f32_weight():
    rng = np.random.default_rng(1)
    for pad, offset in [(8, 8), (3, 1)]:
        x, x64 = U.values(rng, 33, 520, "bf16")
        r, r64 = U.values(rng, 33, 520, "bf16")
        w, w64 = U.values(rng, 1, 520, "f32", extremes=False)
        xv, rv = U.strided(x, pad, offset), U.strided(r, 2 * pad, offset)
        h64 = (x.float() + r.float()).bfloat16().double().cpu().numpy()
        out = U.Guarded(33, 520)
        got = F.taco_rms_norm_fp8(xv, w[0], rv, 0.0, h=rv, out=out.t)
        assert got.h.data_ptr() == rv.data_ptr()
        np.testing.assert_array_equal(rv.double().cpu().numpy(), h64)
        U.check_near(out.get(), Q.rms_norm(h64, w64[0], 0.0)[0], 1e-5)


def test_norm_rows_of_zeros_and_of_no_finite_value():
    x = torch.randn(6, 384, device="cuda")
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    w = torch.ones(384, device="cuda")
    r = F.taco_rms_norm_fp8(x, w, eps=1e-6, checkpoint=True)
    s, c = r.y.scales.cpu(), r.checkpoint.scales.cpu()
    assert (r.y.codes[1] & 0x7F == 0).all() and (s[1] == 127).all()
    assert r.rstd[1].item() == pytest.approx(1e3, rel=1e-6)
    assert (s[2] == 255).all()                       # rstd is NaN: the whole row
    assert s[3, 1] == 255                            # infinity times zero
    assert c[2].tolist() == [255, c[2, 1], c[2, 2]] and c[2, 1] != 255
    assert c[3, 1] == 255 and c[3, 0] != 255
    assert (s[[0, 4, 5]] != 255).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,H", NORM + [(1500, 512)])
@pytest.mark.parametrize("saved,with_dh", [("checkpoint", True), ("checkpoint", False), ("h", True)])
def test_norm_backward(M, H, dtype, saved, with_dh):
    rng = np.random.default_rng([M, H, 5])
    h, h64 = U.values(rng, M, H, dtype)
    w, w64 = U.values(rng, 1, H, dtype, extremes=False)
    dy, dy64 = U.values(rng, M, H, dtype, 1e-2)
    dh, dh64 = U.values(rng, M, H, dtype, 1e-2) if with_dh else (None, None)
    rstd = torch.from_numpy((1 / np.sqrt((h64 ** 2).mean(axis=1) + 1e-3)).astype(np.float32)).cuda()
    if saved == "checkpoint":
        codes, scales = Q.quantize(h64)
        keep, h64 = U.held(codes, scales, extra=16), Q.dequantize(codes, scales)
    else:
        keep = h
    dx, dw = F.taco_rms_norm_fp8_backward(dy, keep, w[0], rstd, dh=dh)
    dx64, dw64, terms = Q.rms_norm_backward(dy64, h64, w64[0], rstd.double().cpu().numpy(), dh64)
    U.check_rounded(dx, dx64, 1e-5 * terms, dtype)
    # dw: at most ceil(M / CTAs) serial additions, then one per CTA
    bound = (M + 600) * 2.0 ** -24 * (np.abs(dy64 * h64 * rstd.double().cpu().numpy()[:, None])).sum(axis=0)
    assert (np.abs(dw.double().cpu().numpy() - dw64) <= bound + 1e-30).all()


def test_norm_backward_strided_in_place_and_repeatable():
    rng = np.random.default_rng(9)
    h, h64 = U.values(rng, 900, 1032, "bf16")
    w, w64 = U.values(rng, 1, 1032, "f32", extremes=False)
    dy, dy64 = U.values(rng, 900, 1032, "bf16", 1e-2)
    dh, dh64 = U.values(rng, 900, 1032, "bf16", 1e-2)
    rstd = torch.rsqrt(h.double().square().mean(dim=1) + 1e-3).float()
    want = F.taco_rms_norm_fp8_backward(dy, h, w[0], rstd, dh=dh)
    for pad, offset in [(8, 8), (5, 3)]:
        a, b = U.strided(dy, pad, offset), U.strided(dh, pad, offset)
        got = F.taco_rms_norm_fp8_backward(a, U.strided(h, pad, offset), w[0], rstd, dh=b, dx=b)
        assert got[0].data_ptr() == b.data_ptr()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for _ in range(20):
        again = F.taco_rms_norm_fp8_backward(dy, h, w[0], rstd, dh=dh)
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def _loss(x, r, w, eps, cy, ch):
    h = x + r
    y, _ = Q.rms_norm(h, w, eps)
    return (y * cy).sum() + (h * ch).sum()


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(4)
    M, H, eps = 3, 40, 1e-3
    x, r, cy, ch = (rng.standard_normal((M, H)).astype(np.float32).astype(np.float64) for _ in range(4))
    w = rng.standard_normal(H).astype(np.float32).astype(np.float64)
    h32 = torch.from_numpy((x + r).astype(np.float32)).cuda()
    _, rstd = Q.rms_norm(x + r, w, eps)

    def cuda(v):
        return torch.from_numpy(v.astype(np.float32)).cuda()

    dx, dw = F.taco_rms_norm_fp8_backward(cuda(cy), h32, cuda(w), cuda(rstd), dh=cuda(ch))
    e = 1e-5
    for i, j in [(0, 0), (1, 17), (2, 39), (0, 23)]:
        d = np.zeros((M, H))
        d[i, j] = e
        want = (_loss(x + d, r, w, eps, cy, ch) - _loss(x - d, r, w, eps, cy, ch)) / (2 * e)
        assert dx[i, j].item() == pytest.approx(want, rel=1e-5, abs=1e-5)
        dj = np.zeros(H)
        dj[j] = e
        want = (_loss(x, r, w + dj, eps, cy, ch) - _loss(x, r, w - dj, eps, cy, ch)) / (2 * e)
        assert dw[j].item() == pytest.approx(want, rel=1e-5, abs=1e-5)


# -------------------------------------------------------------------- swiglu
GATED = [(1, 1), (1, 4096), (3, 7), (5, 128), (257, 1000), (37, 1600), (2, 20000), (1100, 264)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N", GATED)
@pytest.mark.parametrize("checkpoint", [False, True])
def test_swiglu(M, N, dtype, checkpoint):
    rng = np.random.default_rng([M, N])
    x, x64 = U.values(rng, M, 2 * N, dtype, 2.0)
    out, g, u = U.Guarded(M, N), U.Guarded(M, N), U.Guarded(M, N)
    if checkpoint:
        y, ck = F.taco_swiglu_fp8(x, checkpoint=True, out=out.t)
        for i, part in enumerate((x64[:, :N], x64[:, N:])):
            U.check_exact((ck.codes[i].cpu().numpy(), ck.scales[i].cpu().numpy()), part)
    else:
        y, ck = F.taco_swiglu_fp8(x, out=out.t)
        assert ck is None
    gate, up = x64[:, :N], x64[:, N:]
    U.check_near(out.get(), Q.swiglu(gate, up), 2e-6 + 2e-7 * np.abs(gate))


@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 1), (16, 0)])
def test_swiglu_strided(pad, offset):
    rng = np.random.default_rng([pad, offset])
    x, x64 = U.values(rng, 50, 2 * 264, "bf16", 2.0)
    out = U.Guarded(50, 264, extra=16)
    F.taco_swiglu_fp8(U.strided(x, pad, offset), out=out.t)
    U.check_near(out.get(), Q.swiglu(x64[:, :264], x64[:, 264:]), 2e-6 + 2e-7 * np.abs(x64[:, :264]))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N", GATED)
def test_swiglu_backward(M, N, dtype):
    rng = np.random.default_rng([M, N, 8])
    g64, u64 = U.values(rng, M, N, "f32", 2.0)[1], U.values(rng, M, N, "f32", 2.0)[1]
    qg, qu = Q.quantize(g64), Q.quantize(u64)
    kb = qg[1].shape[1]
    ck = F.fp8_empty(2, M, N)
    for i, (c, s) in enumerate((qg, qu)):
        ck.codes[i].copy_(torch.from_numpy(c))
        ck.scales[i].copy_(torch.from_numpy(s))
    assert ck.scales.shape == (2, M, kb)
    dy, dy64 = U.values(rng, M, N, dtype, 1e-2)
    out = F.taco_swiglu_fp8_backward(dy, ck).double().cpu().numpy()
    gate, up = Q.dequantize(*qg), Q.dequantize(*qu)
    dg, du = Q.swiglu_backward(dy64, gate, up)
    # the derivative of silu is a difference near its zero: bound its terms
    s = Q.sigmoid(gate)
    tg = np.abs(dy64 * up) * s * (1 + np.abs(gate) * (1 - s))
    d = 4e-6 + 4e-7 * np.abs(gate)
    U.check_rounded(out[:, :N], dg, d * tg + 1e-36, dtype)
    U.check_rounded(out[:, N:], du, d * np.abs(du) + 1e-36, dtype)


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(2)
    N = 24
    # values that E4M3 holds exactly, so that the checkpoint is the input
    pick = Q.e4m3_decode(np.arange(0x28, 0x4A, dtype=np.uint8))
    gate, up = (rng.choice(pick, (2, N)) * rng.choice([-1, 1], (2, N)) for _ in range(2))
    dy = rng.standard_normal((2, N)).astype(np.float32).astype(np.float64)
    x = torch.from_numpy(np.concatenate([gate, up], axis=1).astype(np.float32)).cuda()
    _, ck = F.taco_swiglu_fp8(x, checkpoint=True)
    out = F.taco_swiglu_fp8_backward(torch.from_numpy(dy.astype(np.float32)).cuda(), ck).cpu().numpy()
    e = 1e-6
    for i, j in [(0, 0), (1, 5), (0, 23)]:
        d = np.zeros((2, N))
        d[i, j] = e
        want = ((Q.swiglu(gate + d, up) - Q.swiglu(gate - d, up)) * dy).sum() / (2 * e)
        assert out[i, j] == pytest.approx(want, rel=2e-5, abs=1e-6)
        want = ((Q.swiglu(gate, up + d) - Q.swiglu(gate, up - d)) * dy).sum() / (2 * e)
        assert out[i, N + j] == pytest.approx(want, rel=2e-5, abs=1e-6)


def test_swiglu_not_finite_and_saturated():
    x = torch.zeros(4, 256, device="cuda")
    x[0, :] = 1
    x[0, 3] = float("nan")                 # gate
    x[1, 128 + 5] = float("inf")           # up
    x[2, :128], x[2, 128:] = -200.0, 3.0   # silu underflows to zero
    x[3, :128], x[3, 128:] = 200.0, 3.0    # silu is the identity
    y, ck = F.taco_swiglu_fp8(x, checkpoint=True)
    assert y.scales[:, 0].tolist()[:2] == [255, 255]
    assert ck.scales[:, :2, 0].tolist() == [[255, 127], [ck.scales[1, 0, 0], 255]]
    assert (y.dequantize()[2].abs() < 1e-30).all()
    assert (y.dequantize()[3] == 600 * 0 + Q.dequantize(*Q.quantize(np.full((1, 128), 600.0)))[0, 0]).all()
    d = F.taco_swiglu_fp8_backward(torch.ones(4, 128, device="cuda"), ck)
    assert torch.isnan(d[0]).all() and torch.isfinite(d[2:]).all()


# ------------------------------------------------------------------- streams
def test_other_stream_and_graph():
    x = torch.randn(512, 1024, device="cuda").bfloat16()
    w = torch.ones(1024, device="cuda").bfloat16()
    want = F.taco_rms_norm_fp8(x, w, checkpoint=True)
    wq, _ = F.taco_fp8_quantize(torch.randn(256, 1024, device="cuda"), tile=128)
    c = F.taco_matmul_fp8(want.y, wq)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = F.taco_rms_norm_fp8(x, w, checkpoint=True, stream=s)
    c2 = F.taco_matmul_fp8(got.y, wq, stream=s)
    s.synchronize()
    assert torch.equal(got.y.codes, want.y.codes) and torch.equal(c2, c)
    out, ck = F.fp8_empty(512, 1024), F.fp8_empty(512, 1024)
    c3, rstd = torch.empty_like(c), torch.empty(512, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        F.taco_rms_norm_fp8(x, w, checkpoint=ck, out=out, rstd=rstd)
        F.taco_matmul_fp8(out, wq, out=c3)
    x.mul_(0.5)
    want = F.taco_rms_norm_fp8(x, w, checkpoint=True)
    c = F.taco_matmul_fp8(want.y, wq)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.codes, want.y.codes) and torch.equal(c3, c) and torch.equal(ck.codes, want.checkpoint.codes)
