"""The FP8 block-tensor entry points without a GPU: argument checks of the C ABI
and of the Python binding. Every call is rejected (or has nothing to do)
before any CUDA call, so the fake addresses are never dereferenced."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import grads_taco_compress_gb300 as taco
from grads_taco_compress_gb300 import binding as tb
from grads_taco_compress_gb300 import fp8 as F
from oracle import fp8_oracle as Q

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake-address host checks run on machines without a GPU")
OK, NULL, SHAPE, BLOCK, ALIGN, ARG, CUDA, WS = range(8)
A = 1 << 24          # fake device addresses, 16 MB apart
BF16, F16, F32 = range(3)


@pytest.fixture(scope="module")
def lib():
    if not tb.LIB_PATH.exists():
        from grads_taco_compress_gb300 import build_lib
        build_lib.build()
    return tb.library()


class Struct(ctypes.Structure):
    """taco_fp8_tensor of taco.h."""

    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("ld_codes", ctypes.c_int64),
                ("ld_scales", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("tile_rows", ctypes.c_int32)]


def fp8(i, rows, cols, tile=1, **kw):
    d = dict(codes=i * A, scales=i * A + (A >> 1), ld_codes=-(-cols // 16) * 16,
             ld_scales=-(-(-(-cols // 128)) // 4) * 4, rows=rows, cols=cols, tile_rows=tile)
    d.update(kw)
    return ctypes.byref(Struct(*(d[k] for k, _ in Struct._fields_)))


@no_gpu_only
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), ARG), (dict(M=-1), SHAPE), (dict(K=0), SHAPE), (dict(ld=255), SHAPE), (dict(x=None), NULL),
    (dict(x=A + 1), ALIGN), (dict(out=None), NULL), (dict(out=fp8(2, 4, 128)), SHAPE),
    (dict(out=fp8(2, 5, 256)), SHAPE),
    (dict(out=fp8(2, 4, 256, tile=64)), BLOCK), (dict(out=fp8(2, 4, 256, ld_codes=264)), SHAPE),
    (dict(out=fp8(2, 4, 256, ld_scales=1)), SHAPE), (dict(out=fp8(2, 4, 256, ld_codes=240)), SHAPE),
    (dict(out=fp8(2, 4, 256, codes=2 * A + 8)), ALIGN), (dict(out=fp8(2, 4, 256, scales=2 * A + 2)), ALIGN),
    (dict(out=fp8(2, 4, 256, codes=None)), NULL), (dict(out=fp8(2, 4, 256, codes=A + 512)), ARG),
    (dict(out=fp8(2, 4, 256, scales=2 * A + 16)), ARG),
    (dict(out_t=fp8(3, 4, 256)), SHAPE), (dict(out_t=fp8(3, 256, 4, tile=128)), BLOCK),
    (dict(out_t=fp8(2, 256, 4)), ARG),
])
def test_quantize_rejects(lib, kw, status):
    a = dict(x=A, dtype=BF16, M=4, K=256, ld=256, out=fp8(2, 4, 256), out_t=None)
    a.update(kw)
    assert lib.taco_fp8_quantize(a["x"], a["dtype"], a["M"], a["K"], a["ld"], a["out"], a["out_t"], None) == status


@no_gpu_only
def test_requantize_rejects(lib):
    assert lib.taco_fp8_requantize(None, fp8(2, 4, 256), None, None) == NULL
    assert lib.taco_fp8_requantize(fp8(1, 4, 256), None, None, None) == NULL
    assert lib.taco_fp8_requantize(fp8(1, 4, 256), fp8(1, 4, 256), None, None) == ARG
    assert lib.taco_fp8_requantize(fp8(1, 4, 256, tile=2), fp8(2, 4, 256), None, None) == BLOCK
    assert lib.taco_fp8_requantize(fp8(1, 4, 256), fp8(2, 256, 4), None, None) == SHAPE


def _norm(lib, **kw):
    a = dict(x=A, ldx=256, res=2 * A, ldr=256, w=3 * A, wd=F32, dtype=BF16, M=4, H=256, eps=1e-6, h=4 * A, ldh=256,
             rstd=5 * A, y=fp8(6, 4, 256), ck=fp8(7, 4, 256))
    a.update(kw)
    return lib.taco_rms_norm_fp8(a["x"], a["ldx"], a["res"], a["ldr"], a["w"], a["wd"], a["dtype"], a["M"], a["H"],
                                 a["eps"], a["h"], a["ldh"], a["rstd"], a["y"], a["ck"], None)


@no_gpu_only
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=-1), ARG), (dict(wd=7), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(eps=float("inf")), ARG), (dict(M=-1), SHAPE), (dict(H=0), SHAPE), (dict(H=32769), SHAPE),
    (dict(ldx=200), SHAPE), (dict(ldr=255), SHAPE), (dict(ldh=0), SHAPE), (dict(x=None), NULL), (dict(w=None), NULL),
    (dict(y=None), NULL), (dict(res=None), NULL), (dict(h=None), NULL), (dict(x=A + 1), ALIGN),
    (dict(w=3 * A + 2), ALIGN),
    (dict(rstd=5 * A + 2), ALIGN), (dict(y=fp8(6, 4, 256, tile=128)), BLOCK), (dict(y=fp8(6, 4, 384)), SHAPE),
    (dict(ck=fp8(6, 4, 256)), ARG), (dict(h=A + 64), ARG), (dict(h=A, ldh=512), ARG), (dict(rstd=4 * A), ARG),
    (dict(rstd=A), ARG), (dict(y=fp8(1, 4, 256)), ARG), (dict(ck=fp8(3, 4, 256)), ARG),
])
def test_norm_rejects(lib, kw, status):
    assert _norm(lib, **kw) == status


def _norm_backward(lib, **kw):
    a = dict(dy=A, lddy=256, ck=fp8(2, 4, 256), h=None, ldh=0, w=3 * A, wd=F32, rstd=4 * A, dh=5 * A, lddh=256,
             dtype=F16, M=4, H=256, dx=6 * A, lddx=256, dw=7 * A, ws=8 * A, wsb=4 * 256 * 4)
    a.update(kw)
    return lib.taco_rms_norm_fp8_backward(a["dy"], a["lddy"], a["ck"], a["h"], a["ldh"], a["w"], a["wd"], a["rstd"],
                                          a["dh"], a["lddh"], a["dtype"], a["M"], a["H"], a["dx"], a["lddx"], a["dw"],
                                          a["ws"], a["wsb"], None)


@no_gpu_only
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=9), ARG), (dict(M=-2), SHAPE), (dict(H=40000), SHAPE), (dict(ck=None), NULL),
    (dict(h=9 * A, ldh=256), NULL),
    (dict(w=None), NULL), (dict(rstd=None), NULL), (dict(dw=None), NULL), (dict(dx=None), NULL), (dict(dy=None), NULL),
    (dict(ws=None), WS), (dict(wsb=4 * 256 * 4 - 1), WS), (dict(ws=8 * A + 4), ALIGN), (dict(dx=6 * A + 1), ALIGN),
    (dict(dw=7 * A + 2), ALIGN), (dict(lddx=100), SHAPE), (dict(dx=A, lddx=512), ARG), (dict(dx=A + 32), ARG),
    (dict(dx=2 * A), ARG), (dict(dw=3 * A), ARG), (dict(ws=A), ARG), (dict(ws=7 * A), ARG),
    (dict(ck=None, h=9 * A, ldh=20), SHAPE),
])
def test_norm_backward_rejects(lib, kw, status):
    assert _norm_backward(lib, **kw) == status


@no_gpu_only
def test_norm_workspace_bytes(lib):
    assert lib.taco_rms_norm_workspace_bytes(4, 256) == 4 * 256 * 4
    assert lib.taco_rms_norm_workspace_bytes(0, 256) == 256 * 4
    assert lib.taco_rms_norm_workspace_bytes(1 << 20, 4096) == 512 * 4096 * 4
    assert lib.taco_rms_norm_workspace_bytes(-1, 256) == lib.taco_rms_norm_workspace_bytes(4, 40000) == 0


@no_gpu_only
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=4), ARG), (dict(F=0), SHAPE), (dict(M=-1), SHAPE), (dict(ldg=100), SHAPE), (dict(g=None), NULL),
    (dict(u=None), NULL), (dict(y=None), NULL), (dict(cu=None), NULL), (dict(g=A + 1), ALIGN),
    (dict(y=fp8(3, 4, 128)), SHAPE), (dict(cu=fp8(4, 4, 256)), ARG), (dict(y=fp8(1, 4, 256)), ARG),
    (dict(cg=fp8(4, 4, 256, tile=128)), BLOCK),
])
def test_swiglu_rejects(lib, kw, status):
    a = dict(g=A, ldg=512, u=A + 512, ldu=512, dtype=BF16, M=4, F=256, y=fp8(3, 4, 256), cg=fp8(4, 4, 256),
             cu=fp8(5, 4, 256))
    a.update(kw)
    assert lib.taco_swiglu_fp8(a["g"], a["ldg"], a["u"], a["ldu"], a["dtype"], a["M"], a["F"], a["y"], a["cg"], a["cu"],
                               None) == status


@no_gpu_only
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=4), ARG), (dict(F=0), SHAPE), (dict(cg=None), NULL), (dict(dy=None), NULL), (dict(dg=None), NULL),
    (dict(lddu=10), SHAPE), (dict(dg=A + 1), ALIGN), (dict(dg=6 * A + 64), ARG), (dict(dg=2 * A), ARG),
    (dict(dg=A, lddg=512), ARG), (dict(du=6 * A + 256), ARG),
])
def test_swiglu_backward_rejects(lib, kw, status):
    a = dict(dy=A, lddy=256, cg=fp8(2, 4, 256), cu=fp8(3, 4, 256), dtype=BF16, M=4, F=256, dg=6 * A, lddg=512,
             du=6 * A + 512, lddu=512)
    a.update(kw)
    assert lib.taco_swiglu_fp8_backward(a["dy"], a["lddy"], a["cg"], a["cu"], a["dtype"], a["M"], a["F"], a["dg"],
                                        a["lddg"], a["du"], a["lddu"], None) == status


@no_gpu_only
@pytest.mark.parametrize("kw,status", [
    (dict(a=None), NULL), (dict(b=None), NULL), (dict(dtype=5), ARG), (dict(b=fp8(2, 64, 512)), SHAPE),
    (dict(a=fp8(1, 4, 256, tile=3)), BLOCK), (dict(a=fp8(1, 4, 256, ld_codes=250)), SHAPE),
    (dict(a=fp8(1, 4, 256, codes=A + 4)), ALIGN), (dict(a=fp8(1, -1, 256)), SHAPE),
    (dict(a=fp8(1, 4, 0), b=fp8(2, 64, 0)), SHAPE), (dict(out=None), NULL), (dict(ldo=63), SHAPE),
    (dict(out=3 * A + 1), ALIGN), (dict(add=4 * A, ldadd=10), SHAPE), (dict(add=3 * A + 64, ldadd=64), ARG),
    (dict(out=A), ARG), (dict(out=2 * A + (A >> 1)), ARG),
])
def test_matmul_rejects(lib, kw, status):
    a = dict(a=fp8(1, 4, 256), b=fp8(2, 64, 256, tile=128), add=None, ldadd=0, out=3 * A, ldo=64, dtype=BF16)
    a.update(kw)
    assert lib.taco_matmul_fp8(a["a"], a["b"], a["add"], a["ldadd"], a["out"], a["ldo"], a["dtype"], None) == status


@no_gpu_only
def test_empty_calls_launch_nothing(lib):
    assert lib.taco_fp8_quantize(None, BF16, 0, 256, 256, fp8(2, 0, 256, codes=None, scales=None), None, None) == OK
    assert _norm(lib, M=0, x=None, res=None, h=None, rstd=None, y=fp8(6, 0, 256), ck=None) == OK
    assert lib.taco_matmul_fp8(fp8(1, 0, 256), fp8(2, 64, 256), None, 0, None, 64, F32, None) == OK


def test_binding_refuses_what_is_not_on_the_gpu():
    x = torch.zeros(4, 256)
    t = F.Fp8Tensor(torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    for call in (lambda: taco.taco_fp8_quantize(x), lambda: taco.taco_rms_norm_fp8(x, x[0]),
                 lambda: taco.taco_rms_norm_fp8_backward(x, t, x[0], x[:, 0]), lambda: taco.taco_swiglu_fp8(x),
                 lambda: taco.taco_swiglu_fp8_backward(x, t), lambda: taco.taco_matmul_fp8(t, t),
                 lambda: taco.taco_fp8_quantize(x, tile=64)):
        with pytest.raises(ValueError):
            call()


def test_binding_fails_loudly_without_its_module(monkeypatch, tmp_path, lib):
    monkeypatch.setattr(F, "BINDING_PATH", tmp_path / "missing.so")
    monkeypatch.setattr(F, "_BINDING", None)
    with pytest.raises(RuntimeError, match="not built"):
        taco.taco_fp8_quantize(torch.zeros(4, 256))


def test_padding_of_a_new_tensor():
    t = F.fp8_empty(5, 130, device="cpu")
    assert t.codes.shape == (5, 130) and t.codes.stride() == (144, 1)
    assert t.scales.shape == (5, 2) and t.scales.stride() == (16, 1)
    t = F.fp8_empty(2, 300, 256, device="cpu")
    assert t.codes.shape == (2, 300, 256) and t.scales.stride() == (300 * 16, 16, 1)
    t = F.fp8_empty(300, 256, tile=128, device="cpu")
    assert t.scales.shape == (3, 2)


# ----------------------------------------------------------------- the oracle
def test_oracle_scale_bytes():
    f = np.float64
    assert Q.scale_byte([0.0, 448.0, np.nextafter(f(448), 1e9), 1.75, 1.76, np.inf, np.nan, 1e-300]).tolist() == \
        [127, 127, 128, 119, 120, 255, 255, 1]


def test_oracle_quantises_to_the_nearest():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((6, 300)) * 10.0 ** rng.integers(-6, 6, (6, 1))
    codes, scales = Q.quantize(x)
    table = Q.e4m3_decode(np.arange(256, dtype=np.uint8))
    table = table[np.isfinite(table)]
    s = Q.spread(scales, *x.shape)
    best = np.abs(table[None, None, :] * s[..., None] - x[..., None]).min(axis=2)
    np.testing.assert_array_equal(np.abs(Q.dequantize(codes, scales) - x), best)
    assert (np.abs(x) <= 448 * s).all() and (Q.block_amax(x) > 224 * (2.0 ** (scales.astype(float) - 127))).all()


def test_oracle_gradients_against_differences():
    rng = np.random.default_rng(1)
    h, w, dy = rng.standard_normal((2, 9)), rng.standard_normal(9), rng.standard_normal((2, 9))
    rstd = Q.rms_norm(h, w, 1e-3)[1]
    dx, dw, _ = Q.rms_norm_backward(dy, h, w, rstd)
    e = 1e-6
    for i, j in [(0, 0), (1, 8)]:
        d = np.zeros_like(h)
        d[i, j] = e
        want = ((Q.rms_norm(h + d, w, 1e-3)[0] - Q.rms_norm(h - d, w, 1e-3)[0]) * dy).sum() / (2 * e)
        assert dx[i, j] == pytest.approx(want, rel=1e-6, abs=1e-8)
    g, u = rng.standard_normal((2, 9)), rng.standard_normal((2, 9))
    dg, du = Q.swiglu_backward(dy, g, u)
    np.testing.assert_allclose(dg, (Q.swiglu(g + e, u) - Q.swiglu(g - e, u)) * dy / (2 * e), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(du, (Q.swiglu(g, u + e) - Q.swiglu(g, u - e)) * dy / (2 * e), rtol=1e-6, atol=1e-8)
