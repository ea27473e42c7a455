"""The gradient at a layer's product against the 64-bit oracle.

Tolerance: a slope is a sum of a few factors of at most 1.2, each to some 2^-21
of itself (reciprocal and exponential to 2^-22, the error function's formula to
1.5e-7 / 2, the exponent's rounding), 2^-19 in all; d rounds once more. The
bias's gradient adds 4 rows a thread, 32 threads' and then every eighth
tile of 128 rows, 8 of those: less than 26 + M / 1024 roundings of at most 2^-24 of the
magnitudes' sum.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_util as U
import grads_taco_compress_gb300 as taco
from grads_taco_compress_gb300 import fp8 as F
from linear_util import ACTS, check_interval
from oracle import fp8_oracle as Q

pytestmark = pytest.mark.gpu
SLOPE = 2.0 ** -19


def inputs(rng, M, N, dtype, act):
    dy, dy64 = U.values(rng, M, N, dtype, 1e-2)
    if act is None:
        return dy, dy64, None, None
    pre = rng.standard_normal((M, N)) * 2
    pre[rng.random((M, N)) < 0.02] *= 30
    pre[rng.random((M, N)) < 0.02] = 0
    q = Q.quantize(pre)
    return dy, dy64, U.held(*q, extra=16), Q.dequantize(*q)


def reference(dy64, pre64, act):
    slope = Q.activation_slope(pre64, act) if act else 1.0
    d = dy64 * slope
    e = (SLOPE * np.abs(dy64) if act else 0) + (2.0 ** -24 * np.abs(d) if act else np.zeros_like(d))
    M = d.shape[0]
    de = e.sum(axis=0) + (26 + M / 1024) * 2.0 ** -24 * (np.abs(d) + e).sum(axis=0)
    return d, e, d.sum(axis=0), de


def check(got, dy64, pre64, act):
    """got: (codes, scales) of rows and of the transpose, and the sums; None for what there is not."""
    d, e, db, de = reference(dy64, pre64, act)
    if got[0] is not None:
        check_interval(got[0], d, e)
    if got[1] is not None:
        check_interval(got[1], d.T, e.T)
    if got[2] is not None:
        assert (np.abs(got[2].double().cpu().numpy() - db) <= de).all()


SHAPES = [(1, 1), (1, 300), (2, 129), (127, 128), (128, 16), (129, 17), (256, 260), (300, 1029), (1000, 200), (2100, 130)]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", ACTS)
def test_backward(M, N, dtype, act):
    rng = np.random.default_rng([M, N])
    dy, dy64, ck, pre64 = inputs(rng, M, N, dtype, act)
    rows, cols = U.Guarded(M, N, extra=16), U.Guarded(N, M)
    q, t, db = taco.taco_linear_fp8_backward(dy, ck, act, out=rows.t, out_t=cols.t)
    assert q.codes is rows.t.codes and t.codes is cols.t.codes
    check((rows.get(), cols.get(), db), dy64, pre64, act)


@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 1), (16, 8), (1, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides(pad, offset, dtype):
    rng = np.random.default_rng(pad)
    dy, dy64, ck, pre64 = inputs(rng, 300, 277, dtype, "gelu")
    q, t, db = taco.taco_linear_fp8_backward(U.strided(dy, pad, offset), ck, "gelu")
    get = lambda p: (p.codes.cpu().numpy(), p.scales.cpu().numpy())  # noqa: E731
    check((get(q), get(t), db), dy64, pre64, "gelu")


@pytest.mark.parametrize("rows,cols,bias", [(r, c, b) for r in (0, 1) for c in (0, 1) for b in (0, 1) if r or c or b])
@pytest.mark.parametrize("M", [100, 500])
def test_each_output_alone(rows, cols, bias, M):
    rng = np.random.default_rng(3)
    dy, _, ck, _ = inputs(rng, M, 200, "bf16", "silu")
    whole = taco.taco_linear_fp8_backward(dy, ck, "silu")
    some = taco.taco_linear_fp8_backward(dy, ck, "silu", rows=rows, cols=cols, bias=bias)
    for there, a, b in zip((rows, cols, bias), some, whole):
        assert (a is not None) == bool(there)
        if there and a is some[2]:
            assert torch.equal(a, b)
        elif there:
            assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


def test_without_an_activation_it_is_the_quantiser():
    rng = np.random.default_rng(4)
    for dtype in ("bf16", "f16", "f32"):
        dy, dy64, _, _ = inputs(rng, 300, 520, dtype, None)
        q, t, db = taco.taco_linear_fp8_backward(dy)
        a, b = taco.taco_fp8_quantize(dy, cols=True)
        for x, y in ((q, a), (t, b)):
            assert torch.equal(x.codes, y.codes) and torch.equal(x.scales, y.scales)


@pytest.mark.parametrize("act", ACTS[1:])
def test_slopes_at_their_ends(act):
    """Pre-activations up to the largest that a block holds, and NaN blocks."""
    N = 128 * 40
    pre = np.zeros((2, N))
    for b in range(40):
        pre[:, 128 * b:128 * b + 128] = np.linspace(-1, 1, 128) * 2.0 ** (3 * b - 20)
    q = Q.quantize(pre)
    ck = U.held(*q)
    dy = torch.ones(2, N, device="cuda")
    _, _, db = taco.taco_linear_fp8_backward(dy, ck, act)
    want = Q.activation_slope(np.clip(Q.dequantize(*q), -1e6, 1e6), act)
    got = db.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want.sum(axis=0)) <= 2 * SLOPE + 2.0 ** -22).all()
    ck.scales[0, 3] = 255
    rows, cols, db = taco.taco_linear_fp8_backward(dy, ck, act)
    bad = torch.isnan(db)
    assert bad[384:512].all() and not bad[:384].any() and not bad[512:].any()
    assert rows.scales[0, 3] == 255 and rows.scales[1, 3] != 255 and (cols.scales[384:512] == 255).all()


def test_nan_blocks_of_a_ragged_row_stay_in_it():
    rng = np.random.default_rng(5)
    dy, _, ck, _ = inputs(rng, 200, 130, "bf16", "gelu")
    ck.scales[7, 1] = 255
    rows, cols, db = taco.taco_linear_fp8_backward(dy, ck, "gelu")
    assert torch.isnan(db[128:]).all() and not torch.isnan(db[:128]).any()
    assert (rows.scales[:, 0] != 255).all() and (cols.scales[128:, 0] == 255).all() and (cols.scales[:128] != 255).all()


def test_no_rows():
    dy = torch.zeros(0, 300, device="cuda")
    q, t, db = taco.taco_linear_fp8_backward(dy)
    assert q.codes.shape == (0, 300) and t.codes.shape == (300, 0) and db.tolist() == [0.0] * 300


def test_repeats_on_any_stream_and_in_a_graph():
    rng = np.random.default_rng(6)
    M, N = 1000, 520
    dy, _, ck, _ = inputs(rng, M, N, "bf16", "gelu_tanh")
    first = taco.taco_linear_fp8_backward(dy, ck, "gelu_tanh")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    again = taco.taco_linear_fp8_backward(dy, ck, "gelu_tanh", stream=side)
    torch.cuda.synchronize()
    out, out_t, db = F.fp8_empty(M, N), F.fp8_empty(N, M), torch.empty(N, device="cuda")
    ws = torch.empty(8 * N * 4, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        taco.taco_linear_fp8_backward(dy, ck, "gelu_tanh", out=out, out_t=out_t, db=db, workspace=ws)
    graph.replay()
    for other in (again, (out, out_t, db)):
        for a, b in zip(first[:2], other[:2]):
            assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
        assert torch.equal(first[2], other[2])


@pytest.mark.parametrize("act", ACTS)
def test_gradients_of_a_layer(act):
    """dx, dw and db of y = act(x w^T + b) through the FP8 products against the
    formula's at the same quantised operands: what differs are the roundings of
    d, rows and transpose, 3.6% in the root mean square of each value, which the
    products' sums only make smaller relative to the result of independent terms."""
    rng = np.random.default_rng(7)
    M, N, K = 512, 384, 640
    x, w = rng.standard_normal((M, K)), rng.standard_normal((N, K)) * K ** -0.5
    xq, wq = Q.quantize(x), Q.quantize(w, 128)
    x64, w64 = Q.dequantize(*xq), Q.dequantize(*wq)
    xf, wf = U.held(*xq), U.held(*wq)
    b = torch.randn(N, device="cuda")
    y, kept = taco.taco_linear_fp8(xf, wf, b, act, checkpoint=True)
    dy = torch.from_numpy(rng.standard_normal((M, N))).bfloat16().cuda()
    d, dt, db = taco.taco_linear_fp8_backward(dy, kept if act else None, act)
    _, wt = taco.taco_fp8_quantize(wf, rows=False, cols=True)
    _, xt = taco.taco_fp8_quantize(xf, rows=False, cols=True)
    dx = taco.taco_matmul_fp8(d, wt, out_dtype=torch.float32)
    dw = taco.taco_matmul_fp8(dt, xt, out_dtype=torch.float32)
    pre = x64 @ w64.T + b.double().cpu().numpy()
    d64 = dy.double().cpu().numpy() * Q.activation_slope(pre, act)
    far = lambda a, r: np.linalg.norm(a.double().cpu().numpy() - r) / np.linalg.norm(r)  # noqa: E731
    bound = 0.036 * 3 ** 0.5 if act != "relu" else 0.15   # relu: signs of values that the checkpoint rounds to zero
    assert far(db, d64.sum(axis=0)) < bound
    assert far(dx, d64 @ w64) < bound and far(dw, d64.T @ x64) < bound
