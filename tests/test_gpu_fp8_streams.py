"""FP8 entry points on other streams than the tensors' own, at the same time on
two streams, on tensors whose offsets pass 32 bits, and at the ends of the
scales' range."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_util as U
from grads_taco_compress_gb300 import binding as tb
from grads_taco_compress_gb300 import fp8 as F

pytestmark = pytest.mark.gpu


def test_what_a_call_allocates_belongs_to_its_stream():
    """Calls on a side stream that is held up: memory that they allocate (the
    outputs, the gradient's workspace) must not be handed out on the main
    stream before they have run."""
    torch.manual_seed(0)
    M, H = 2048, 2048
    dy, h, dh = (torch.randn(M, H, device="cuda").bfloat16() for _ in range(3))
    w, rstd = torch.randn(H, device="cuda"), torch.rand(M, device="cuda") + 0.5
    gate_up = torch.randn(M, H, device="cuda").bfloat16()
    want = F.taco_rms_norm_fp8_backward(dy, h, w, rstd, dh=dh)
    wq, wt = F.taco_fp8_quantize(h, cols=True)
    wy, wck = F.taco_swiglu_fp8(gate_up, checkpoint=True)
    wc = F.taco_matmul_fp8(wq, wq, out_dtype=torch.float32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)          # about a millisecond
        got = F.taco_rms_norm_fp8_backward(dy, h, w, rstd, dh=dh, stream=side)
        q, t = F.taco_fp8_quantize(h, cols=True, stream=side)
        y, ck = F.taco_swiglu_fp8(gate_up, checkpoint=True, stream=side)
        c = F.taco_matmul_fp8(q, q, out_dtype=torch.float32, stream=side)
        # the main stream meanwhile allocates blocks of the same sizes and fills them
        junk = [torch.full((n,), 0x7B, dtype=torch.uint8, device="cuda")
                for n in (512 * H * 4, M * H * 2, M * H, H * 4, M * 16) for _ in range(4)]
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(q.codes, wq.codes) and torch.equal(t.codes, wt.codes)
        assert torch.equal(y.codes, wy.codes) and torch.equal(ck.codes, wck.codes)
        assert torch.equal(c, wc)
        del junk, got, q, t, y, ck, c


def test_two_streams_at_once():
    torch.manual_seed(1)
    shapes = [(2048, 1600, 2048), (8, 4096, 4096), (300, 520, 640), (96, 2048, 1024)]
    ops = []
    for M, N, K in shapes:
        a, _ = F.taco_fp8_quantize(torch.randn(M, K, device="cuda"))
        b, _ = F.taco_fp8_quantize(torch.randn(N, K, device="cuda"), tile=128)
        ops.append((a, b, F.taco_matmul_fp8(a, b, out_dtype=torch.float32)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(c) for _, _, c in ops] for _ in streams]
    for i in range(40):
        for s, out in zip(streams, outs):
            for j, (a, b, _) in enumerate(ops if s is streams[0] else ops[::-1]):
                F.taco_matmul_fp8(a, b, out=out[j if s is streams[0] else len(ops) - 1 - j], stream=s)
    torch.cuda.synchronize()
    for out in outs:
        for got, (_, _, want) in zip(out, ops):
            assert torch.equal(got, want)
    assert tb.taco_get_fault() == 0


def test_offsets_beyond_32_bits():
    """More than 2^32 elements: the last rows and columns against the same rows alone."""
    M, K = 270_400, 16_384
    gen = torch.Generator(device="cuda").manual_seed(5)
    tail = 384
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    for r in range(0, M, 65_536):
        x[r:r + 65_536].normal_(generator=gen)
    assert x.numel() > 1 << 32 and M % 128 == 64
    last = x[M - tail - 64:]                      # starts on a block of 128 rows
    q, t = F.taco_fp8_quantize(x, cols=True)
    qs, ts = F.taco_fp8_quantize(last, cols=True)
    assert torch.equal(q.codes[M - tail - 64:], qs.codes) and torch.equal(q.scales[M - tail - 64:], qs.scales)
    assert torch.equal(t.codes[:, M - tail - 64:], ts.codes)
    assert torch.equal(t.scales[:, -ts.scales.shape[1]:], ts.scales)
    del t, ts
    b, _ = F.taco_fp8_quantize(torch.randn(264, K, device="cuda"), tile=128)
    c = F.taco_matmul_fp8(q, b)
    torch.testing.assert_close(c[M - tail - 64:].float(), F.taco_matmul_fp8(qs, b).float(), rtol=2 ** -7, atol=1e-3)
    del c, q
    w = torch.ones(K, device="cuda")
    n, ns = F.taco_rms_norm_fp8(x, w, checkpoint=True), F.taco_rms_norm_fp8(last, w, checkpoint=True)
    assert torch.equal(n.y.codes[M - tail - 64:], ns.y.codes) and torch.equal(n.rstd[M - tail - 64:], ns.rstd)
    dx, _ = F.taco_rms_norm_fp8_backward(x, n.checkpoint, w, n.rstd)
    dxs, _ = F.taco_rms_norm_fp8_backward(last, ns.checkpoint, w, ns.rstd)
    assert torch.equal(dx[M - tail - 64:], dxs)
    del n, dx
    y, ck = F.taco_swiglu_fp8(x, checkpoint=True)
    ys, cks = F.taco_swiglu_fp8(last, checkpoint=True)
    assert torch.equal(y.codes[M - tail - 64:], ys.codes) and torch.equal(ck.codes[:, M - tail - 64:], cks.codes)
    d = F.taco_swiglu_fp8_backward(x[:, :K // 2], ck)
    ds = F.taco_swiglu_fp8_backward(last[:, :K // 2], cks)
    assert torch.equal(d[M - tail - 64:], ds)


@pytest.mark.parametrize("M,N", [(4, 256), (300, 700)])
@pytest.mark.parametrize("sa,sb", [(1, 247), (10, 240), (247, 1), (60, 190), (127, 1), (90, 90)])
def test_matmul_scales_at_the_ends(M, N, sa, sb):
    """Every pair of scales whose products fp32 holds: the result is that of unit scales times their product."""
    K = 384
    rng = np.random.default_rng([M, sa])
    codes = [rng.integers(0x20, 0x50, (R, K)).astype(np.uint8) for R in (M, N)]

    def product(s, t):
        a, b = (U.held(c, np.full((c.shape[0], 3), v, dtype=np.uint8)) for c, v in zip(codes, (s, t)))
        return F.taco_matmul_fp8(a, b, out_dtype=torch.float32).double().cpu().numpy()

    want = product(127, 127) * 2.0 ** (sa + sb - 254)
    np.testing.assert_allclose(product(sa, sb), want, rtol=2.0 ** -20)
