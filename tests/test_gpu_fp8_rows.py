"""Rows that start anywhere: inputs and outputs as views into wider matrices at
every alignment give bit for bit what contiguous ones do, and nothing beside
the rows is written."""

from __future__ import annotations

import pytest
import torch

import fp8_util as U
from grads_taco_compress_gb300 import fp8 as F

pytestmark = pytest.mark.gpu
WIDTHS = [1, 7, 8, 9, 15, 16, 17, 31, 127, 130, 500, 511, 512, 513, 519, 1029, 4095, 9001]


class View:
    """A NaN-filled matrix with an output view of [rows, cols] inside."""

    def __init__(self, rows, cols, dtype, pad, offset):
        self.big = torch.full((rows, offset + cols + pad), float("nan"), dtype=dtype, device="cuda")
        self.view, self.o, self.c = self.big[:, offset:offset + cols], offset, cols

    def check(self, want):
        assert torch.equal(self.view, want)
        assert torch.isnan(self.big[:, :self.o]).all() and torch.isnan(self.big[:, self.o + self.c:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (3, 1), (5, 2), (2, 3), (9, 5), (1, 7), (8, 8)])
def test_rows_that_start_anywhere(cols, pad, offset, dtype):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    t, M = U.DTYPES[dtype], 5

    def rand(n=cols):
        return torch.randn(M, n, generator=gen, device="cuda").to(t)

    x, r, dy, dh, gu = rand(), rand(), rand(), rand(), rand(2 * cols)
    w = torch.randn(cols, generator=gen, device="cuda").to(t)

    def at(v):
        return U.strided(v, pad, offset)

    want = F.taco_rms_norm_fp8(x, w, r, checkpoint=True)
    h = View(M, cols, t, pad, offset)
    got = F.taco_rms_norm_fp8(at(x), w, at(r), checkpoint=True, h=h.view)
    h.check(want.h)
    assert torch.equal(got.y.codes, want.y.codes) and torch.equal(got.y.scales, want.y.scales)
    assert torch.equal(got.checkpoint.codes, want.checkpoint.codes) and torch.equal(got.rstd, want.rstd)

    for saved, there in ((want.checkpoint, want.checkpoint), (want.h, at(want.h))):
        dx, dw = F.taco_rms_norm_fp8_backward(dy, saved, w, want.rstd, dh=dh)
        out = View(M, cols, t, pad, offset)
        _, dw2 = F.taco_rms_norm_fp8_backward(at(dy), there, w, want.rstd, dh=at(dh), dx=out.view)
        out.check(dx)
        assert torch.equal(dw, dw2)

    y, ck = F.taco_swiglu_fp8(gu, checkpoint=True)
    y2, ck2 = F.taco_swiglu_fp8(at(gu), checkpoint=True)
    assert torch.equal(y.codes, y2.codes) and torch.equal(ck.codes, ck2.codes) and torch.equal(ck.scales, ck2.scales)
    out = View(M, 2 * cols, t, pad, offset)
    F.taco_swiglu_fp8_backward(at(dy), ck, out=out.view)
    out.check(F.taco_swiglu_fp8_backward(dy, ck))

    for a, b in zip(F.taco_fp8_quantize(at(x), cols=True), F.taco_fp8_quantize(x, cols=True)):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
