"""Activations of infinite values, which a bias brings: +infinity stays what it is;
-infinity becomes 0 by relu and NaN by the others, whose formulas multiply it by 0.
Exact."""

from __future__ import annotations

import math

import pytest
import torch

import grads_taco_compress_gb300 as taco
from linear_util import ACTS

pytestmark = pytest.mark.gpu
INF = math.inf


@pytest.mark.parametrize("M,N,K", [(1, 130, 128), (40, 300, 256), (300, 513, 640), (700, 520, 130)])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ACTS)
def test_infinite_biases(M, N, K, kind, act):
    g = torch.Generator(device="cuda").manual_seed(M)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, _ = taco.taco_fp8_quantize(rand(M, K))
    w, _ = taco.taco_fp8_quantize(rand(N, K), tile=128)
    bias = rand(N)
    plain, _ = taco.taco_linear_fp8(x, w, bias, act, out_dtype=kind)
    bias[5], bias[N - 1], bias[64] = INF, INF, -INF
    y, kept = taco.taco_linear_fp8(x, w, bias, act, out_dtype=kind, checkpoint=True)
    assert (y[:, [5, N - 1]] == INF).all()
    low = y[:, 64]
    assert (low == -INF).all() if act is None else (low == 0).all() if act == "relu" else torch.isnan(low).all()
    rest = [n for n in range(N) if n not in (5, 64, N - 1)]
    assert torch.equal(y[:, rest], plain[:, rest])
    residual = torch.full_like(y, -1.0)
    assert (taco.taco_linear_fp8(x, w, bias, act, residual=residual, out_dtype=kind)[0][:, [5, N - 1]] == INF).all()
    assert (kept.scales[:, [0, (N - 1) // 128]] == 255).all()      # their blocks hold an infinity: NaN
