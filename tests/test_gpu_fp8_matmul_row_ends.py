"""The FP8 product into columns of a wider matrix whose rows start on 16 bytes
but whose own rows end elsewhere: what lies behind a row is left alone."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_util as U
from grads_taco_compress_gb300 import binding as tb
from grads_taco_compress_gb300 import fp8 as F
from test_gpu_fp8_matmul import operand
from test_gpu_fp8_matmul_tiles import check16

pytestmark = pytest.mark.gpu
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# few rows; pairs of CTAs on tiles 128 wide; on tiles 256 wide (f32: 128), several a pair
@pytest.mark.parametrize("M,N0,K", [(5, 248, 640), (100, 248, 130), (300, 1152, 384), (100, 0, 256), (2100, 5376, 260)])
@pytest.mark.parametrize("dtype,end", [(t, e) for t, size in SIZE.items() for e in range(1, 16 // size)])
@pytest.mark.parametrize("add", [False, True])
def test_columns_of_a_wider_matrix(M, N0, K, dtype, end, add):
    per = 16 // SIZE[dtype]
    N = N0 + end
    width = N0 + 2 * per            # a multiple of 16 bytes
    rng = np.random.default_rng([M, N, K])
    a, a64 = operand(rng, M, K, 1)
    b, b64 = operand(rng, N, K, 1)
    if dtype == "f16":              # keep the sums inside the type's range
        a, b = (U.held(t.codes.cpu().numpy(), (t.scales - 14).cpu().numpy()) for t in (a, b))
        a64, b64 = a64 * 2.0 ** -14, b64 * 2.0 ** -14
    c, c64 = U.values(rng, M, N, dtype, 1.0)
    behind = torch.randn(M, width - N, device="cuda").to(U.DTYPES[dtype])
    wide = torch.cat([c if add else torch.zeros_like(c), behind], dim=1)
    assert wide.stride(0) * SIZE[dtype] % 16 == 0 and N * SIZE[dtype] % 16
    out = wide[:, :N]
    F.taco_matmul_fp8(a, b, out=out, add=out if add else None)
    assert torch.equal(wide[:, N:], behind)
    check16(out, a64, b64, K, dtype, c64 if add else np.zeros((1, 1)))
    assert tb.taco_get_fault() == 0
