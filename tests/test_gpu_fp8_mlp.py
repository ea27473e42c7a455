"""The tensor-parallel MLP block (norm, two FP8 products, gated activation,
compressed AllReduce, and their gradients) against the same block in fp64.

Tolerance: rounding to E4M3 is off by at most 2^-4 of a value and by 2^-4 /
sqrt(3) = 3.6% in the root mean square where the values fill a binade evenly.
Errors of independent roundings add in squares: the output passes four (norm
output, gate/up product's weights, gated output, second weights) and the
AllReduce's two, the gradients up to five more, so 3.6% sqrt(11) = 12% bounds
the relative distance of every tensor.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

from grads_taco_compress_gb300 import binding as tb
from grads_taco_compress_gb300.mlp import TensorParallelMlp

pytestmark = pytest.mark.gpu
BOUND = 0.12


def reference(m, x, residual, dout, dh):
    w_norm = m.w_norm.double().requires_grad_()
    w_in = [w.double().requires_grad_() for w in m.w_in]
    w_out = [w.double().requires_grad_() for w in m.w_out]
    x = x.double().requires_grad_()
    h = x + residual.double()
    n = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + m.eps) * w_norm
    out = 0
    for a, b in zip(w_in, w_out):
        gate, up = (n @ a.t()).chunk(2, dim=1)
        out = out + (gate * torch.sigmoid(gate) * up) @ b.t()
    ((out * dout.double()).sum() + (h * dh.double()).sum()).backward()
    return out.detach(), h.detach(), x.grad, w_norm.grad, [w.grad for w in w_in], [w.grad for w in w_out]


def far(a, b):
    a, b = a.double(), b.double()
    return ((a - b).norm() / b.norm()).item()


@pytest.mark.parametrize("R,M,h,f", [(2, 512, 1024, 1024), (4, 256, 1600, 3200), (1, 384, 512, 640)])
def test_block_and_gradients(R, M, h, f):
    torch.manual_seed(R)
    m = TensorParallelMlp(R, M, h, f, block=64)
    m.w_norm.copy_(1 + 0.1 * torch.randn(h, device="cuda"))
    x, residual, dout, dh = (torch.randn(M, h, device="cuda").bfloat16() for _ in range(4))
    dout = dout * 0.01
    dh = dh * 0.01
    out, stream = m.forward(x, residual)
    dx = m.backward(dout, dh)
    want = reference(m, x, residual, dout, dh)
    assert far(stream, want[1]) < 2 ** -8
    assert far(out, want[0]) < BOUND
    assert far(dx, want[2]) < BOUND
    assert far(m.dw_norm, want[3]) < BOUND
    for r in range(R):
        assert far(m.dw_in[r], want[4][r]) < BOUND
        assert far(m.dw_out[r], want[5][r]) < BOUND
    # a second step adds to the running gradients
    first = [g.clone() for g in (m.dw_norm, m.dw_in[0], m.dw_out[0])]
    m.forward(x, residual)
    m.backward(dout, dh)
    for a, b in zip((m.dw_norm, m.dw_in[0], m.dw_out[0]), first):
        np.testing.assert_allclose(a.cpu().numpy(), 2 * b.cpu().numpy(), rtol=1e-5, atol=1e-6 * float(b.abs().max()))
    assert tb.taco_get_fault() == 0

