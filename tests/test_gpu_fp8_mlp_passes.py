"""Several passes of the tensor-parallel MLP block: what a caller holds of one
stays as it was, and each backward pass belongs to the forward pass meant."""

from __future__ import annotations

import pytest
import torch

from grads_taco_compress_gb300 import binding as tb
from grads_taco_compress_gb300.allreduce import EmulatedTwoShotAllReduce
from grads_taco_compress_gb300.mlp import TensorParallelMlp

pytestmark = pytest.mark.gpu
R, M, H, FF = 2, 256, 512, 768


def block():
    torch.manual_seed(0)
    return TensorParallelMlp(R, M, H, FF, block=64)


def batches(n):
    gen = torch.Generator(device="cuda").manual_seed(1)
    return [[torch.randn(M, H, generator=gen, device="cuda").bfloat16() for _ in range(4)] for _ in range(n)]


def gradients(m):
    return [g.clone() for g in (m.dw_norm, *m.dw_in, *m.dw_out)]


def test_outputs_that_a_caller_holds_stay():
    m = block()
    (x1, r1, _, _), (x2, r2, _, _) = batches(2)
    out1, h1 = m.forward(x1, r1)
    held = out1.clone(), h1.clone()
    out2, h2 = m.forward(x2, r2)
    assert torch.equal(out1, held[0]) and torch.equal(h1, held[1])
    assert not torch.equal(out2, out1) and not torch.equal(h2, h1)
    mine = torch.empty_like(out1)
    out, _ = m.forward(x1, r1, out=mine)
    assert out is mine and torch.equal(mine, held[0])
    assert tb.taco_get_fault() == 0


@pytest.mark.parametrize("order", [(0, 1, 2), (2, 1, 0), (1, 2, 0)])
def test_micro_batches(order):
    """Three forward passes, then their backward passes in any order, against one after the other."""
    data = batches(3)
    one = block()
    dx = {}
    for i in order:
        x, r, dout, dh = data[i]
        one.forward(x, r)
        dx[i] = one.backward(dout, dh)
    m = block()
    saved = []
    for x, r, _, _ in data:
        m.forward(x, r)
        saved.append(m.saved)
    for i in order:
        assert torch.equal(m.backward(data[i][2], data[i][3], saved[i]), dx[i])
    for a, b in zip(gradients(m), gradients(one)):
        assert torch.equal(a, b)


def test_backward_without_its_forward_pass_is_refused():
    m = block()
    (x1, r1, dout, dh), (x2, r2, _, _) = batches(2)
    with pytest.raises(ValueError, match="no forward pass"):
        m.backward(dout, dh)
    m.forward(x1, r1)
    first = m.saved
    m.forward(x2, r2)
    before = gradients(m)
    with pytest.raises(ValueError, match="more than one forward pass"):
        m.backward(dout, dh)
    for a, b in zip(gradients(m), before):
        assert torch.equal(a, b)
    m.backward(dout, dh, first)
    m.backward(dout, dh, m.saved)
    assert m.saved is None
    with pytest.raises(ValueError, match="no forward pass"):
        m.backward(dout, dh)
    m.forward(x1, r1)
    m.backward(dout, dh)


def test_saved_state_is_in_8_bits():
    m = block()
    x, r, _, _ = batches(1)[0]
    m.forward(x, r)
    s = m.saved
    tensors = [*s.y, *s.checkpoint, *(t for pair in s.gated for fp8 in pair for t in fp8)]
    assert all(t.dtype == torch.uint8 for t in tensors)
    assert s.rstd.dtype == torch.float32 and s.rstd.shape == (M,)


def test_allreduce_into_a_given_tensor():
    gen = torch.Generator(device="cuda").manual_seed(2)
    xs = torch.randn(R, M, H, generator=gen, device="cuda").bfloat16()
    reduce = EmulatedTwoShotAllReduce(R, M, H, 64)
    want = reduce(xs)
    assert want is reduce.out
    mine = torch.empty_like(want)
    assert reduce(xs, out=mine) is mine and torch.equal(mine, want)
    for bad in (torch.empty(M, H, device="cuda"), torch.empty_like(mine)[:-2], torch.empty_like(mine).t()):
        with pytest.raises(ValueError, match="out must be"):
            reduce(xs, out=bad)
