"""Whole training steps of the tensor-parallel MLP block: forward, backward, the
norm of all gradients, an AdamW step, weights quantised again.

Distances: as in tests/test_gpu_fp8_mlp.py, independent roundings to E4M3 (3.6%
in the root mean square each) add in squares; the longest path has eleven, 12%.
relu's slope jumps, so a rounding of what lies near zero flips it: its gradients
are looked at through the block without that, by their formulas
(tests/test_gpu_fp8_linear_backward.py), and only run here.
"""

from __future__ import annotations

import pytest
import torch

import grads_taco_compress_gb300 as taco
from grads_taco_compress_gb300 import binding as tb
from grads_taco_compress_gb300.mlp import TensorParallelMlp

pytestmark = pytest.mark.gpu
BOUND = 0.12
ACT = {"gelu": torch.nn.functional.gelu, "gelu_tanh": lambda x: torch.nn.functional.gelu(x, approximate="tanh"),
       "silu": torch.nn.functional.silu, "relu": torch.relu}


def far(a, b):
    a, b = a.double(), b.double()
    return ((a - b).norm() / b.norm()).item()


def reference(m, x, residual, dout, dh):
    params = [p.double().requires_grad_() for p in m.parameters()]
    R = m.R
    w_norm, w_in, w_out, b_in, b_out = params[0], params[1:1 + R], params[1 + R:1 + 2 * R], params[1 + 2 * R:-1], params[-1]
    x = x.double().requires_grad_()
    h = x + residual.double()
    n = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + m.eps) * w_norm
    out = b_out
    for a, b, c in zip(w_in, w_out, b_in):
        out = out + ACT[m.activation](n @ a.t() + c) @ b.t()
    ((out * dout.double()).sum() + (h * dh.double()).sum()).backward()
    return out.detach(), x.grad, [p.grad for p in params]


def batch(M, h):
    x, residual, dout, dh = (torch.randn(M, h, device="cuda").bfloat16() for _ in range(4))
    return x, residual, dout * 0.01, dh * 0.01


@pytest.mark.parametrize("R,M,h,f", [(2, 512, 1024, 1024), (4, 256, 1600, 3200), (1, 384, 512, 640)])
@pytest.mark.parametrize("activation", ["gelu", "gelu_tanh", "silu"])
def test_block_without_a_gate(R, M, h, f, activation):
    torch.manual_seed(R)
    m = TensorParallelMlp(R, M, h, f, block=64, activation=activation)
    for b in (*m.b_in, m.b_out):
        b.normal_(0, 0.3)
    x, residual, dout, dh = batch(M, h)
    out, stream = m.forward(x, residual)
    dx = m.backward(dout, dh)
    want, want_dx, grads = reference(m, x, residual, dout, dh)
    assert far(out, want) < BOUND and far(dx, want_dx) < BOUND
    for got, g in zip(m.gradients(), grads):
        assert got.shape == g.shape and far(got, g) < BOUND
    assert tb.taco_get_fault() == 0


@pytest.mark.parametrize("activation", ["swiglu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("bits", [8, 32])
def test_steps(activation, bits):
    """Two micro-batches and a step: the masters move as an fp64 AdamW step on the
    block's own gradients moves them, and what the products read is theirs."""
    torch.manual_seed(1)
    m = TensorParallelMlp(2, 256, 512, 512, block=64, activation=activation)
    opt = taco.AdamW(m.parameters(), lr=1e-2, weight_decay=0.0, bits=bits, masters=True)
    for t in (1, 2):
        for _ in range(2):
            x, residual, dout, dh = batch(256, 512)
            m.forward(x, residual)
            m.backward(dout, dh)
        grads = [g.double().clone() for g in m.gradients()]
        before = [p.double().clone() if w is None else w.double().clone() for p, w in zip(m.parameters(), opt.masters)]
        norm = torch.sqrt(sum(g.square().sum() for g in grads)).item()
        got = m.step(opt, max_norm=0.5 * norm)
        assert abs(got[0].item() / norm - 1) < 1e-5 and abs(got[1].item() - 0.5) < 1e-5
        if t == 1:   # from zero states m / sqrt(v) is the sign, but where eps counts
            for p, w, b, g in zip(m.parameters(), opt.masters, before, grads):
                now = (p if w is None else w).double()
                want = b - 1e-2 * (0.5 * g) / ((0.5 * g).abs() + opt.eps)
                assert (now - want).abs().max() < 1e-6 + 2 ** -22 * b.abs().max()
        assert opt.counter.tolist() == [t, 0] and all(not g.any() for g in m.gradients())
        for w, (q, _) in zip(m.w_in + m.w_out, m._in + m._out):
            e, _ = taco.taco_fp8_quantize(w, tile=128)
            assert torch.equal(e.codes, q.codes) and torch.equal(e.scales, q.scales)
    assert tb.taco_get_fault() == 0


@pytest.mark.parametrize("activation", ["swiglu", "gelu"])
def test_a_captured_step_is_the_same_step(activation):
    """Forward, backward and step in one CUDA graph, replayed: equal, bit for bit,
    to the calls one by one, with the optimiser's count going on."""
    def build():
        torch.manual_seed(2)
        m = TensorParallelMlp(2, 256, 512, 512, block=64, activation=activation)
        return m, taco.AdamW(m.parameters(), lr=1e-2, bits=8)

    torch.manual_seed(3)
    data = [batch(256, 512) for _ in range(3)]
    x, residual, dout, dh = (t.clone() for t in data[0])

    def train(m, opt):
        out, _ = m.forward(x, residual)
        dx = m.backward(dout, dh)
        return out, dx, m.step(opt, max_norm=1.0)

    warm = build()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train(*warm)
    torch.cuda.current_stream().wait_stream(side)
    a, b = build(), build()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = train(*a)
    for t, d in enumerate(data, 1):
        for to, from_ in zip((x, residual, dout, dh), d):
            to.copy_(from_)
        graph.replay()
        eager = train(*b)
        assert a[1].counter.tolist() == b[1].counter.tolist() == [t, 0]
        for p, q in zip(captured, eager):
            assert torch.equal(p, q)
        for p, q in zip(a[0].parameters(), b[0].parameters()):
            assert torch.equal(p, q)
    assert tb.taco_get_fault() == 0


def test_arguments():
    with pytest.raises(ValueError):
        TensorParallelMlp(1, 128, 128, 128, block=64, activation="tanh")
