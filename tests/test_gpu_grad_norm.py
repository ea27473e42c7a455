"""The norm of many tensors and its clipping factor against 64-bit sums.

Tolerance: a thread sums fp32 squares of one sign, at most a few thousand; the
rounding of a square (2^-24 of it) and of each partial sum (2^-24 of that) add
to less than 2^-24 (1 + k) of a thread's sum of k additions, here k <= 64 for
what the tests make, the root halves it, and its own rounding is 2^-24.
"""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import grads_taco_compress_gb300 as taco
from grads_taco_compress_gb300 import binding as tb

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
REL = 2.0 ** -24 * (1 + 65 / 2)


def make(seed, specs, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for n, dtype in specs:
        t = torch.randn(n + offset, generator=g, device="cuda").to(DTYPES[dtype])
        out.append(t[offset:])
    return out


def exact(grads):
    return math.sqrt(sum(float(t.double().square().sum()) for t in grads))


@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("specs", [
    [(1, "f32")], [(17, "bf16"), (4096, "f16"), (4097, "f32")], [(0, "f32"), (5, "f16"), (0, "bf16")],
    [(100003, "bf16"), (65536, "f32"), (129, "f16"), (300000, "f16")],
    [(1 + i % 50, ("f32", "bf16", "f16")[i % 3]) for i in range(3000)],
    [(1000, "bf16")] * 128, [(1000, "bf16")] * 129])
def test_norm_and_factor(specs, offset):
    grads = make(len(specs), specs, offset)
    want = exact(grads)
    norm, factor = taco.taco_grad_norm(grads).tolist()
    assert abs(norm - want) <= REL * want and factor == 1.0
    norm2, factor = taco.taco_grad_norm(grads, max_norm=0.25 * want).tolist()
    assert norm2 == norm and abs(factor - 0.25) <= 0.25 * (REL + 2.0 ** -22)
    assert taco.taco_grad_norm(grads, max_norm=1.01 * want)[1] == 1.0
    assert taco.taco_grad_norm(grads, max_norm=0.0)[1] == 0.0


def test_zeros_and_ends_of_the_range():
    z = torch.zeros(5000, device="cuda")
    assert taco.taco_grad_norm([z], max_norm=0.0).tolist() == [0.0, 1.0]
    assert taco.taco_grad_norm([z[:0]]).tolist() == [0.0, 1.0]
    for e in (62, -62):
        r = taco.taco_grad_norm([torch.full((3,), 2.0 ** e, device="cuda")]).tolist()[0]
        assert abs(r / (math.sqrt(3) * 2.0 ** e) - 1) <= REL


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_what_is_not_finite_gives_no_factor(bad, dtype):
    grads = make(3, [(70000, dtype), (100, dtype)])
    grads[1][99] = bad
    norm, factor = taco.taco_grad_norm(grads, max_norm=1.0).tolist()
    assert not math.isfinite(norm) and math.isnan(factor)


def test_order_is_fixed_and_outputs_and_workspace_are_the_callers():
    grads = make(4, [(1234567, "f32"), (99, "bf16")])
    out, ws = torch.empty(2, device="cuda"), torch.full((1024 * 8,), 0xA5, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    first = taco.taco_grad_norm(grads, 1.0)
    got = taco.taco_grad_norm(grads, 1.0, out=out, workspace=ws, stream=side)
    torch.cuda.synchronize()
    assert got is out and torch.equal(first, out)


def test_captured():
    grads = make(5, [(30000, "bf16"), (77, "f32")])
    out = torch.empty(2, device="cuda")
    ws = torch.empty(1024 * 8, dtype=torch.uint8, device="cuda")
    taco.taco_grad_norm(grads, 1.0, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        taco.taco_grad_norm(grads, 1.0, out=out, workspace=ws)
    for k in (1.0, 3.0):
        for t in grads:
            t.mul_(k)
        graph.replay()
        assert abs(out[0].item() - exact(grads)) <= REL * exact(grads)


def test_offsets_past_32_bits():
    n = 2 ** 32 + 1000
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[-3:] = 2.0
    t[0] = 1.0
    assert taco.taco_grad_norm([t])[0].item() == pytest.approx(math.sqrt(13), rel=1e-7)


def test_optimiser_clips_and_counts():
    p = [torch.ones(1000, dtype=torch.bfloat16, device="cuda"), torch.ones(10, device="cuda")]
    opt = taco.AdamW(p, lr=0.1, weight_decay=0.0, bits=8)
    g = [torch.full((1000,), 0.5, device="cuda"), torch.full((10,), 0.5, device="cuda")]
    norm = opt.step(g, max_norm=1.0)
    assert abs(norm[0].item() - 0.5 * math.sqrt(1010)) < 1e-4 and opt.counter.tolist() == [1, 0]
    np.testing.assert_allclose(p[1].cpu().numpy(), 0.9, rtol=1e-5)
    g[0][5] = float("nan")
    keep = [t.clone() for t in p]
    opt.step(g, max_norm=1.0)
    assert opt.counter.tolist() == [1, 0] and all(torch.equal(a, b) for a, b in zip(keep, p))
    assert tb.taco_get_fault() == 0
