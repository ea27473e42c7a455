"""The norm of values at the ends of their types' ranges.

Tolerance, u = 2^-24: a square is off by u of itself, and where it is a square of
a scaled value that counts, by no more; a sum of up to 32 of one sign by 31 u more
at most; the root halves that and is rounded once: 17 u. Where the norm itself is
below 2^-126 it is a multiple of 2^-149, off by half of that, and so is max_norm.
The factor, one by the other: a norm that is not zero is at least 2^-149, so the
rounded one is at least half of it, and the factor is off by at most
2 2^-150 / norm for max_norm and 2 2^-150 / norm of itself for the norm more.
"""

from __future__ import annotations

import math

import pytest
import torch

import grads_taco_compress_gb300 as taco

pytestmark = pytest.mark.gpu
REL = 17 * 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def check(grads, want, max_norm=math.inf):
    norm, factor = taco.taco_grad_norm(grads, max_norm=max_norm).tolist()
    assert abs(norm - want) <= REL * want + 2.0 ** -150
    if norm > max_norm:
        assert abs(factor - max_norm / want) <= ((2 * REL * max_norm + 2.0 ** -149 * (1 + max_norm / want)) / want
                                                 + 2.0 ** -149)
    else:
        assert factor == 1.0


@pytest.mark.parametrize("n", [1, 2, 3, 15, 16, 31, 33, 100000])
@pytest.mark.parametrize("dtype,e", [
    (dtype, e) for dtype, smallest in ((F32, -149), (BF16, -133))
    for e in (-149, -140, -133, -127, -126, -100, -75, -64, -63, -62, -46, -45, -44, 56, 57, 58, 62, 63, 64, 80, 100, 118)
    if e >= smallest])
def test_equal_values(n, dtype, e):
    t = torch.full((n,), 2.0 ** e, dtype=dtype, device="cuda")
    if n > 2:
        t[1] *= -1
    want = math.sqrt(n) * 2.0 ** e
    check([t], want)
    check([t], want, max_norm=0.25 * want)


@pytest.mark.parametrize("big,small", [(2.0 ** 100, 1.0), (2.0 ** 63, 2.0 ** 62), (1.0, 2.0 ** -100), (2.0 ** -60, 2.0 ** -75),
                                       (3e38, 1e-40), (2.0 ** -46, 2.0 ** -126)])
@pytest.mark.parametrize("apart", [False, True])
def test_values_of_different_sizes(big, small, apart):
    """In one thread's elements, and in different ones' and different tensors."""
    a = torch.zeros(70000, device="cuda")
    a[:8] = small
    b = torch.zeros(5000, dtype=BF16, device="cuda") if apart else a
    b[4999 if apart else 9] = big
    grads = [a, b] if apart else [a]
    check(grads, math.sqrt(sum(float(g.double().square().sum()) for g in grads)))


def test_largest_and_smallest():
    most = torch.finfo(F32).max
    check([torch.tensor([most], device="cuda")], most)
    check([torch.full((4,), most / 4, device="cuda"), torch.full((4,), -most / 4, device="cuda")], math.sqrt(8) * most / 4)
    for t in (torch.full((2,), most, device="cuda"), torch.full((2,), torch.finfo(BF16).max, dtype=BF16, device="cuda")):
        norm, factor = taco.taco_grad_norm([t], 1.0).tolist()
        assert norm == math.inf and math.isnan(factor)      # the norm itself is no fp32 number
    for v in (65504.0, 2.0 ** -24):
        check([torch.full((100000,), v, dtype=F16, device="cuda")], math.sqrt(100000) * v)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_random_magnitudes(dtype):
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(300000, generator=g, device="cuda").double()
    for lo, hi in ((-149, -60), (-120, 20), (50, 118), (-149, 118)):
        e = torch.randint(lo, hi, x.shape, generator=g, device="cuda")
        t = (x * torch.exp2(e.double())).to(dtype)
        check([t[1:]], math.sqrt(float(t[1:].double().square().sum())))


def test_a_clipped_step_after_large_gradients():
    """Gradients whose squares lie beyond fp32 are clipped, and the step is taken."""
    p = [torch.zeros(1000, device="cuda")]
    opt = taco.AdamW(p, lr=0.5, weight_decay=0.0)
    norm = opt.step([torch.full((1000,), 2.0 ** 64, device="cuda")], max_norm=1.0)
    assert opt.counter.tolist() == [1, 0] and norm[0].item() == pytest.approx(math.sqrt(1000) * 2.0 ** 64, rel=1e-6)
    assert (p[0] + 0.5).abs().max() < 1e-6    # the rate, against the sign
