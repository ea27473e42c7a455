"""The norm of very many elements: a thread goes through thousands of chunks.

Tolerance, u = 2^-24: a square is off by u of itself, a sum of up to 32 of one
sign (four running sums of up to 8, joined) by 9 u more, sums in fp64 by nothing
that counts; the root halves that and is rounded once: 6 u.
"""

from __future__ import annotations

import math

import pytest
import torch

import grads_taco_compress_gb300 as taco

pytestmark = pytest.mark.gpu
REL = 6 * 2.0 ** -24


def squares(t):
    return sum(float(p.double().square().sum()) for p in t.view(-1).split(2 ** 26))


@pytest.mark.parametrize("dtype,value", [(torch.float32, 1.2109375), (torch.float32, 0.7), (torch.bfloat16, 1.2109375),
                                         (torch.bfloat16, 0.59765625), (torch.float16, 1.2109375)])
def test_the_same_tensor_a_thousand_times(dtype, value):
    """2^34 equal elements in one launch, of the same memory: the additions of a long
    sum would be rounded alike."""
    t = torch.full((2 ** 24,), value, dtype=dtype, device="cuda")
    want = math.sqrt(1024) * math.sqrt(squares(t))
    norm = taco.taco_grad_norm([t] * 1024)[0].item()
    assert abs(norm - want) <= REL * want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_large_dense_tensor(dtype):
    n = 2 ** 30 + 12345
    t = torch.empty(n, dtype=dtype, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    many = [t] * 7 + [t[:1000]]
    want = math.sqrt(7 * squares(t) + squares(t[:1000]))
    norm, factor = taco.taco_grad_norm(many, max_norm=0.5 * want).tolist()
    assert abs(norm - want) <= REL * want and abs(factor - 0.5) <= 0.5 * (REL + 2.0 ** -24)
    torch.cuda.empty_cache()
