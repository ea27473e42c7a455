"""Second moments at the ends of fp32: their roots and what is divided by them.

Tolerances, u = 2^-24, as in test_gpu_adamw.py: m is off by 6 u of the sum of its
terms' magnitudes. v is off by 8 u of itself and, below 2^-126, by half of
fp32's smallest step, 2^-150, for each of its product, its sum and (in 8 bits)
the square of the root that was held. The root is off by half of v's relative
error and 2 u, the update by its own 32 u, by what m is off and by what the
root's share of the denominator is off.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import grads_taco_compress_gb300 as taco
from oracle import fp8_oracle as Q
from oracle import optim_oracle as O
from test_gpu_adamw import codes_of, f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LR, B1, B2 = 1e-3, 0.9, 0.95
N = 1000


def moments(state, bits):
    """m and v in fp64."""
    if bits == 32:
        return f64(state.m), f64(state.v)
    m, r = (O.state_values(*codes_of(s)) for s in state)
    return m, r * r


def check_codes(state, y, dy, w, rounding):
    """Codes and scales that are the rounding of some value within dy of y."""
    codes, scales = codes_of(state)
    lo = Q.scale_byte(Q.block_amax(np.maximum(np.abs(y) - dy, 0)[None])[0])
    hi = Q.scale_byte(Q.block_amax((np.abs(y) + dy)[None])[0])
    assert ((scales >= np.minimum(lo, hi)) & (scales <= np.maximum(lo, hi))).all()
    s = np.repeat(2.0 ** (scales.astype(np.float64) - 127), 128)[:y.size]
    have = O.state_values(codes, scales) / s
    ends = [rounding(np.clip((y + k * dy) / s, -448, 448), w) for k in (-1, 1)]
    assert ((have >= ends[0]) & (have <= ends[1])).all()


@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-30, 1e-25, 1e-20, 1e-8])
@pytest.mark.parametrize("exponents", [(-66, -60), (-70, -62), (-64, -50), (-66, -60, -40, 0), (-66, 0, 40, 55), (50, 55)])
@pytest.mark.parametrize("bits", [32, 8])
def test_small_second_moments(bits, exponents, eps):
    rng = np.random.default_rng([bits, -min(exponents) + 100, len(exponents)])
    p = torch.zeros(N, device="cuda")
    state = taco.taco_adam_state(p, bits)
    counter = torch.zeros(2, dtype=torch.int32, device="cuda")
    for t in (1, 2, 3):
        g = torch.from_numpy((1 + rng.random(N)) * 2.0 ** rng.choice(exponents, N) * rng.choice([-1, 1], N)).float().cuda()
        x0, d = f64(p), f64(g)
        m0, v0 = moments(state, bits)
        taco.taco_adamw([p], [g], [state], counter, lr=LR, betas=(B1, B2), eps=eps, weight_decay=0.0)
        x, m, v, update, den = O.adamw(x0, d, m0, v0, t, LR, B1, B2, eps, 0.0)
        root = np.sqrt(v)
        dm = 6 * U * (B1 * np.abs(m0) + (1 - B1) * np.abs(d)) + 2.0 ** -149
        dv = 8 * U * v + 3 * 2.0 ** -150
        assert (dv < v / 4).all()            # or nothing below would be said
        droot = dv / root + 2 * U * root     # more than half of dv / v, as much as v - dv may be below v
        dden = droot / np.sqrt(1 - B2 ** t)
        dx = (4 * U * np.abs(x) + 4 * U * np.abs(x0) + 32 * U * np.abs(update) + LR / (1 - B1 ** t) * dm / den
              + np.abs(update) * dden / (den - dden))
        assert (np.abs(f64(p) - x) <= dx).all()
        if bits == 32:
            assert (np.abs(f64(state.m) - m) <= dm).all() and (np.abs(f64(state.v) - v) <= dv).all()
        else:
            w = O.thresholds(N, t)
            check_codes(state.m, m, dm, w, lambda a, b: O.by_threshold(a, b, "e4m3"))
            check_codes(state.v, root, droot, w, O.root_codes)
            assert (state.v.codes != 0).all()
    assert counter.tolist() == [3, 0]


@pytest.mark.parametrize("bits", [32, 8])
def test_the_first_step_is_the_rate_where_eps_counts_for_nothing(bits):
    """sign(g) lr, whatever the gradient's size."""
    for e in (-66, -60, -30, 0, 30, 60):
        p = torch.zeros(300, device="cuda")
        g = torch.full((300,), -2.0 ** e, device="cuda")
        taco.taco_adamw([p], [g], [taco.taco_adam_state(p, bits)], torch.zeros(2, dtype=torch.int32, device="cuda"),
                        lr=LR, betas=(0.9, 0.999), eps=1e-36, weight_decay=0.0)
        # v = 2^(2 e) / 1000 in steps of 2^-149: 2^-8 of it at e = -66
        assert (p - LR).abs().max() < LR * (2.0 ** -8 if e < -62 else 2.0 ** -18)
