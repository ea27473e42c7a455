"""The AdamW step over many tensors against the 64-bit oracle.

Tolerances, u = 2^-24 (half a step of fp32): m is two products and a sum of
rounded constants, off by at most 6 u of the sum of its terms' magnitudes; v by
8 u of itself; the root by half of that and 2 u of the square root; the update
by the quotient (4 u), its denominator (10 u) and its rate (8 u: a rounded
exponent, its expm1, a quotient), 32 u in all, and by what m is off; x by 4 u of
itself more. A value that is then rounded by a threshold lies between the
roundings of the ends of that interval.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import grads_taco_compress_gb300 as taco
from oracle import fp8_oracle as Q
from oracle import optim_oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
KW = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8)


def f64(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def codes_of(state):
    return state.codes.cpu().numpy().reshape(-1), state.scales.cpu().numpy().reshape(-1)


def blocks_of_one(x):
    return Q.block_amax(x[None])[0]


class Case:
    """Tensors with their states on the GPU, and the oracle's check of one step."""

    def __init__(self, seed, specs, offset=0, zero=False):
        """specs: (n, param type, gradient type, bits, master)."""
        rng = np.random.default_rng(seed)
        self.specs, self.params, self.grads, self.states, self.masters = specs, [], [], [], []
        for n, p, g, bits, master in specs:
            x = torch.from_numpy(rng.standard_normal(n) * 0.5).float().cuda()
            self.params.append(self.place(x.to(DTYPES[p]), offset))
            self.masters.append(self.place(x, offset) if master else None)
            d = rng.standard_normal(n) * 2.0 ** rng.integers(-12, 4, n)
            d[rng.random(n) < 0.1] = 0
            self.grads.append(self.place(torch.from_numpy(d).to(DTYPES[g]).cuda(), offset))
            m, v = rng.standard_normal(n) * 0.1, rng.random(n) ** 4
            m[rng.random(n) < 0.1] = 0
            v[rng.random(n) < 0.1] = 0
            if zero:
                self.states.append(taco.taco_adam_state(self.params[-1], bits))
            elif bits == 8:
                pair = []
                for s in (m, np.sqrt(v)):
                    c, e = Q.quantize(s[None])
                    pair.append(taco.Fp8Tensor(torch.from_numpy(c).cuda(), torch.from_numpy(e).cuda()))
                self.states.append(taco.AdamState(*pair))
            else:
                self.states.append(taco.AdamState(*(self.place(torch.from_numpy(s).float().cuda(), offset)
                                                    for s in (m, v))))
        self.counter = torch.zeros(2, dtype=torch.int32, device="cuda")

    @staticmethod
    def place(t, offset):
        """t, starting `offset` elements behind an aligned address."""
        b = torch.zeros(t.numel() + offset, dtype=t.dtype, device="cuda")
        b[offset:] = t
        return b[offset:]

    def before(self):
        out = []
        for i, (n, p, g, bits, master) in enumerate(self.specs):
            s = self.states[i]
            if bits == 8:
                m, r = (O.state_values(*codes_of(q)) for q in s)
                v = r * r
            else:
                m, v = f64(s.m), f64(s.v)
            out.append((f64(self.masters[i] if master else self.params[i]), f64(self.grads[i]), m, v))
        return out

    @np.errstate(invalid="ignore")
    def check(self, before, t, decay, factor=1.0, lr=KW["lr"]):
        b1, b2 = KW["betas"]
        for i, (n, p, g, bits, master) in enumerate(self.specs):
            if n == 0:
                continue
            x0, d, m0, v0 = before[i]
            d = d * factor
            x, m, v, update, den = O.adamw(x0, d, m0, v0, t, lr, b1, b2, KW["eps"], decay[i])
            dm = 6 * U * (b1 * np.abs(m0) + (1 - b1) * np.abs(d)) + 2.0 ** -149
            dx = 4 * U * np.abs(x) + 4 * U * np.abs(x0) + 32 * U * np.abs(update) + lr / (1 - b1 ** t) * dm / den
            w = O.thresholds(n, t)
            got = f64(self.params[i])
            if master:
                exact = f64(self.masters[i])
                assert (np.abs(exact - x) <= dx).all()
                assert torch.equal(self.params[i], self.masters[i].to(self.params[i].dtype))
            elif p == "f32":
                assert (np.abs(got - x) <= dx).all()
            else:
                fine = np.isfinite(x0)   # a parameter that a step took beyond its type stays infinite
                assert (got[~fine] == x0[~fine]).all()
                ends = [O.by_threshold((x + s * dx)[fine], w[fine], p) for s in (-1, 1)]
                assert ((got[fine] >= ends[0]) & (got[fine] <= ends[1])).all()
            if bits == 32:
                assert (np.abs(f64(self.states[i].m) - m) <= dm).all()
                assert (np.abs(f64(self.states[i].v) - v) <= 8 * U * v + 2.0 ** -149).all()
                continue
            root = np.sqrt(v)
            for state, y, dy, rounding in ((self.states[i].m, m, dm, lambda a, b: O.by_threshold(a, b, "e4m3")),
                                           (self.states[i].v, root, 6 * U * root, O.root_codes)):
                codes, scales = codes_of(state)
                lo = Q.scale_byte(blocks_of_one(np.maximum(np.abs(y) - dy, 0)))
                hi = Q.scale_byte(blocks_of_one(np.abs(y) + dy))
                assert ((scales >= np.minimum(lo, hi)) & (scales <= np.maximum(lo, hi))).all()
                s = np.repeat(2.0 ** (scales.astype(np.float64) - 127), 128)[:n]
                have = O.state_values(codes, scales) / s
                ends = [rounding(np.clip((y + k * dy) / s, -448, 448), w) for k in (-1, 1)]
                assert ((have >= ends[0]) & (have <= ends[1])).all()
        assert self.counter.tolist() == [t, 0]

    def step(self, decay, **kw):
        taco.taco_adamw(self.params, self.grads, self.states, self.counter, weight_decay=decay, masters=self.masters,
                        **{**KW, **kw})


SIZES = [1, 15, 16, 17, 127, 128, 129, 4095, 4096, 4097, 70001]
FORMS = [(p, g, bits, master) for p, g in (("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"),
                                           ("f32", "f32"))
         for bits in (32, 8) for master in ((False, True) if p != "f32" else (False,))]


@pytest.mark.parametrize("p,g,bits,master", FORMS)
@pytest.mark.parametrize("offset", [0, 3, 8])
def test_step(p, g, bits, master, offset):
    c = Case(hash((p, g, bits, offset)) % 1000, [(n, p, g, bits, master) for n in SIZES], offset)
    decay = [0.1 * (i % 3) for i in range(len(SIZES))]
    for t in (1, 2, 3):
        before = c.before()
        c.step(decay)
        c.check(before, t, decay)


@pytest.mark.parametrize("bits", [8, 32])
def test_from_zero_with_scale_and_rate_on_the_device(bits):
    c = Case(5, [(1000, "bf16", "f32", bits, False), (0, "bf16", "bf16", bits, False), (5000, "f32", "f32", bits, False)],
             zero=True)
    before = c.before()
    c.step(0.0, lr=torch.tensor([3e-3], device="cuda"), grad_scale=torch.tensor([0.125], device="cuda"))
    c.check(before, 1, [0.0] * 3, factor=0.125, lr=float(np.float32(3e-3)))


def test_many_tensors_of_all_forms():
    """More of one form than a launch takes, forms in turn, sizes that end anywhere."""
    forms = FORMS * 60
    specs = [(1 + (37 * i) % 400, *f) for i, f in enumerate(forms)]
    c = Case(6, specs + [(300, "bf16", "f32", 8, False)] * 450)
    decay = [0.05] * len(c.specs)
    before = c.before()
    c.step(decay)
    c.check(before, 1, decay)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_scale_that_is_not_finite_changes_nothing(bad):
    c = Case(7, [(3000, p, g, bits, master) for p, g, bits, master in FORMS])
    keep = [t.clone() for t in c.params + [m for m in c.masters if m is not None]]
    before = c.before()
    c.step(0.1, grad_scale=torch.tensor([bad], device="cuda"))
    assert c.counter.tolist() == [0, 0]
    assert all(torch.equal(a, b) for a, b in zip(keep, c.params + [m for m in c.masters if m is not None]))
    after = c.before()
    assert all(np.array_equal(a, b) for x, y in zip(before, after) for a, b in zip(x, y))
    c.step([0.1] * len(c.specs))   # and the next step is the first
    c.check(before, 1, [0.1] * len(c.specs))


@pytest.mark.parametrize("bits", [8, 32])
def test_infinite_gradients_stay_in_their_block(bits):
    c = Case(8, [(1000, "bf16", "bf16", bits, False)])
    c.grads[0][200] = float("inf")
    c.grads[0][700] = float("nan")
    c.step(0.0)
    x, state = c.params[0].float(), c.states[0]
    assert not torch.isfinite(x[700])
    if bits == 8:
        assert state.v.scales.view(-1)[1] == 255 and state.v.scales.view(-1)[5] == 255
        assert (state.v.scales.view(-1)[[0, 2, 3, 4, 6, 7]] != 255).all()
    fine = torch.ones(1000, dtype=torch.bool, device="cuda")
    fine[[200, 700]] = False
    assert torch.isfinite(x[fine]).all()


def test_no_elements_count_the_step():
    c = Case(9, [(0, "bf16", "f32", 8, False)])
    c.step(0.0)
    assert c.counter.tolist() == [1, 0]
    taco.taco_adamw([], [], [], c.counter, lr=1e-3)
    assert c.counter.tolist() == [2, 0]


def test_captured_steps_go_on_counting():
    specs = [(5000, "bf16", "f32", 8, False), (4097, "f32", "f32", 32, False), (777, "f16", "f16", 8, True)]
    c, d = Case(10, specs), Case(10, specs)
    rate, scale = torch.tensor([1e-2], device="cuda"), torch.tensor([1.0], device="cuda")
    graph = torch.cuda.CUDAGraph()
    warm = Case(11, specs)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        warm.step(0.1)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.step(0.1, lr=rate, grad_scale=scale)
    assert c.counter.tolist() == [0, 0]
    for t, (r, f) in enumerate([(1e-2, 1.0), (2e-2, 0.5), (5e-3, 0.25)], 1):
        rate.fill_(r)
        scale.fill_(f)
        graph.replay()
        d.step(0.1, lr=rate, grad_scale=scale)
        assert c.counter.tolist() == d.counter.tolist() == [t, 0]
        for a, b in zip(c.params, d.params):
            assert torch.equal(a, b)
        for a, b in zip(c.before(), d.before()):
            assert all(np.array_equal(x, y) for x, y in zip(a, b))


def test_repeated_calls_are_equal_bit_for_bit_and_streams_are_followed():
    specs = [(300001, "bf16", "f32", 8, False), (65536, "f16", "f16", 32, False)]
    c, d = Case(12, specs), Case(12, specs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        c.step(0.1)
        d.step(0.1, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(c.params, d.params):
        assert torch.equal(a, b)
    for a, b in zip(c.before(), d.before()):
        assert all(np.array_equal(x, y) for x, y in zip(a, b))


def test_small_changes_are_kept_on_average():
    """Roots whose target lies far above: each step moves them by a fiftieth of a
    code's step or less, so rounding to nearest would leave them where they
    started. A threshold sequence keeps their mean within a code's step (2^-3)
    of the exact moment's root, and so do bf16 parameters under a small rate."""
    n, steps = 16384, 300
    p = torch.full((n,), 1.0, dtype=torch.bfloat16, device="cuda")
    g = torch.full((n,), 1.0, device="cuda")
    c, e = Q.quantize(np.full((1, n), 0.5))
    m = taco.Fp8Tensor(torch.from_numpy(c).cuda(), torch.from_numpy(e).cuda())
    state = taco.AdamState(m, taco.Fp8Tensor(m.codes.clone(), m.scales.clone()))
    counter = torch.tensor([10 ** 6, 0], dtype=torch.int32, device="cuda")
    lr = 1e-5
    for _ in range(steps):
        taco.taco_adamw([p], [g], [state], counter, lr=lr, betas=(0.9, 0.999), weight_decay=0.0)
    v, x, mm = 0.25, 1.0, 0.5
    for _ in range(steps):
        mm = 0.9 * mm + 0.1
        v = 0.999 * v + 0.001
        x -= lr * mm / v ** 0.5
    root = O.state_values(*codes_of(state.v))
    assert abs(root.mean() / v ** 0.5 - 1) < 2 ** -5
    assert root.std() / root.mean() < 2 ** -3
    assert abs(float(p.double().mean()) - x) < 0.1 * (1 - x)


def test_roots_that_are_not_zero_keep_a_code():
    g = torch.zeros(128, device="cuda")
    g[0], g[1] = 1.0, 1e-7
    p = torch.zeros(128, device="cuda")
    state = taco.taco_adam_state(p, 8)
    counter = torch.zeros(2, dtype=torch.int32, device="cuda")
    for _ in range(5):
        taco.taco_adamw([p], [g], [state], counter, lr=1.0, weight_decay=0.0)
        codes = state.v.codes.view(-1)
        assert codes[0] > 1 and codes[1] == 1 and (codes[2:] == 0).all()
    assert p[1].abs() < 5


@pytest.mark.parametrize("bits", [8, 32])
def test_offsets_past_32_bits(bits):
    n = 2 ** 31 + 4096 + 5
    if torch.cuda.mem_get_info()[0] < n * 16:
        pytest.skip("memory")
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    tail = 4096 + 200
    a = torch.randn(tail, device="cuda").bfloat16()
    d = torch.randn(tail, device="cuda").bfloat16()
    p[-tail:] = a
    g[-tail:] = d
    state = taco.taco_adam_state(p, bits)
    counter = torch.zeros(2, dtype=torch.int32, device="cuda")
    taco.taco_adamw([p], [g], [state], counter, weight_decay=0.0, **KW)
    x, m, v, update, _ = O.adamw(f64(a), f64(d), 0.0, 0.0, 1, KW["lr"], *KW["betas"], KW["eps"], 0.0)
    dx = 8 * U * np.abs(f64(a)) + 64 * U * np.abs(update)
    w = O.thresholds(tail, 1, n - tail)
    got = f64(p[-tail:])
    ends = [O.by_threshold(x + s * dx, w, "bf16") for s in (-1, 1)]
    assert ((got >= ends[0]) & (got <= ends[1])).all()
    assert not p[: 10 ** 6].any() and not p[2 ** 31 - 10 ** 6: 2 ** 31 - 300].any()
    if bits == 32:
        assert np.abs(f64(state.m[-tail:]) - m).max() < 1e-6
    else:
        m8 = state.m.codes.view(-1)[-tail:].view(torch.float8_e4m3fn).double()
        s = state.m.scales.view(-1).view(torch.float8_e8m0fnu)[-((tail + 127) // 128 + 1):].double()
        at = (torch.arange(n - tail, n, device="cuda") // 128) - ((n + 127) // 128 - s.numel())
        have = (m8 * s[at]).cpu().numpy()
        assert (np.abs(have - m) <= 2.0 ** -3 * np.abs(m) + 2.0 ** -8 * np.abs(m).max()).all()


def test_statuses_become_errors():
    c = Case(13, [(100, "bf16", "f32", 32, False)])
    for kw in (dict(betas=(1.0, 0.9)), dict(eps=0.0), dict(lr=float("nan"))):
        with pytest.raises(taco.TacoError):
            c.step(0.0, **kw)
    with pytest.raises(taco.TacoError):     # the parameter itself
        taco.taco_adamw(c.params, c.params, c.states, c.counter, lr=1e-3)
    with pytest.raises(taco.TacoError):     # twice in a call
        taco.taco_adamw(c.params * 2, c.grads * 2, c.states * 2, c.counter, lr=1e-3)
    with pytest.raises(taco.TacoError):
        taco.taco_grad_norm(c.grads, max_norm=-1.0)
    assert c.counter.tolist() == [0, 0]
