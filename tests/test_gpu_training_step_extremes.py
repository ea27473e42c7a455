"""The layer's product, its gradient and the optimiser's step beyond 32-bit
offsets, and two of each at once on two streams."""

from __future__ import annotations

import pytest
import torch

import grads_taco_compress_gb300 as taco
from grads_taco_compress_gb300 import binding as tb

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def same(a, b):
    return torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


def rows(t, a, b):
    return taco.Fp8Tensor(t.codes[a:b], t.scales[a:b])


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def need(gb):
    if torch.cuda.mem_get_info()[0] < gb * 2 ** 30:
        pytest.skip("memory")


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_layer_beyond_32_bits(kind):
    """Rows at the end of an output of more than 2^32 elements: those of the same
    product on these rows alone."""
    need(40)
    M, N, K, tail = 2 ** 18 + 300, 16416, 256, 556
    x, _ = taco.taco_fp8_quantize(torch.randn(M, K, device="cuda").bfloat16())
    w, _ = taco.taco_fp8_quantize(torch.randn(N, K, device="cuda").bfloat16(), tile=128)
    bias = torch.randn(N, device="cuda").bfloat16()
    args = dict(bias=bias, activation="silu", checkpoint=True, out_dtype=F8 if kind == "fp8" else torch.bfloat16)
    y, kept = taco.taco_linear_fp8(x, w, **args)
    for a, b in ((M - tail, M), (0, 256), (2 ** 32 // N - 100, 2 ** 32 // N + 300)):
        e, k = taco.taco_linear_fp8(rows(x, a, b), w, **args)
        assert same(rows(kept, a, b), k)
        assert same(rows(y, a, b), e) if kind == "fp8" else torch.equal(y[a:b], e)
    assert tb.taco_get_fault() == 0


def test_gradient_beyond_32_bits():
    need(60)
    M, N = 2 ** 18 + 200, 16416
    dy = torch.randn(1024, N, device="cuda").bfloat16().repeat(-(-M // 1024), 1)[:M]
    kept, _ = taco.taco_fp8_quantize(dy)
    q, t, db = taco.taco_linear_fp8_backward(dy, kept, "gelu")
    for a in (0, 2 ** 32 // N // 128 * 128, M // 128 * 128):
        b = min(a + 256, M)
        e, et, _ = taco.taco_linear_fp8_backward(dy[a:b], rows(kept, a, b), "gelu")
        assert same(rows(q, a, b), e)
        assert torch.equal(t.codes[:, a:b], et.codes) and torch.equal(t.scales[:, a // 128:-(-b // 128)], et.scales)
    # 256 whole repetitions and 200 rows more
    one, rest = (taco.taco_linear_fp8_backward(dy[:n], rows(kept, 0, n), "gelu", rows=False, cols=False)[2].double()
                 for n in (1024, 200))
    want = 256 * one + rest
    # 2^-24 a rounding, 26 + M / 1024 of them at most on sums that are at most sqrt(M) deviations of 1.2
    assert (db.double() - want).abs().max() < (26 + M / 1024) * 2.0 ** -24 * 1.2 * M


def test_two_at_once():
    """Calls on two streams with tensors of their own: what they give one by one."""
    def work(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        x, _ = taco.taco_fp8_quantize(rand(700, 640).bfloat16())
        w, _ = taco.taco_fp8_quantize(rand(900, 640).bfloat16(), tile=128)
        b, dy = rand(900), rand(700, 900).bfloat16()
        p, gr = [rand(70001).bfloat16(), rand(4099)], [rand(70001), rand(4099)]
        opt = taco.AdamW(p, lr=1e-2, bits=8)

        def run(stream=None):
            y, kept = taco.taco_linear_fp8(x, w, b, "gelu", out_dtype=F8, checkpoint=True, stream=stream)
            d, dt, db = taco.taco_linear_fp8_backward(dy, kept, "gelu", stream=stream)
            norm = opt.step(gr, max_norm=1.0, stream=stream)
            return [y.codes, y.scales, kept.codes, d.codes, d.scales, dt.codes, dt.scales, db, norm.clone()]
        return run, p

    once = []
    for seed in (1, 2):
        run, p = work(seed)
        once.append([run() for _ in range(8)][-1][:-1] + p)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    jobs = [work(seed) for seed in (1, 2)]
    torch.cuda.synchronize()
    out = [None, None]
    for _ in range(8):
        for i, (run, _) in enumerate(jobs):
            out[i] = run(streams[i])
    torch.cuda.synchronize()
    for i, (_, p) in enumerate(jobs):
        for a, b in zip(out[i][:-1] + p, once[i]):
            assert torch.equal(a, b)
    assert tb.taco_get_fault() == 0
