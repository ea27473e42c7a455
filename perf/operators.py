"""Measured cases of the FP8 block-tensor operators.

An FP8 block tensor [R, C] is a pair: E4M3 codes (uint8) and one E8M0 scale
byte b (scale 2^(b - 127)) per row and 128 columns, or per 128 x 128 tile for
weights. The operators that make and read it:

  quantize   a tensor to FP8 blocks, its rows, its transpose or both; the
             source may itself be an FP8 block tensor (a checkpoint re-blocked
             along the tokens for the weight gradient)
  norm       residual addition and root-mean-square norm with the 8-bit output
             the next matrix product reads and an 8-bit checkpoint of the sum;
             its backward pass from that checkpoint
  swiglu     silu(gate) * up with an 8-bit output and 8-bit checkpoints of gate
             and up; its backward pass from the checkpoints
  matmul     C = A B^T of two FP8 block tensors (forward, gradients, single
             tokens)

``run`` computes each in its plain form (elementary torch operations in
32 bits), or with ``own`` through the package's entry points.
"""

import math

import torch

own = False

BLOCK = 128
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # A few sequences answering token by token: one norm before a linear layer; all latency.
        dict(name="norm_tokens", op="norm", M=4, H=4096, type="bf16", residual=True, checkpoint=False),
        # A training step's norm over a long batch, the sum kept in 8 bits for the backward pass.
        dict(name="norm_train", op="norm", M=16384, H=3584, type="bf16", residual=True, checkpoint=True),
        # The backward pass of such a norm, with the residual stream's own gradient added.
        dict(name="norm_backward", op="norm_bwd", M=8192, H=4096, type="bf16", dh=True),
        # A ragged batch with rows that end inside a block of 128, in 16-bit floats, no residual.
        dict(name="norm_backward_odd", op="norm_bwd", M=1023, H=1600, type="f16", dh=False),
        # One rank's gated activation in a training step, checkpointed in 8 bits.
        dict(name="swiglu_train", op="swiglu", M=16384, F=4096, type="bf16", checkpoint=True),
        # Its backward pass from the checkpoints.
        dict(name="swiglu_backward", op="swiglu_bwd", M=16384, F=4096, type="bf16"),
        # A small ragged chunk of a prompt.
        dict(name="swiglu_odd", op="swiglu", M=257, F=1000, type="bf16", checkpoint=False),
        # An output gradient quantised both ways: rows for the input's gradient, columns for the weight's.
        dict(name="quantize_gradient", op="quantize", M=8192, K=4096, type="bf16", rows=True, cols=True, tile=1),
        # A checkpoint re-blocked along the tokens for the weight gradient.
        dict(name="reblock_checkpoint", op="quantize", M=8192, K=1600, type="fp8", rows=False, cols=True, tile=1),
        # Single tokens of a few sequences through a linear layer: the weight's bytes.
        dict(name="matmul_tokens", op="matmul", M=8, N=4096, K=4096, tile=128, type="bf16", add=False),
        # A linear layer's forward pass over a long batch.
        dict(name="matmul_train", op="matmul", M=16384, N=4096, K=3584, tile=128, type="bf16", add=False),
        # A weight gradient added to the 32-bit running one, over a ragged number of tokens.
        dict(name="matmul_weight_grad", op="matmul", M=1600, N=4096, K=8190, tile=1, type="f32", add=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width of the kinds that models have: mostly multiples of 64, some of 8, some odd."""
    w = _log(rng, lo, hi)
    kind = rng.random()
    step = 64 if kind < 0.6 else 8 if kind < 0.85 else 1
    return max(step, w // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "swiglu", "swiglu_bwd", "quantize", "matmul", "matmul"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    M = _log(rng, 1, 16384)
    if op == "norm":
        return dict(op=op, M=M, H=_width(rng, 256, 8192), type=dtype, residual=rng.random() < 0.7,
                    checkpoint=rng.random() < 0.5)
    if op == "norm_bwd":
        return dict(op=op, M=M, H=_width(rng, 256, 8192), type=dtype, dh=rng.random() < 0.7)
    if op == "swiglu":
        return dict(op=op, M=M, F=_width(rng, 128, 8192), type=dtype, checkpoint=rng.random() < 0.7)
    if op == "swiglu_bwd":
        return dict(op=op, M=M, F=_width(rng, 128, 8192), type=dtype)
    if op == "quantize":
        kind = rng.choice(["rows", "cols", "both", "fp8", "weight"])
        return dict(op=op, M=M, K=_width(rng, 128, 8192), type="fp8" if kind == "fp8" else dtype,
                    rows=kind not in ("cols", "fp8"), cols=kind != "rows", tile=128 if kind == "weight" else 1)
    while True:
        M, N, K = _log(rng, 1, 16384), _width(rng, 128, 16384), _width(rng, 128, 16384)
        if M * N * K <= 16384 * 4096 * 3584:
            break
    grad = rng.random() < 0.3
    return dict(op=op, M=M, N=N, K=K, tile=1 if grad else 128, type="f32" if grad else rng.choice(["bf16", "f16"]),
                add=grad)


# ----------------------------------------------------------------- plain form
def _scale_exponent(amax):
    """Exponent of the smallest power of two >= amax / 448, at least -126; 0 for an all-zero block."""
    m, x = torch.frexp(amax)
    e = torch.where(m > 0.875, x - 8, x - 9).clamp(min=-126)
    return torch.where(amax == 0, torch.zeros_like(e), e)


def _blocks(x):
    """[R, C] -> [R, ceil(C / 128), 128], zero-filled."""
    R, C = x.shape
    kb = -(-C // BLOCK)
    return torch.nn.functional.pad(x, (0, kb * BLOCK - C)).view(R, kb, BLOCK)


def _quantize(x, tile=1):
    """fp32 [R, C] -> (codes as float8_e4m3fn [R, C], scales as float8_e8m0fnu)."""
    R, C = x.shape
    b = _blocks(x)
    amax = b.abs().amax(dim=2)
    if tile == BLOCK:
        rb = -(-R // BLOCK)
        amax = torch.nn.functional.pad(amax, (0, 0, 0, rb * BLOCK - R)).view(rb, BLOCK, -1).amax(dim=1)
    e = _scale_exponent(amax)
    rows = e.repeat_interleave(BLOCK, dim=0)[:R] if tile == BLOCK else e
    q = torch.ldexp(b, -rows[:, :, None])
    codes = q.view(R, -1)[:, :C].to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _dequantize(t):
    codes, scales = t
    R, C = codes.shape
    s = scales.view(torch.float8_e8m0fnu).float()
    if s.shape[0] != R:
        s = s.repeat_interleave(BLOCK, dim=0)[:R]
    return codes.view(torch.float8_e4m3fn).float() * s.repeat_interleave(BLOCK, dim=1)[:, :C]


def _values(t):
    """An FP8 block tensor's codes and scales as the values they stand for."""
    return None if t is None else [t[0].view(torch.float8_e4m3fn), t[1].view(torch.float8_e8m0fnu)]


def _run_plain(s):
    op, dtype = s["op"], s["dtype"]
    if op == "norm":
        x = s["x"].float()
        h = (x + s["residual"].float()).to(dtype) if s["residual"] is not None else s["x"]
        hf = h.float()
        rstd = torch.rsqrt(hf.square().mean(dim=1) + EPS)
        y = hf * rstd[:, None] * s["weight"].float()
        return [list(_quantize(y)), h, rstd, list(_quantize(hf)) if s["checkpoint"] else None]
    if op == "norm_bwd":
        rstd = s["rstd"][:, None]
        xh = _dequantize(s["ckpt"]) * rstd
        dy = s["dy"].float()
        g = dy * s["weight"].float()
        dx = rstd * (g - xh * (g * xh).mean(dim=1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return [dx.to(dtype), (dy * xh).sum(dim=0)]
    if op == "swiglu":
        g, u = s["gate_up"].float().chunk(2, dim=1)
        y = list(_quantize(g / (1 + torch.exp(-g)) * u))
        return [y, [list(_quantize(g)), list(_quantize(u))] if s["checkpoint"] else None]
    if op == "swiglu_bwd":
        g, u = (_dequantize((s["ckpt"][0][i], s["ckpt"][1][i])) for i in (0, 1))
        dy = s["dy"].float()
        sig = 1 / (1 + torch.exp(-g))
        return torch.cat([dy * u * sig * (1 + g * (1 - sig)), dy * g * sig], dim=1).to(dtype)
    if op == "quantize":
        x = _dequantize(s["x"]) if isinstance(s["x"], tuple) else s["x"].float()
        return [list(_quantize(x, s["tile"])) if s["rows"] else None,
                list(_quantize(x.t().contiguous(), s["tile"])) if s["cols"] else None]
    c = _dequantize(s["a"]) @ _dequantize(s["b"]).t()
    return (c + s["add"] if s["add"] is not None else c).to(dtype)


# ------------------------------------------------------------------ framework
def _run_own(s):
    import grads_taco_compress_gb300 as taco

    op = s["op"]
    if op == "norm":
        r = taco.taco_rms_norm_fp8(s["x"], s["weight"], s["residual"], EPS, checkpoint=s["checkpoint"])
        return [_values(r.y), r.h, r.rstd, _values(r.checkpoint)]
    if op == "norm_bwd":
        return list(taco.taco_rms_norm_fp8_backward(s["dy"], taco.Fp8Tensor(*s["ckpt"]), s["weight"], s["rstd"],
                                                    dh=s["dh"]))
    if op == "swiglu":
        y, c = taco.taco_swiglu_fp8(s["gate_up"], checkpoint=s["checkpoint"])
        return [_values(y), None if c is None else [_values((c.codes[i], c.scales[i])) for i in (0, 1)]]
    if op == "swiglu_bwd":
        return taco.taco_swiglu_fp8_backward(s["dy"], taco.Fp8Tensor(*s["ckpt"]))
    if op == "quantize":
        x = taco.Fp8Tensor(*s["x"]) if isinstance(s["x"], tuple) else s["x"]
        q, t = taco.taco_fp8_quantize(x, rows=s["rows"], cols=s["cols"], tile=s["tile"])
        return [_values(q), _values(t)]
    return taco.taco_matmul_fp8(taco.Fp8Tensor(*s["a"]), taco.Fp8Tensor(*s["b"]), out_dtype=s["dtype"], add=s["add"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------- inputs
def _padded(t, multiple):
    """A uint8 tensor's copy whose rows start at multiples of `multiple` bytes."""
    C = t.shape[-1]
    p = torch.zeros(*t.shape[:-1], -(-C // multiple) * multiple, dtype=torch.uint8, device=t.device)
    p[..., :C] = t.view(torch.uint8)
    return p[..., :C]


def _held(pair):
    """An FP8 block tensor as a program holds it: rows of codes on 16 bytes, rows of scales on 4."""
    return _padded(pair[0], 16), _padded(pair[1], 4)


def _activations(gen, M, C, dtype):
    """Heavy-tailed values with a scale for each channel and a few massive channels."""
    u = torch.rand(M, C, generator=gen, device="cuda") - 0.5
    x = -0.05 * u.sign() * torch.log1p(-1.998 * u.abs())
    x *= torch.exp(0.5 * torch.randn(C, generator=gen, device="cuda"))
    x[:, torch.randint(0, C, (max(1, C // 512),), generator=gen, device="cuda")] *= 30
    return x.to(dtype)


def _gradients(gen, M, C, dtype):
    """Small values with rare spikes and some exact zeros."""
    x = 1e-3 * torch.randn(M, C, generator=gen, device="cuda")
    r = torch.rand(M, C, generator=gen, device="cuda")
    x = torch.where(r < 0.001, 50 * x, x)
    return torch.where(r > 0.95, torch.zeros_like(x), x).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    dtype = TYPES.get(case["type"], torch.bfloat16)
    s = dict(op=op, dtype=dtype)
    if op in ("norm", "norm_bwd"):
        M, H = case["M"], case["H"]
        s["weight"] = (1 + 0.2 * torch.randn(H, generator=gen, device="cuda")).to(dtype)
        if op == "norm":
            s["x"] = _activations(gen, M, H, dtype)
            s["residual"] = _activations(gen, M, H, dtype) if case["residual"] else None
            s["checkpoint"] = case["checkpoint"]
        else:
            h = _activations(gen, M, H, dtype).float()
            s["ckpt"] = _held(_quantize(h))
            s["rstd"] = torch.rsqrt(h.square().mean(dim=1) + EPS)
            s["dy"] = _gradients(gen, M, H, dtype)
            s["dh"] = _gradients(gen, M, H, dtype) if case["dh"] else None
    elif op in ("swiglu", "swiglu_bwd"):
        M, F = case["M"], case["F"]
        gate_up = 10 * _activations(gen, M, 2 * F, dtype)
        if op == "swiglu":
            s["gate_up"] = gate_up
            s["checkpoint"] = case["checkpoint"]
        else:
            pairs = [_quantize(t) for t in gate_up.float().chunk(2, dim=1)]
            s["ckpt"] = _held([torch.stack([p[i].view(torch.uint8) for p in pairs]) for i in (0, 1)])
            s["dy"] = _gradients(gen, M, F, dtype)
    elif op == "quantize":
        M, K = case["M"], case["K"]
        s.update(rows=case["rows"], cols=case["cols"], tile=case["tile"])
        if case["type"] == "fp8":
            s["x"] = _held(_quantize(_activations(gen, M, K, dtype).float()))
        else:
            s["x"] = _gradients(gen, M, K, dtype)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        if case["add"]:
            # both operands run along the tokens: an output gradient and a checkpointed input
            s["a"] = _held(_quantize(_gradients(gen, M, K, torch.float32)))
            s["b"] = _held(_quantize(_activations(gen, N, K, torch.float32)))
            s["add"] = 0.01 * torch.randn(M, N, generator=gen, device="cuda")
        else:
            s["a"] = _held(_quantize(_activations(gen, M, K, torch.float32)))
            s["b"] = _held(_quantize(0.02 * torch.randn(N, K, generator=gen, device="cuda"), case["tile"]))
            s["add"] = None
    return s


# ----------------------------------------------------------------------- work
def _fp8_bytes(R, C, tile=1):
    return R * C + -(-R // tile) * -(-C // BLOCK)


def work(case):
    op = case["op"]
    b = SIZE.get(case["type"], 2)
    M = case["M"]
    if op == "norm":
        H = case["H"]
        n = M * H
        return dict(bytes=n * b * (3 if case["residual"] else 1) + H * b + 4 * M
                    + _fp8_bytes(M, H) * (2 if case["checkpoint"] else 1), flops=10 * n)
    if op == "norm_bwd":
        H = case["H"]
        return dict(bytes=M * H * b * (3 if case["dh"] else 2) + _fp8_bytes(M, H) + H * (b + 4) + 4 * M,
                    flops=12 * M * H)
    if op == "swiglu":
        F = case["F"]
        return dict(bytes=2 * M * F * b + _fp8_bytes(M, F) * (3 if case["checkpoint"] else 1), flops=10 * M * F)
    if op == "swiglu_bwd":
        F = case["F"]
        return dict(bytes=3 * M * F * b + 2 * _fp8_bytes(M, F), flops=16 * M * F)
    if op == "quantize":
        K, t = case["K"], case["tile"]
        source = _fp8_bytes(M, K) if case["type"] == "fp8" else M * K * b
        return dict(bytes=source + (_fp8_bytes(M, K, t) if case["rows"] else 0)
                    + (_fp8_bytes(K, M, t) if case["cols"] else 0), flops=4 * M * K)
    N, K = case["N"], case["K"]
    return dict(bytes=_fp8_bytes(M, K) + _fp8_bytes(N, K, case["tile"]) + M * N * b * (2 if case["add"] else 1),
                flops=2 * M * N * K)


# ------------------------------------------------------- definition in 64 bits
def _round_e4m3(v):
    """Nearest E4M3 value (ties to even) of |v| <= 448."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _quantize64(x, tile=1):
    R, C = x.shape
    rb, cb = -(-R // tile), -(-C // BLOCK)
    padded = torch.zeros(rb * tile, cb * BLOCK, dtype=torch.float64, device=x.device)
    padded[:R, :C] = x
    grid = padded.view(rb, tile, cb, BLOCK)
    amax = grid.abs().amax(dim=(1, 3))
    scale = torch.exp2(torch.ceil(torch.log2(amax / 448)).clamp(min=-126))
    # log2 may round to the wrong side of a whole number: step to the smallest power that holds amax
    scale = torch.where(scale * 448 < amax, scale * 2, scale)
    scale = torch.where((scale * 224 >= amax) & (scale > 2.0 ** -126), scale / 2, scale)
    scale = torch.where(amax == 0, torch.ones_like(scale), scale)
    values = _round_e4m3(grid / scale[:, None, :, None]).reshape(rb * tile, cb * BLOCK)[:R, :C]
    return [values, scale]


def _dequantize64(codes, scales):
    R, C = codes.shape
    table = torch.arange(256, device=codes.device)
    sign = 1.0 - 2.0 * (table >> 7)
    e, m = (table >> 3) & 15, (table & 7).double()
    value = sign * torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))
    scale = torch.exp2(scales.double() - 127)
    rows = torch.arange(R, device=codes.device) // (1 if scales.shape[0] == R else BLOCK)
    cols = torch.arange(C, device=codes.device) // BLOCK
    return value[codes.long()] * scale[rows][:, cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(s["dtype"]).double()
        rstd = 1 / torch.sqrt((h * h).sum(dim=1) / h.shape[1] + EPS)
        return [_quantize64(h * rstd[:, None] * s["weight"].double()), h, rstd,
                _quantize64(h) if s["checkpoint"] else None]
    if op == "norm_bwd":
        r = s["rstd"].double()[:, None]
        n = _dequantize64(*s["ckpt"]) * r
        dy, w = s["dy"].double(), s["weight"].double()
        along = (dy * w * n).sum(dim=1, keepdim=True) / n.shape[1]
        dx = r * (dy * w) - r * along * n
        return [dx if s["dh"] is None else dx + s["dh"].double(), torch.einsum("mh,mh->h", dy, n)]
    if op == "swiglu":
        F = s["gate_up"].shape[1] // 2
        g, u = s["gate_up"][:, :F].double(), s["gate_up"][:, F:].double()
        return [_quantize64(g * torch.sigmoid(g) * u), [_quantize64(g), _quantize64(u)] if s["checkpoint"] else None]
    if op == "swiglu_bwd":
        g, u = (_dequantize64(s["ckpt"][0][i], s["ckpt"][1][i]) for i in (0, 1))
        dy, sig = s["dy"].double(), torch.sigmoid(g)
        silu = g * sig
        return torch.cat([dy * u * (sig + silu * (1 - sig)), dy * silu], dim=1)
    if op == "quantize":
        x = _dequantize64(*s["x"]) if isinstance(s["x"], tuple) else s["x"].double()
        return [_quantize64(x, s["tile"]) if s["rows"] else None,
                _quantize64(x.t(), s["tile"]) if s["cols"] else None]
    c = torch.einsum("mk,nk->mn", _dequantize64(*s["a"]), _dequantize64(*s["b"]))
    return c + s["add"].double() if s["add"] is not None else c
