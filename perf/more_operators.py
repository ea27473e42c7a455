"""Measured cases of the operators of a training step around the FP8 products.

  linear         y = act(x W^T + bias) + residual of two FP8 block tensors, in
                 16 or 32 bits or as an FP8 block tensor, with the values in
                 front of the activation kept in 8 bits for the backward pass
  linear_bwd     the gradient at the product's output, dy act'(kept), as the
                 FP8 operands of the two products that follow (its rows, its
                 transpose), and the bias's gradient
  grad_norm      the norm of all gradients of a model and the factor that
                 clips it
  adamw          an AdamW step over many tensors at once, states in 32 bits or
                 in FP8 blocks (the second moment as its square root)

An FP8 block tensor [R, C] is a pair: E4M3 codes (uint8) and one E8M0 scale
byte b (scale 2^(b - 127)) per row and 128 columns, or per 128 x 128 tile for
weights. States in 8 bits are block tensors of one row, [1, n].

What is rounded to 8 bits, or to a 16-bit parameter that has no 32-bit master,
in an AdamW step is rounded up or down by a threshold that runs through a Weyl
sequence over steps and elements, so that changes far below half a step of the
type are kept on average:
    u = frac(i 0xC13FA9A9 / 2^32 + t 0x9E3779B1 / 2^32),   element i, step t
    |x| -> step floor(|x| / step + u),  step: the type's at |x|
A second moment that is not zero is never rounded to zero.

``run`` computes each in its plain form (elementary torch operations in
32 bits), or with ``own`` through the package's entry points.
"""

import math

import torch

own = False

BLOCK = 128
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "fp8": 1}
BETA1, BETA2, EPS, DECAY, LR = 0.9, 0.95, 1e-8, 0.1, 3e-4
WEYL_I, WEYL_T = 0xC13FA9A9, 0x9E3779B1
VECTOR = 32768   # parameters with fewer elements are norm weights and biases: 32 bits, no decay


def listed():
    return [
        # A few sequences answering token by token through a biased layer: one launch's latency.
        dict(name="linear_tokens", op="linear", M=8, N=6400, K=1600, type="fp8", act="gelu_tanh", residual=False,
             keep=False),
        # The first layer of a biased MLP in a training step, everything that leaves it in 8 bits.
        dict(name="linear_train", op="linear", M=8192, N=16384, K=4096, type="fp8", act="gelu_tanh", residual=False,
             keep=True),
        # Its second layer, with the residual stream added.
        dict(name="linear_residual", op="linear", M=8192, N=4096, K=16384, type="bf16", act="none", residual=True,
             keep=False),
        # A ragged batch through a layer of odd widths, with 32-bit outputs.
        dict(name="linear_odd", op="linear", M=777, N=2806, K=1000, type="f32", act="silu", residual=True, keep=True),
        # Backward through the activation of a training step.
        dict(name="linear_backward", op="linear_bwd", M=8192, N=16384, type="bf16", act="gelu_tanh"),
        # A ragged output gradient and the bias's, no activation.
        dict(name="bias_backward_odd", op="linear_bwd", M=1023, N=1600, type="f16", act="none"),
        # All gradients of one layer's MLP, running 32-bit sums.
        dict(name="grad_norm_layer", op="grad_norm", sizes="67108864,67108864,16384,4096,4096", grad="f32"),
        # Norm weights and biases of a model's layers, odd lengths: latency over many tensors.
        dict(name="grad_norm_vectors", op="grad_norm", sizes=",".join(["1600,1600,6400,1601"] * 24), grad="bf16"),
        # The same vectors stepped, all in 32 bits.
        dict(name="adamw_vectors", op="adamw", sizes=",".join(["1600,1600,6400,1601"] * 24), type="f32", grad="f32",
             bits=32, master=False),
        # One layer's MLP stepped with 32-bit states and masters.
        dict(name="adamw_layer_32", op="adamw", sizes="67108864,67108864,16384,4096,4096", type="bf16", grad="f32",
             bits=32, master=True),
        # The same with states in 8 bits and no masters.
        dict(name="adamw_layer_8", op="adamw", sizes="67108864,67108864,16384,4096,4096", type="bf16", grad="f32",
             bits=8, master=False),
        # A few ragged tensors, 16-bit gradients.
        dict(name="adamw_odd_8", op="adamw", sizes="2565001,10240000,1601,777,129,1,5120003", type="bf16",
             grad="bf16", bits=8, master=False),
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
    op = rng.choice(["linear", "linear", "linear_bwd", "grad_norm", "adamw", "adamw"])
    act = rng.choice(["none", "gelu", "gelu_tanh", "gelu_tanh", "silu", "relu"])
    if op == "linear":
        while True:
            M, N, K = _log(rng, 1, 16384), _width(rng, 128, 16384), _width(rng, 128, 16384)
            if M * N * K <= 8192 * 16384 * 4096:
                break
        kind = rng.choice(["fp8", "fp8", "bf16", "f16", "f32"])
        return dict(op=op, M=M, N=N, K=K, type=kind, act=act, residual=kind != "fp8" and rng.random() < 0.6,
                    keep=rng.random() < 0.5)
    if op == "linear_bwd":
        return dict(op=op, M=_log(rng, 1, 8192), N=_width(rng, 128, 16384), type=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    act=act)
    total, count = _log(rng, 2000, 134217728), _log(rng, 1, 300)
    cuts = sorted(rng.random() for _ in range(count - 1))
    sizes = ",".join(str(max(1, int((b - a) * total))) for a, b in zip([0.0] + cuts, cuts + [1.0]))
    if op == "grad_norm":
        return dict(op=op, sizes=sizes, grad=rng.choice(["f32", "bf16", "f16"]))
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    return dict(op=op, sizes=sizes, type=kind, grad=rng.choice(["f32", kind]), bits=rng.choice([8, 32]),
                master=kind != "f32" and rng.random() < 0.5)


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


def _pair(q, e, C):
    """Scaled values and exponents -> (codes as float8_e4m3fn, scales as float8_e8m0fnu)."""
    return [q.view(q.shape[0], -1)[:, :C].to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)]


def _quantize(x, tile=1):
    """fp32 [R, C] -> (codes, scales), to nearest."""
    R, C = x.shape
    b = _blocks(x)
    amax = b.abs().amax(dim=2)
    if tile == BLOCK:
        rb = -(-R // BLOCK)
        amax = torch.nn.functional.pad(amax, (0, 0, 0, rb * BLOCK - R)).view(rb, BLOCK, -1).amax(dim=1)
    e = _scale_exponent(amax)
    rows = e.repeat_interleave(BLOCK, dim=0)[:R] if tile == BLOCK else e
    return _pair(torch.ldexp(b, -rows[:, :, None]), e, C)


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


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _act(x, kind):
    if kind == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return x * _sigmoid(math.sqrt(8 / math.pi) * (x + 0.044715 * x * x * x))
    if kind == "silu":
        return x * _sigmoid(x)
    return x.clamp(min=0) if kind == "relu" else x


def _act_slope(x, kind):
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) * (1 / math.sqrt(2 * math.pi))
    if kind == "gelu_tanh":
        c = math.sqrt(8 / math.pi)
        s = _sigmoid(c * (x + 0.044715 * x * x * x))
        return s + x * s * (1 - s) * c * (1 + 3 * 0.044715 * x * x)
    if kind == "silu":
        s = _sigmoid(x)
        return s * (1 + x * (1 - s))
    return (x > 0).to(x.dtype)


def _thresholds(n, t, device):
    """Weyl thresholds of n elements at step t, whole numbers below 2^32."""
    return (torch.arange(n, device=device) * WEYL_I + t * WEYL_T) & 0xFFFFFFFF


def _dither(x, w, step):
    """x rounded by its threshold to a multiple of `step` (fp32, a power of two)."""
    a = x.abs() / step
    down = torch.floor(a)
    # the threshold's 20 bits against what lies between two multiples
    up = (a - down) + (w >> 12).float() * 2.0 ** -20 >= 1
    return torch.copysign((down + up.float()) * step, x)


def _step_of(x, bits, low):
    """Step of a float type with `bits` mantissa bits and smallest normal exponent `low` at x."""
    _, e = torch.frexp(x.abs())
    return torch.ldexp(torch.ones_like(x), torch.where(x == 0, low, e - 1).clamp(min=low) - bits)


def _to_state(x, w, root):
    """fp32 [n] -> FP8 blocks [1, n], rounded by thresholds."""
    n = x.shape[0]
    b = _blocks(x[None])
    e = _scale_exponent(b.abs().amax(dim=2))
    a = torch.ldexp(b, -e[:, :, None])
    q = _dither(a, _blocks(w[None]), _step_of(a, 3, -6))
    return _pair(torch.where((q == 0) & (a > 0), 2.0 ** -9, q) if root else q, e, n)


def _to_param(x, w, dtype):
    if dtype == torch.float32:
        return x
    return _dither(x, w, _step_of(x, 7, -126) if dtype == torch.bfloat16 else _step_of(x, 10, -14)).to(dtype)


def _adam_plain(s, i, t, factor):
    """One tensor's step in place."""
    p, g, m, v, master = s["params"][i], s["grads"][i], s["m"][i], s["v"][i], s["masters"][i]
    n = p.shape[0]
    w = _thresholds(n, t, p.device)
    x = (p if master is None else master).float()
    g = g.float() * factor
    small = s["bits"] == 8
    m0 = _dequantize(m)[0] if small else m
    v0 = _dequantize(v)[0].square() if small else v
    m1 = BETA1 * m0 + (1 - BETA1) * g
    v1 = BETA2 * v0 + (1 - BETA2) * g * g
    root = torch.sqrt(v1)
    c1, c2 = 1 - BETA1 ** t.double(), 1 - BETA2 ** t.double()
    x = x * (1 - LR * s["decay"][i]) - (LR / c1).float() * m1 / (root * c2.rsqrt().float() + EPS)
    if master is None:
        p.copy_(_to_param(x, w, p.dtype))
    else:
        master.copy_(x)
        p.copy_(x.to(p.dtype))
    if small:
        new = [_to_state(m1, w, False), _to_state(root, w, True)]
        [a.view(torch.uint8).copy_(b.view(torch.uint8)) for old, q in zip((m, v), new) for a, b in zip(old, q)]
    else:
        m.copy_(m1)
        v.copy_(v1)


def _state_values(s):
    """What a step leaves: parameters, masters, both states (first moments, then second), the number of steps."""
    return [s["all_params"], s["all_masters"], s["all_states"], s["counter"][:1]]


def _run_plain(s):
    op = s["op"]
    if op == "linear":
        pre = _dequantize(s["a"]) @ _dequantize(s["b"]).t() + s["bias"].float()
        y = _act(pre, s["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        y = _quantize(y) if s["dtype"] == torch.float8_e4m3fn else y.to(s["dtype"])
        return [y, _quantize(pre) if s["keep"] else None]
    if op == "linear_bwd":
        d = s["dy"].float()
        if s["kept"] is not None:
            d = d * _act_slope(_dequantize(s["kept"]), s["act"])
        return [_quantize(d), _quantize(d.t().contiguous()), d.sum(dim=0)]
    if op == "grad_norm":
        norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
        return torch.stack([norm, torch.where(norm > s["most"], s["most"] / norm, torch.ones_like(norm))])
    s["counter"][0] += 1
    [_adam_plain(s, i, s["counter"][0], s["factor"]) for i in range(len(s["params"]))]
    return _state_values(s)


# ------------------------------------------------------------------ framework
def _run_own(s):
    import grads_taco_compress_gb300 as taco

    op = s["op"]
    act = None if s.get("act") == "none" else s.get("act")
    if op == "linear":
        y, kept = taco.taco_linear_fp8(taco.Fp8Tensor(*s["a"]), taco.Fp8Tensor(*s["b"]), bias=s["bias"], activation=act,
                                       residual=s["residual"], out_dtype=s["dtype"], checkpoint=s["keep"])
        return [_values(y) if s["dtype"] == torch.float8_e4m3fn else y, _values(kept)]
    if op == "linear_bwd":
        kept = None if s["kept"] is None else taco.Fp8Tensor(*s["kept"])
        q, t, db = taco.taco_linear_fp8_backward(s["dy"], kept, activation=act)
        return [_values(q), _values(t), db]
    if op == "grad_norm":
        return taco.taco_grad_norm(s["grads"], max_norm=s["most"])
    small = s["bits"] == 8
    states = [taco.AdamState(taco.Fp8Tensor(*m), taco.Fp8Tensor(*v)) if small else taco.AdamState(m, v)
              for m, v in zip(s["m"], s["v"])]
    taco.taco_adamw(s["params"], s["grads"], states, s["counter"], lr=LR, betas=(BETA1, BETA2), eps=EPS,
                    weight_decay=s["decay"], grad_scale=s["factor"], masters=s["masters"])
    return _state_values(s)


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
    x = -0.5 * u.sign() * torch.log1p(-1.998 * u.abs())
    x *= torch.exp(0.5 * torch.randn(C, generator=gen, device="cuda"))
    x[:, torch.randint(0, C, (max(1, C // 512),), generator=gen, device="cuda")] *= 30
    return x.to(dtype)


def _gradients(gen, n, dtype):
    """Small values with rare spikes and some exact zeros."""
    x = 1e-3 * torch.randn(n, generator=gen, device="cuda")
    r = torch.rand(n, generator=gen, device="cuda")
    x = torch.where(r < 0.001, 50 * x, x)
    return torch.where(r > 0.95, torch.zeros_like(x), x).to(dtype)


def _sizes(case):
    return [int(n) for n in case["sizes"].split(",")]


def _param_type(case, n):
    return torch.float32 if n < VECTOR else TYPES[case["type"]]


def _grad_type(case, n):
    return torch.float32 if n < VECTOR and "type" in case else TYPES[case["grad"]]


def _in_buffers(tensors, multiple=512):
    """The tensors (None for one that there is not) as parts of one buffer for each type, each at a multiple of
    elements, and the buffers."""
    starts = [0]
    [starts.append(starts[-1] + (0 if t is None else -(-t.shape[0] // multiple) * multiple)) for t in tensors]
    kinds = sorted({t.dtype for t in tensors if t is not None}, key=str)
    buffers = {k: torch.zeros(starts[-1], dtype=k, device="cuda") for k in kinds}
    parts = [None if t is None else buffers[t.dtype][a:a + t.shape[0]].copy_(t) for t, a in zip(tensors, starts)]
    return parts, [buffers[k] for k in kinds]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    s = dict(op=op)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s.update(act=case["act"], keep=case["keep"], dtype=TYPES[case["type"]])
        s["a"] = _held(_quantize(_activations(gen, M, K, torch.float32)))
        s["b"] = _held(_quantize(randn(N, K) * K ** -0.5, BLOCK))
        s["bias"] = (0.5 * randn(N)).to(torch.float32 if case["type"] == "f32" else torch.bfloat16)
        s["residual"] = _activations(gen, M, N, s["dtype"]) if case["residual"] else None
    elif op == "linear_bwd":
        M, N = case["M"], case["N"]
        s["act"] = case["act"]
        s["dy"] = _gradients(gen, M * N, TYPES[case["type"]]).view(M, N)
        s["kept"] = _held(_quantize(_activations(gen, M, N, torch.float32))) if case["act"] != "none" else None
    else:
        sizes = _sizes(case)
        grads = [_gradients(gen, n, _grad_type(case, n)) for n in sizes]
        if op == "grad_norm":
            s["grads"] = grads
            s["most"] = 0.5e-3 * math.sqrt(sum(sizes))   # about a seventh of what the norm comes to
            return s
        s["bits"] = case["bits"]
        # values that have been trained for a thousand steps, each kind of them in one buffer
        w = [0.02 * randn(n) for n in sizes]
        types = [_param_type(case, n) for n in sizes]
        mastered = [case["master"] and t != torch.float32 for t in types]
        m = [3e-4 * randn(n) for n in sizes]
        v = [(1e-3 * (0.5 + torch.rand(n, generator=gen, device="cuda"))).square() for n in sizes]
        s["grads"] = grads
        s["params"], s["all_params"] = _in_buffers([x.to(t) for x, t in zip(w, types)])
        s["masters"], s["all_masters"] = _in_buffers([x if k else None for x, k in zip(w, mastered)])
        if case["bits"] == 8:
            pairs = [_quantize(x[None]) for x in m] + [_quantize(x.sqrt()[None]) for x in v]
            codes, all_codes = _in_buffers([c.view(torch.uint8).view(-1) for c, _ in pairs], 512)
            scales, all_scales = _in_buffers([e.view(torch.uint8).view(-1) for _, e in pairs], 4)
            states = [[c[None], e[None]] for c, e in zip(codes, scales)]
            s["all_states"] = [all_codes[0].view(torch.float8_e4m3fn), all_scales[0].view(torch.float8_e8m0fnu)]
        else:
            states, s["all_states"] = _in_buffers(m + v)
        s.update(m=states[:len(sizes)], v=states[len(sizes):], decay=[0.0 if n < VECTOR else DECAY for n in sizes])
        s["counter"] = torch.tensor([1000, 0], dtype=torch.int32, device="cuda")
        s["factor"] = torch.tensor([0.25], device="cuda")
    return s


# ----------------------------------------------------------------------- work
def _fp8_bytes(R, C, tile=1):
    return R * C + -(-R // tile) * -(-C // BLOCK)


def work(case):
    op = case["op"]
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        out = _fp8_bytes(M, N) if case["type"] == "fp8" else M * N * SIZE[case["type"]]
        return dict(bytes=_fp8_bytes(M, K) + _fp8_bytes(N, K, BLOCK) + N * (4 if case["type"] == "f32" else 2)
                    + out * (2 if case["residual"] else 1) + (_fp8_bytes(M, N) if case["keep"] else 0),
                    flops=2 * M * N * K)
    if op == "linear_bwd":
        M, N = case["M"], case["N"]
        return dict(bytes=M * N * SIZE[case["type"]] + (_fp8_bytes(M, N) if case["act"] != "none" else 0)
                    + _fp8_bytes(M, N) + _fp8_bytes(N, M) + 4 * N, flops=16 * M * N)
    sizes = _sizes(case)
    if op == "grad_norm":
        return dict(bytes=sum(sizes) * SIZE[case["grad"]] + 8, flops=2 * sum(sizes))
    total = 0
    for n in sizes:
        p = 4 if n < VECTOR else SIZE[case["type"]]
        g = 4 if n < VECTOR else SIZE[case["grad"]]
        state = 16 * n if case["bits"] == 32 else 4 * _fp8_bytes(1, n)
        total += n * (p + 8 if case["master"] and p < 4 else 2 * p) + n * g + state
    return dict(bytes=total + 12, flops=20 * sum(sizes))


# ------------------------------------------------------- definition in 64 bits
def _grid64(x, bits, low):
    """Step at |x| of a float type with `bits` mantissa bits and smallest normal exponent `low`."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** low)))
    # log2 may round to the wrong side of a whole number
    e = torch.where(torch.exp2(e) > x.abs(), e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= x.abs(), e + 1, e).clamp(min=low)
    return torch.exp2(e - bits)


def _scales64(amax):
    scale = torch.exp2(torch.ceil(torch.log2(amax / 448)).clamp(min=-126))
    scale = torch.where(scale * 448 < amax, scale * 2, scale)
    scale = torch.where((scale * 224 >= amax) & (scale > 2.0 ** -126), scale / 2, scale)
    return torch.where(amax == 0, torch.ones_like(scale), scale)


def _quantize64(x, thresholds=None, root=False):
    """Values of codes [R, C] and scales of x: to nearest, or by thresholds in [0, 1)."""
    R, C = x.shape
    cb = -(-C // BLOCK)
    grid = torch.zeros(R, cb * BLOCK, dtype=torch.float64, device=x.device)
    grid[:, :C] = x
    grid = grid.view(R, cb, BLOCK)
    scale = _scales64(grid.abs().amax(dim=2))
    q = (grid / scale[:, :, None]).view(R, -1)[:, :C]
    step = _grid64(q, 3, -6)
    if thresholds is None:
        return [torch.round(q / step) * step, scale]
    codes = torch.sign(q) * torch.floor(q.abs() / step + thresholds) * step
    return [torch.where((codes == 0) & (q > 0), 2.0 ** -9, codes) if root else codes, scale]


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


def _act64(x, kind):
    if kind == "gelu":
        return x * 0.5 * torch.erfc(-x / math.sqrt(2))
    if kind == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    if kind == "silu":
        return x * torch.sigmoid(x)
    return torch.maximum(x, torch.zeros_like(x)) if kind == "relu" else x


def _slope64(x, kind):
    if kind == "gelu":
        return 0.5 * torch.erfc(-x / math.sqrt(2)) + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x ** 3))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 0.134145 * x * x)
    if kind == "silu":
        s = torch.sigmoid(x)
        return s + x * s * (1 - s)
    return torch.where(x > 0, 1.0, 0.0).double()


def _adam64(s, i, t):
    p, master = s["params"][i], s["masters"][i]
    n = p.shape[0]
    index = torch.arange(n, device=p.device)
    u = ((index * WEYL_I + t * WEYL_T) % 2 ** 32).double() / 2 ** 32
    x = (p if master is None else master).double()
    g = s["grads"][i].double() * 0.25
    small = s["bits"] == 8
    m = _dequantize64(*s["m"][i])[0] if small else s["m"][i].double()
    v = _dequantize64(*s["v"][i])[0] ** 2 if small else s["v"][i].double()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    update = (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    x = x - LR * s["decay"][i] * x - LR * update
    rounded = x
    if master is None and p.dtype != torch.float32:
        step = _grid64(x, 7, -126) if p.dtype == torch.bfloat16 else _grid64(x, 10, -14)
        rounded = torch.sign(x) * torch.floor(x.abs() / step + u) * step
    states = [_quantize64(m[None], u, False), _quantize64(torch.sqrt(v)[None], u, True)] if small else [m, v]
    return rounded, None if master is None else x, states


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "linear":
        pre = torch.einsum("mk,nk->mn", _dequantize64(*s["a"]), _dequantize64(*s["b"])) + s["bias"].double()
        y = _act64(pre, s["act"])
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return [_quantize64(y) if s["dtype"] == torch.float8_e4m3fn else y, _quantize64(pre) if s["keep"] else None]
    if op == "linear_bwd":
        d = s["dy"].double()
        if s["kept"] is not None:
            d = d * _slope64(_dequantize64(*s["kept"]), s["act"])
        return [_quantize64(d), _quantize64(d.t()), torch.einsum("mn->n", d)]
    if op == "grad_norm":
        norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in s["grads"]))
        return torch.tensor([norm, min(1.0, s["most"] / norm)], dtype=torch.float64)
    done = [_adam64(s, i, 1001) for i in range(len(s["params"]))]

    def together(values, buffers, parts):
        """Values in the places that the parts have in the buffers."""
        new = [torch.zeros(b.shape, dtype=torch.float64, device=b.device) for b in buffers]
        for x, part in zip(values, parts):
            for b, to in zip(buffers, new):
                if part is not None and part.untyped_storage().data_ptr() == b.untyped_storage().data_ptr():
                    at = part.storage_offset()
                    to[at:at + part.numel()] = x.reshape(-1)
        return new

    states, parts = [d[2][0] for d in done] + [d[2][1] for d in done], s["m"] + s["v"]
    if s["bits"] == 8:
        states = [q for q, _ in states] + [e for _, e in states]
        parts = [q for q, _ in parts] + [e for _, e in parts]
    return [together([d[0] for d in done], s["all_params"], s["params"]),
            together([d[1] for d in done], s["all_masters"], s["masters"]),
            together(states, s["all_states"], parts), s["counter"][:1] + 1]
