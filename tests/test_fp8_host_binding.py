"""What the compiled binding of the FP8 entry points refuses before any CUDA
call: tensors on a CUDA device with made-up addresses, which nothing reads."""

from __future__ import annotations

import pytest
import torch

import grads_taco_compress_gb300 as taco
from grads_taco_compress_gb300 import fp8 as F
from test_fp8_host import A, no_gpu_only

pytestmark = no_gpu_only


def fake(*shape, dtype=torch.bfloat16, device=0, at=1):
    storage = torch._C._construct_storage_from_data_pointer(at * A, torch.device("cuda", device), A >> 1)
    return torch._C._construct_CUDA_Tensor_From_Storage_And_Metadata(
        dict(dtype=dtype, size=torch.Size(shape), stride=torch.empty(shape, device="meta").stride(), storage_offset=0),
        storage)


def fake_fp8(*shape, device=0, scales_device=None, at=1):
    scales_device = device if scales_device is None else scales_device
    return F.Fp8Tensor(fake(*shape, dtype=torch.uint8, device=device, at=at),
                       fake(*shape[:-1], 4, dtype=torch.uint8, device=scales_device, at=at + 1))


def arguments():
    """Every entry point with all its tensors on one device, by name."""
    x, f32 = fake(4, 512), torch.float32
    return [
        (taco.taco_fp8_quantize, dict(x=x, cols=True, out=fake_fp8(4, 512, at=2), out_t=fake_fp8(512, 4, at=4))),
        (taco.taco_fp8_quantize, dict(x=fake_fp8(4, 512), out=fake_fp8(4, 512, at=4))),
        (taco.taco_rms_norm_fp8, dict(x=x, weight=fake(512), residual=fake(4, 512), checkpoint=fake_fp8(4, 512),
                                      out=fake_fp8(4, 512), h=fake(4, 512), rstd=fake(4, dtype=f32))),
        (taco.taco_rms_norm_fp8_backward, dict(dy=x, saved=fake_fp8(4, 512), weight=fake(512), rstd=fake(4, dtype=f32),
                                               dh=fake(4, 512), dx=fake(4, 512), dw=fake(512, dtype=f32),
                                               workspace=fake(1 << 16, dtype=torch.uint8))),
        (taco.taco_rms_norm_fp8_backward, dict(dy=x, saved=fake(4, 512), weight=fake(512), rstd=fake(4, dtype=f32))),
        (taco.taco_swiglu_fp8, dict(gate_up=fake(4, 1024), checkpoint=fake_fp8(2, 4, 512), out=fake_fp8(4, 512))),
        (taco.taco_swiglu_fp8_backward, dict(dy=x, checkpoint=fake_fp8(2, 4, 512), out=fake(4, 1024))),
        (taco.taco_matmul_fp8, dict(a=fake_fp8(4, 512), b=fake_fp8(64, 512), out=fake(4, 64), add=fake(4, 64))),
    ]


CASES = [(i, name, part) for i, (_, kw) in enumerate(arguments()) for name, v in kw.items()
         for part in ((0, 1) if isinstance(v, tuple) else (None,)) if name != "cols"]


@pytest.mark.parametrize("i,name,part", CASES)
def test_tensors_on_another_device(i, name, part):
    call, kw = arguments()[i]
    v = kw[name]
    if part is None:
        kw[name] = fake(*v.shape, dtype=v.dtype, device=1)
    else:
        kw[name] = fake_fp8(*v.codes.shape, device=1, scales_device=0) if part == 0 else \
            fake_fp8(*v.codes.shape, device=0, scales_device=1)
    with pytest.raises(ValueError, match="one device"):
        call(**kw)


@pytest.mark.parametrize("call,kw,name", [
    (taco.taco_fp8_quantize, dict(x=(4, 512)), "rows"), (taco.taco_fp8_quantize, dict(x=(4, 512)), "cols"),
    (taco.taco_rms_norm_fp8, dict(x=(4, 512), weight=(512,)), "checkpoint"),
    (taco.taco_swiglu_fp8, dict(gate_up=(4, 1024)), "checkpoint")])
def test_flags_without_a_truth_value(call, kw, name):
    """Such as a tensor in the place of an Fp8Tensor: refused, with the argument's name."""
    with pytest.raises(ValueError, match=name):
        call(**{k: fake(*shape) for k, shape in kw.items()}, **{name: torch.zeros(2)})
