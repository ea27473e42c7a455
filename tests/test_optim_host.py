"""The entry points over many tensors without a GPU: argument checks of the C
ABI and of the Python binding. Every call is rejected before any CUDA call, so
the made-up addresses are never read."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import grads_taco_compress_gb300 as taco
from oracle import optim_oracle as O
from test_fp8_host import A, ALIGN, ARG, BF16, F16, F32, NULL, SHAPE, WS, lib, no_gpu_only  # noqa: F401
from test_fp8_host_binding import fake


class Tensor(ctypes.Structure):
    """taco_adamw_tensor of taco.h."""

    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("n", ctypes.c_int64), ("weight_decay", ctypes.c_float),
                ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32)]


class Grad(ctypes.Structure):
    """taco_grad_tensor of taco.h."""

    _fields_ = [("data", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32)]


def tensor(i=0, **kw):
    d = dict(param=(8 * i + 1) * A, grad=(8 * i + 2) * A, master=None, m=(8 * i + 3) * A, v=(8 * i + 4) * A,
             m_scales=None, v_scales=None, n=1000, weight_decay=0.1, param_dtype=BF16, grad_dtype=F32)
    d.update(kw)
    return Tensor(*(d[k] for k, _ in Tensor._fields_))


def adamw(lib, tensors, **kw):
    a = dict(n=len(tensors), lr=1e-3, lr_dev=None, b1=0.9, b2=0.99, eps=1e-8, scale=None, counter=100 * A)
    a.update(kw)
    array = (Tensor * max(len(tensors), 1))(*tensors)
    return lib.taco_adamw(array, a["n"], a["lr"], a["lr_dev"], a["b1"], a["b2"], a["eps"], a["scale"], a["counter"], None)


@no_gpu_only
@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), SHAPE), (dict(n=(1 << 20) + 1), SHAPE), (dict(counter=None), NULL), (dict(counter=100 * A + 2), ALIGN),
    (dict(b1=1.0), ARG), (dict(b1=-0.1), ARG), (dict(b2=1.0), ARG), (dict(b2=float("nan")), ARG), (dict(eps=0.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(eps=1e-60), ARG), (dict(eps=-1e-8), ARG),
    (dict(lr=float("nan")), ARG), (dict(lr=float("inf")), ARG), (dict(lr_dev=99 * A + 1), ALIGN),
    (dict(scale=99 * A + 2), ALIGN), (dict(scale=100 * A), ARG), (dict(lr_dev=A), ARG), (dict(counter=A + 8), ARG),
])
def test_step_rejects(lib, kw, status):  # noqa: F811
    assert adamw(lib, [tensor()], **kw) == status


@no_gpu_only
@pytest.mark.parametrize("kw,status", [
    (dict(param_dtype=3), ARG), (dict(grad_dtype=-1), ARG), (dict(grad_dtype=F16), ARG),
    (dict(param_dtype=F32, grad_dtype=BF16), ARG), (dict(param_dtype=F32, master=5 * A), ARG),
    (dict(weight_decay=float("nan")), ARG), (dict(weight_decay=float("inf")), ARG), (dict(n=-1), SHAPE),
    (dict(n=(1 << 40) + 1), SHAPE), (dict(param=None), NULL), (dict(grad=None), NULL), (dict(m=None), NULL),
    (dict(v=None), NULL), (dict(m_scales=5 * A), NULL), (dict(v_scales=5 * A), NULL), (dict(param=A + 1), ALIGN),
    (dict(grad=2 * A + 2), ALIGN), (dict(master=5 * A + 2), ALIGN), (dict(m=3 * A + 2), ALIGN),
    (dict(v=4 * A + 1), ALIGN),
    (dict(m=3 * A + 8, m_scales=5 * A, v_scales=6 * A), ALIGN), (dict(grad=A), ARG), (dict(grad=A + 1996), ARG),
    (dict(m=4 * A - 3996), ARG), (dict(master=A), ARG), (dict(m_scales=3 * A + 992, v_scales=6 * A), ARG),
    (dict(m_scales=5 * A, v_scales=5 * A + 7), ARG),
])
def test_tensor_rejects(lib, kw, status):  # noqa: F811
    for before in ([], [tensor(1), tensor(2)]):
        assert adamw(lib, before + [tensor(**kw)]) == status


@no_gpu_only
def test_the_same_tensor_twice(lib):  # noqa: F811
    assert adamw(lib, [tensor(), tensor()]) == ARG
    assert adamw(lib, [tensor(), tensor(1, param=A + 1000)]) == ARG
    assert adamw(lib, [tensor(), tensor(1), tensor(2, v=11 * A)]) == ARG
    assert adamw(lib, [tensor(), tensor(1, grad=A)]) == ARG     # a gradient that is another's parameter


def grad_norm(lib, grads, **kw):
    a = dict(n=len(grads), most=1.0, out=90 * A, ws=91 * A, wsb=lib.taco_grad_norm_workspace_bytes(len(grads)))
    a.update(kw)
    array = (Grad * max(len(grads), 1))(*(Grad(*g) for g in grads))
    return lib.taco_grad_norm(array, a["n"], a["most"], a["out"], a["ws"], a["wsb"], None)


@no_gpu_only
@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), SHAPE), (dict(n=1 << 21), SHAPE), (dict(most=-1.0), ARG), (dict(most=float("nan")), ARG),
    (dict(out=None), NULL), (dict(ws=None), WS), (dict(wsb=8191), WS), (dict(ws=91 * A + 4), ALIGN),
    (dict(out=90 * A + 2), ALIGN), (dict(out=A), ARG), (dict(ws=A), ARG), (dict(out=91 * A + 16), ARG)])
def test_norm_rejects(lib, kw, status):  # noqa: F811
    assert grad_norm(lib, [(A, 1000, F16)], **kw) == status


@no_gpu_only
@pytest.mark.parametrize("grad,status", [
    ((A, 10, 3), ARG), ((A, -1, F32), SHAPE), ((A, (1 << 40) + 1, F32), SHAPE), ((None, 10, F32), NULL),
    ((A + 1, 10, BF16), ALIGN), ((A + 2, 10, F32), ALIGN)])
def test_norm_tensor_rejects(lib, grad, status):  # noqa: F811
    assert grad_norm(lib, [(2 * A, 5, F32), grad]) == status


@no_gpu_only
def test_norm_workspace(lib):  # noqa: F811
    assert [lib.taco_grad_norm_workspace_bytes(n) for n in (-1, 0, 1, 1300, 1301)] == [0, 8192, 8192, 8192, 16384]


def state(n=512, bits=32, device=0, at=1):
    if bits == 32:
        return taco.AdamState(fake(n, dtype=torch.float32, device=device, at=at),
                              fake(n, dtype=torch.float32, device=device, at=at + 1))
    pair = [taco.Fp8Tensor(fake(1, n, dtype=torch.uint8, device=device, at=at + 2 * k),
                           fake(1, n // 128, dtype=torch.uint8, device=device, at=at + 2 * k + 1)) for k in range(2)]
    return taco.AdamState(*pair)


def call(**kw):
    d = dict(params=[fake(512)], grads=[fake(512, at=5)], states=[state(at=6)],
             counter=fake(2, dtype=torch.int32, at=20), lr=1e-3)
    d.update(kw)
    return taco.taco_adamw(**d)


f32 = torch.float32


def every_other(n):
    """n elements with gaps between them."""
    storage = torch._C._construct_storage_from_data_pointer(A, torch.device("cuda", 0), A >> 1)
    return torch._C._construct_CUDA_Tensor_From_Storage_And_Metadata(
        dict(dtype=torch.bfloat16, size=torch.Size([n]), stride=(2,), storage_offset=0), storage)


@no_gpu_only
@pytest.mark.parametrize("kw,text", [
    (dict(params=fake(512)), "list"), (dict(params=[None]), "tensor"), (dict(params=[torch.zeros(512)]), "CUDA"),
    (dict(params=[fake(512, dtype=torch.float64)]), "bf16"), (dict(params=[every_other(512)]), "contiguous"),
    (dict(grads=[]), "as many"), (dict(grads=[fake(256)]), r"grads\[0\].*shape"), (dict(grads=[fake(2, 256)]), "shape"),
    (dict(grads=[fake(512, dtype=torch.float16)]), "type"), (dict(grads=[fake(512, device=1)]), "one device"),
    (dict(states=[]), "as many"), (dict(states=[None]), "AdamState"),
    (dict(states=[state(256)]), r"states\[0\]\.m.*512"),
    (dict(states=[state(256, 8)]), "512"), (dict(states=[(state().m, state(bits=8).v)]), "both"),
    (dict(states=[state(device=1)]), "one device"), (dict(states=[state(bits=8, device=1)]), "one device"),
    (dict(counter=fake(2)), "int32"), (dict(counter=fake(3, dtype=torch.int32)), "int32"), (dict(counter=1), "tensor"),
    (dict(counter=fake(2, dtype=torch.int32, device=1)), "one device"), (dict(lr="x"), "lr"), (dict(lr=None), "lr"),
    (dict(lr=fake(2, dtype=f32)), "lr"), (dict(lr=fake(1)), "lr"), (dict(betas=0.9), "betas"),
    (dict(betas=(1, 2, 3)), "betas"),
    (dict(betas=("a", 0.9)), "betas"), (dict(eps=None), "eps"), (dict(weight_decay=[0.1, 0.1]), "as many"),
    (dict(weight_decay=["x"]), "weight_decay"), (dict(weight_decay=None), "weight_decay"),
    (dict(grad_scale=0.5), "grad_scale"), (dict(grad_scale=fake(2, dtype=f32)), "grad_scale"),
    (dict(masters=[]), "as many"), (dict(masters=[fake(512)]), "f32"), (dict(masters=[fake(256, dtype=f32)]), "512"),
    (dict(params=[fake(512, dtype=f32)], grads=[fake(512, dtype=f32)], masters=[fake(512, dtype=f32)]), "no master"),
])
def test_binding_refuses(kw, text):
    with pytest.raises(ValueError, match=text):
        call(**kw)


@no_gpu_only
@pytest.mark.parametrize("kw,text", [
    (dict(grads=[]), "a tensor"), (dict(grads=fake(3)), "list"), (dict(grads=[fake(3), 1]), "tensor"),
    (dict(grads=[torch.zeros(3)]), "CUDA"), (dict(grads=[fake(3, dtype=torch.int32)]), "bf16"),
    (dict(grads=[fake(3), fake(3, device=1)]), "one device"), (dict(max_norm="x"), "max_norm"),
    (dict(out=fake(2)), "out"), (dict(out=fake(3, dtype=f32)), "out"),
    (dict(out=fake(2, dtype=f32, device=1)), "one device"),
    (dict(workspace=every_other(8192)), "workspace"), (dict(workspace=torch.zeros(9)), "workspace"),
])
def test_norm_binding_refuses(kw, text):
    with pytest.raises(ValueError, match=text):
        taco.taco_grad_norm(**{**dict(grads=[fake(3)], out=fake(2, dtype=f32, at=3),
                                      workspace=fake(8192, dtype=torch.uint8, at=5)), **kw})


def test_state_and_optimiser_arguments():
    with pytest.raises(ValueError):
        taco.taco_adam_state(torch.zeros(3), bits=16)
    with pytest.raises(ValueError):
        taco.AdamW([])
    s = taco.taco_adam_state(torch.zeros(300), bits=8)
    assert s.m.codes.shape == (1, 300) and s.m.scales.shape == (1, 3) and not s.v.dequantize().any()


def test_rounding_by_thresholds_keeps_the_mean():
    """The oracle itself: over 4096 steps a value is rounded up as often as its
    place between two codes says, within the discrepancy of the sequence."""
    for x in (0.3, 1.01, 17.7, 2.0 ** -8 * 1.3, 400.0, -3.14):
        u = np.concatenate([O.thresholds(1, t) for t in range(1, 4097)])
        q = O.by_threshold(np.full(u.size, x), u, "e4m3")
        assert abs(q.mean() - x) < 4e-3 * O.step_at(np.array(x), "e4m3")
        assert set(np.unique(np.abs(q) / O.step_at(np.array(x), "e4m3"))) <= {np.floor(abs(x) / O.step_at(np.array(x), "e4m3")),
                                                                             np.ceil(abs(x) / O.step_at(np.array(x), "e4m3"))}


@no_gpu_only
def test_refusals_hold_no_reference_and_drop_none():
    import sys

    lists = [[fake(512)], [fake(512, at=5)], [state(at=6)], [fake(512, dtype=f32)]]
    empty = [[] for _ in lists]
    before = [sys.getrefcount(x) for x in lists + empty]
    for _ in range(50):
        for k in (1, 2, 3):
            arg = ("params", "grads", "states", "masters")[k]
            with pytest.raises(ValueError):
                call(**{"params": lists[0], "grads": lists[1], "states": lists[2], arg: empty[k]})
    assert [sys.getrefcount(x) for x in lists + empty] == before
