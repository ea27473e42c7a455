"""The layer's product and its gradient without a GPU: argument checks of the C
ABI and of the Python binding (made-up addresses, which nothing reads), and the
oracle's slopes against differences."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import grads_taco_compress_gb300 as taco
from linear_util import ACTS
from oracle import fp8_oracle as Q
from test_fp8_host import A, ALIGN, ARG, BF16, BLOCK, F32, NULL, OK, SHAPE, WS, fp8, lib, no_gpu_only  # noqa: F401
from test_fp8_host_binding import fake

F8 = torch.float8_e4m3fn


def fp8_fake(rows, cols, device=0, at=1, scale_rows=None):
    """A block tensor whose rows of scales start on 4 bytes."""
    def padded(r, c, at):
        storage = torch._C._construct_storage_from_data_pointer(at * A, torch.device("cuda", device), A >> 1)
        ld = -(-c // 16) * 16
        return torch._C._construct_CUDA_Tensor_From_Storage_And_Metadata(
            dict(dtype=torch.uint8, size=torch.Size((r, c)), stride=(ld, 1), storage_offset=0), storage)
    return taco.Fp8Tensor(padded(rows, cols, at), padded(scale_rows or rows, -(-cols // 128), at + 1))


def _linear(lib, **kw):
    a = dict(a=fp8(1, 4, 256), b=fp8(2, 300, 256), bias=3 * A, bd=F32, act=2, res=None, ldr=0, out=4 * A, ldo=304,
             dtype=BF16, y=None, ck=fp8(5, 4, 300))
    a.update(kw)
    return lib.taco_linear_fp8(a["a"], a["b"], a["bias"], a["bd"], a["act"], a["res"], a["ldr"], a["out"], a["ldo"],
                               a["dtype"], a["y"], a["ck"], None)


FP8_OUT = dict(out=None, y=fp8(6, 4, 300), dtype=77)


@no_gpu_only
@pytest.mark.parametrize("kw,status", [
    (dict(a=None), NULL), (dict(b=None), NULL), (dict(act=-1), ARG), (dict(act=5), ARG), (dict(bd=3), ARG),
    (dict(dtype=4), ARG), (dict(out=None), NULL), (dict(y=fp8(6, 4, 300)), ARG),
    (dict(FP8_OUT, res=7 * A, ldr=300), ARG), (dict(b=fp8(2, 300, 384)), SHAPE),
    (dict(a=fp8(1, 4, 256, tile=3)), BLOCK),
    (dict(bias=3 * A + 2), ALIGN), (dict(res=7 * A, ldr=299), SHAPE), (dict(res=7 * A + 1, ldr=300), ALIGN),
    (dict(ldo=200), SHAPE), (dict(out=4 * A + 1), ALIGN), (dict(ck=fp8(5, 5, 300)), SHAPE),
    (dict(ck=fp8(5, 4, 300, tile=128)), BLOCK), (dict(FP8_OUT, y=fp8(6, 4, 300, tile=128)), BLOCK),
    (dict(FP8_OUT, y=fp8(6, 3, 300)), SHAPE), (dict(b=fp8(2, 0, 256), ck=fp8(5, 4, 1)), SHAPE),
    (dict(out=A), ARG), (dict(out=3 * A), ARG), (dict(out=5 * A), ARG), (dict(ck=fp8(2, 4, 300)), ARG),
    (dict(res=4 * A, ldr=600), ARG), (dict(res=4 * A + 16, ldr=304), ARG), (dict(FP8_OUT, ck=fp8(6, 4, 300)), ARG),
    (dict(FP8_OUT, y=fp8(1, 4, 300)), ARG), (dict(bias=4 * A + 64), ARG),
    (dict(a=fp8(1, 0, 256), ck=fp8(5, 0, 300)), OK), (dict(b=fp8(2, 0, 256), ck=None, bias=None), OK),
])
def test_linear_rejects(lib, kw, status):  # noqa: F811
    assert _linear(lib, **kw) == status


def _backward(lib, **kw):
    a = dict(dy=A, lddy=300, dtype=BF16, M=200, N=300, ck=fp8(2, 200, 300), act=1, rows=fp8(3, 200, 300),
             cols=fp8(4, 300, 200), db=5 * A, ws=6 * A, wsb=2 * 300 * 4)
    a.update(kw)
    return lib.taco_linear_fp8_backward(a["dy"], a["lddy"], a["dtype"], a["M"], a["N"], a["ck"], a["act"], a["rows"],
                                        a["cols"], a["db"], a["ws"], a["wsb"], None)


@no_gpu_only
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), ARG), (dict(act=9), ARG), (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(dy=None), NULL),
    (dict(lddy=299), SHAPE), (dict(dy=A + 1), ALIGN), (dict(ck=None), NULL), (dict(act=0), ARG),
    (dict(ck=fp8(2, 200, 299)), SHAPE), (dict(ck=fp8(2, 200, 300, tile=128)), BLOCK),
    (dict(rows=None, cols=None, db=None), NULL), (dict(rows=fp8(3, 200, 300, tile=128)), BLOCK),
    (dict(rows=fp8(3, 199, 300)), SHAPE), (dict(cols=fp8(4, 200, 300)), SHAPE), (dict(db=5 * A + 2), ALIGN),
    (dict(ws=None), WS), (dict(wsb=2399), WS), (dict(ws=6 * A + 8), ALIGN), (dict(rows=fp8(1, 200, 300)), ARG),
    (dict(cols=fp8(2, 300, 200)), ARG), (dict(cols=fp8(3, 300, 200)), ARG), (dict(db=A + 512), ARG),
    (dict(ws=5 * A), ARG),
    (dict(ws=4 * A), ARG),
])
def test_backward_rejects(lib, kw, status):  # noqa: F811
    assert _backward(lib, **kw) == status


@no_gpu_only
def test_backward_workspace(lib):  # noqa: F811
    w = lib.taco_linear_backward_workspace_bytes
    assert [w(-1, 5), w(5, 0), w(0, 5), w(128, 5), w(129, 5), w(257, 7)] == [0, 0, 0, 0, 40, 84]


def linear(**kw):
    d = dict(x=fp8_fake(4, 256), w=fp8_fake(64, 256, at=3), bias=fake(64, at=5), out=fake(4, 64, at=6),
             checkpoint=fp8_fake(4, 64, at=7))
    d.update(kw)
    return taco.taco_linear_fp8(**d)


@no_gpu_only
@pytest.mark.parametrize("kw,text", [
    (dict(x=fake(4, 256)), "x must be an Fp8Tensor"), (dict(w=None), "w must be"),
    (dict(activation="tanh"), "activation"),
    (dict(activation=1), "activation"), (dict(bias=fake(63)), "bias"), (dict(bias=fake(64, dtype=torch.int32)), "bias"),
    (dict(bias=fake(64, device=1)), "one device"), (dict(out=fake(4, 63)), "rows of x and of w"),
    (dict(out=fake(4, 64, dtype=torch.int8)), "out"), (dict(residual=fake(4, 63)), "residual"),
    (dict(residual=fake(4, 64, dtype=torch.float32)), "another type"),
    (dict(residual=fake(4, 64, device=1)), "one device"),
    (dict(out=fp8_fake(4, 64, at=9), residual=fake(4, 64)), "16 or 32"),
    (dict(out=None, out_dtype=F8, residual=fake(4, 64)), "16 or 32"), (dict(out=None, out_dtype="f8"), "out_dtype"),
    (dict(out=None, out_dtype=torch.int32), "out_dtype"), (dict(out=None, out_dtype=torch.float8_e5m2), "out_dtype"),
    (dict(checkpoint=fake(3, 2)), "checkpoint"), (dict(checkpoint=fp8_fake(4, 64, device=1)), "one device"),
    (dict(x=fp8_fake(4, 256, scale_rows=3)), "scales"),
    (dict(w=fp8_fake(0, 256), bias=None, out=None, out_dtype=F8, checkpoint=False), "a column"),
])
def test_linear_binding_refuses(kw, text):
    with pytest.raises(ValueError, match=text):
        linear(**kw)


def backward(**kw):
    d = dict(dy=fake(200, 64), checkpoint=fp8_fake(200, 64, at=2), activation="gelu", out=fp8_fake(200, 64, at=4),
             out_t=fp8_fake(64, 200, at=6), db=fake(64, dtype=torch.float32, at=8),
             workspace=fake(512, dtype=torch.uint8, at=9))
    d.update(kw)
    return taco.taco_linear_fp8_backward(**d)


@no_gpu_only
@pytest.mark.parametrize("kw,text", [
    (dict(dy=fake(200)), "dy"), (dict(dy=fake(200, 0)), "a column"), (dict(checkpoint=None), "takes the checkpoint"),
    (dict(activation=None), "where there is an activation"), (dict(activation="Gelu"), "activation"),
    (dict(rows=False, cols=False, bias=False), "nothing"), (dict(rows=fake(3, 2)), "rows"),
    (dict(out=fake(200, 64)), "out"),
    (dict(out_t=fp8_fake(64, 200, device=1)), "one device"), (dict(db=fake(64)), "db"),
    (dict(db=fake(63, dtype=torch.float32)), "db"), (dict(workspace=torch.zeros(9)), "workspace"),
    (dict(workspace=fake(512, dtype=torch.uint8, device=1)), "one device"),
])
def test_backward_binding_refuses(kw, text):
    with pytest.raises(ValueError, match=text):
        backward(**kw)


@pytest.mark.parametrize("act", ACTS[1:])
def test_oracle_slopes_are_the_activations_differences(act):
    x = np.concatenate([np.linspace(-8, 8, 801) + 1e-3, [-30.0, 30.0]])
    h = 1e-5
    diff = (Q.activate(x + h, act) - Q.activate(x - h, act)) / (2 * h)
    assert np.abs(diff - Q.activation_slope(x, act)).max() < 1e-9 + 1e-9
