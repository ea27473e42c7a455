"""Outputs on the memory of inputs that an FP8 entry point does not name as in
place: refused, also where address, rows, width and stride all agree. Every
such call is rejected before any CUDA call; one that the header allows gets as
far as the missing device."""

from __future__ import annotations

import pytest

from test_fp8_host import (A, ARG, BF16, CUDA, F16, F32, _norm, _norm_backward, fp8, lib, no_gpu_only)  # noqa: F401

pytestmark = no_gpu_only


@pytest.mark.parametrize("dtype,size", [(BF16, 2), (F16, 2), (F32, 4)])
@pytest.mark.parametrize("operand", ["a", "b"])
def test_product_exactly_over_its_operands(lib, dtype, size, operand):
    """out [M, N] with N elements as wide as K codes."""
    N = 64
    K = N * size
    M = 300 if operand == "a" else N
    out = (1 if operand == "a" else 2) * A
    for add, ldadd in ((None, 0), (4 * A, N)):
        assert lib.taco_matmul_fp8(fp8(1, M, K), fp8(2, N, K), add, ldadd, out, N, dtype, None) == ARG


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_norm_of_one_row_over_the_weight(lib, dtype):
    assert _norm(lib, M=1, dtype=dtype, wd=dtype, h=3 * A, y=fp8(6, 1, 256), ck=fp8(7, 1, 256)) == ARG


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_norm_gradient_of_one_row_over_the_weight(lib, dtype):
    assert _norm_backward(lib, M=1, dtype=dtype, wd=dtype, dx=3 * A, ck=fp8(2, 1, 256)) == ARG


def test_named_inputs_stay_in_place(lib):
    assert _norm(lib, h=A) == _norm(lib, h=2 * A) == CUDA
    for kw in (dict(dx=A), dict(dx=5 * A), dict(ck=None, h=9 * A, ldh=256, dx=9 * A)):
        assert _norm_backward(lib, **kw) == CUDA
    assert lib.taco_matmul_fp8(fp8(1, 4, 256), fp8(2, 64, 256), 3 * A, 64, 3 * A, 64, F32, None) == CUDA
    for dg, du in ((A, 6 * A), (6 * A, A)):
        assert lib.taco_swiglu_fp8_backward(A, 256, fp8(2, 4, 256), fp8(3, 4, 256), BF16, 4, 256, dg, 256, du, 256,
                                            None) == CUDA


def test_one_row_in_place_whatever_the_stride(lib):
    """The stride of a single row describes nothing: dy as the first half of a [1, 2 F] gradient."""
    for dg, du in ((A, A + 512), (A - 512, A)):
        assert lib.taco_swiglu_fp8_backward(A, 256, fp8(2, 1, 256), fp8(3, 1, 256), BF16, 1, 256, dg, 512, du, 512,
                                            None) == CUDA
    assert _norm(lib, M=1, h=A, ldx=300, y=fp8(6, 1, 256), ck=fp8(7, 1, 256)) == CUDA
    assert _norm_backward(lib, M=1, dx=A, lddy=300, ck=fp8(2, 1, 256)) == CUDA
    assert lib.taco_matmul_fp8(fp8(1, 1, 256), fp8(2, 64, 256), 3 * A, 64, 3 * A, 128, F32, None) == CUDA
    # another width or start of the same memory is still no input in place
    assert lib.taco_swiglu_fp8_backward(A, 256, fp8(2, 1, 256), fp8(3, 1, 256), BF16, 1, 256, A + 64, 512, 6 * A, 512,
                                        None) == ARG
