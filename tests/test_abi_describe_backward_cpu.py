"""Refusals of swiglu_describe_backward (no GPU): it takes the sizes that the calls take."""
import ctypes
import os

import pytest

from gated_mlp_gemm_amd import swiglu as sw

ERR_NULL, ERR_SHAPE, ERR_UNSUP = sw.SWIGLU_ERR_NULL, sw.SWIGLU_ERR_SHAPE, sw.SWIGLU_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sw.LIBRARY):
        pytest.fail("libswiglu.so is not built (python -m gated_mlp_gemm_amd.build)")
    return sw.load_library()


def describe(lib, M=64, N=72, K=136, call=2, kind=0, add=0, size=64):
    buf = ctypes.create_string_buffer(b"x" * 63, 64)
    status = lib.swiglu_describe_backward(M, N, K, call, kind, add, 0, buf, size)
    if status != ERR_NULL:
        assert buf.value == b""
    return status


@pytest.mark.parametrize("call", [0, 1, 2])
def test_shapes(lib, call):
    assert describe(lib, call=call, M=-1) == ERR_SHAPE
    assert describe(lib, call=call, M=(1 << 30) + 1) == ERR_SHAPE
    for bad in (0, 4, 12, -8, (1 << 21) + 8):
        assert describe(lib, call=call, N=bad) == ERR_SHAPE
        assert describe(lib, call=call, K=bad) == ERR_SHAPE
    assert describe(lib, call=call, N=(1 << 20) + 8) == ERR_SHAPE or call == 0
    assert describe(lib, call=call, kind=2) == ERR_UNSUP
    assert describe(lib, call=call, size=0) == ERR_NULL


def test_calls(lib):
    assert describe(lib, call=3) == ERR_UNSUP and describe(lib, call=-1) == ERR_UNSUP
    assert lib.swiglu_describe_backward(64, 72, 136, 2, 0, 0, 0, None, 64) == ERR_NULL
    with pytest.raises(KeyError):
        sw.swiglu_describe_backward(64, 72, 136, "forward")
    with pytest.raises(TypeError):
        sw.swiglu_describe_backward(64, 72, 136, grad_dtype=None.__class__)
