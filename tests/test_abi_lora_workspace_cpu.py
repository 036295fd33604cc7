"""The adapters' workspace size for every shape that their calls take (no GPU: what
is refused is refused before any HIP call, what is not fails at the device)."""
import ctypes
import os

import pytest

from gated_mlp_gemm_amd import swiglu as sw


@pytest.fixture(scope="module")
def size():
    if not os.path.exists(sw.LIBRARY):
        pytest.fail("libswiglu.so is not built (python -m gated_mlp_gemm_amd.build)")
    lib = sw.load_library()

    def call(M, N, K, slots=1, rank=8):
        n = ctypes.c_uint64(7)
        return lib.swiglu_lora_workspace_size(M, N, K, slots, rank, ctypes.byref(n)), n.value
    return call


def test_a_down_projections_columns(size):
    """[M][N] . [N][D]: D up to 2^22, none among them; N up to 2^21."""
    assert size(64, 512, 0) == (0, 0)
    for D in ((1 << 21) + 8, 1 << 22):
        assert size(64, 512, D)[0] not in (sw.SWIGLU_ERR_SHAPE, sw.SWIGLU_ERR_NULL)
    assert size(64, 512, (1 << 22) + 8) == (sw.SWIGLU_ERR_SHAPE, 0)
    assert size(64, 512, (1 << 21) + 4) == (sw.SWIGLU_ERR_SHAPE, 0)
    assert size(64, (1 << 21) + 8, 1 << 22) == (sw.SWIGLU_ERR_SHAPE, 0)


def test_gate_and_ups_columns(size):
    """[M][K] . [K][2 N]: N up to 2^22, none among them; K up to 2^21."""
    assert size(64, 0, 512) == (0, 0)
    assert size(64, 1 << 22, 512)[0] not in (sw.SWIGLU_ERR_SHAPE, sw.SWIGLU_ERR_NULL)
    assert size(64, (1 << 22) + 8, 512) == (sw.SWIGLU_ERR_SHAPE, 0)
    assert size(64, 0, 4) == (sw.SWIGLU_ERR_SHAPE, 0)
    assert size(-1, 512, 512) == (sw.SWIGLU_ERR_SHAPE, 0)
