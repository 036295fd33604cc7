"""Refusals of the router's and the low-rank adapters' entry points (no GPU):
invalid arguments are rejected before any HIP call.  Fake device addresses are
used; validation fails before they could be dereferenced."""
import ctypes
import os

import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw

ERR_NULL, ERR_SHAPE, ERR_ALIGN = sw.SWIGLU_ERR_NULL, sw.SWIGLU_ERR_SHAPE, sw.SWIGLU_ERR_ALIGN
ERR_UNSUP, ERR_ALIAS = sw.SWIGLU_ERR_UNSUPPORTED, sw.SWIGLU_ERR_ALIAS

NAMES = ("z", "valid", "ids", "w", "counts", "loss", "ws", "dw", "dl", "dz", "X", "W", "W3", "A",
         "B", "s", "A2", "B2", "s2", "Y", "H")
AT = {n: 0x10_0000_0000 * (i + 1) for i, n in enumerate(NAMES)}


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sw.LIBRARY):
        pytest.fail("libswiglu.so is not built (python -m gated_mlp_gemm_amd.build)")
    return sw.load_library()


def route(lib, M=64, E=16, k=2, kind=0, wsb=1 << 16, **kw):
    p = {**AT, **kw}
    return lib.swiglu_route(p["z"], kind, p["valid"], p["ids"], p["w"], p["counts"], p["loss"], M, E,
                            k, 1, p["ws"], wsb, None)


def route_backward(lib, M=64, E=16, k=2, kind=0, **kw):
    p = {**AT, **kw}
    return lib.swiglu_route_backward(p["z"], kind, p["valid"], p["ids"], p["w"], p["counts"],
                                     p["dw"], p["dl"], p["dz"], M, E, k, 1, None)


@pytest.mark.parametrize("call", [route, route_backward])
def test_route_shapes_and_types(lib, call):
    assert call(lib, kind=2) == ERR_UNSUP
    assert call(lib, kind=-1) == ERR_UNSUP
    assert call(lib, M=-1) == ERR_SHAPE
    assert call(lib, M=1 << 31) == ERR_SHAPE
    assert call(lib, E=0) == ERR_SHAPE
    assert call(lib, E=513) == ERR_SHAPE
    assert call(lib, k=0) == ERR_SHAPE
    assert call(lib, k=17, E=32) == ERR_SHAPE
    assert call(lib, k=9, E=8) == ERR_SHAPE


def test_route_pointers(lib):
    for name in ("z", "ids", "w", "counts", "loss"):
        assert route(lib, **{name: None}) == ERR_NULL, name
        assert route(lib, **{name: AT[name] + 2}) == ERR_ALIGN, name
    assert route(lib, kind=1, z=AT["z"] + 1) == ERR_ALIGN
    assert route(lib, ws=AT["ws"] + 64) == ERR_ALIGN
    assert route(lib, M=0, z=None, ids=None, w=None, counts=None) == ERR_NULL
    assert route(lib, ids=AT["z"] + 64) == ERR_ALIAS
    assert route(lib, w=AT["ids"] + 64) == ERR_ALIAS
    assert route(lib, loss=AT["counts"] + 16 * 4) == ERR_ALIAS     # counts has E + 1
    assert route(lib, counts=AT["valid"] + 60) == ERR_ALIAS
    assert route(lib, ws=AT["z"] & ~255) == ERR_ALIAS


def test_route_backward_pointers(lib):
    for name in ("z", "ids", "w", "counts", "dz"):
        assert route_backward(lib, **{name: None}) == ERR_NULL, name
        assert route_backward(lib, **{name: AT[name] + 2}) == ERR_ALIGN, name
    for name in ("dw", "dl"):
        assert route_backward(lib, **{name: AT[name] + 2}) == ERR_ALIGN, name
    assert route_backward(lib, dz=AT["z"]) == ERR_ALIAS
    assert route_backward(lib, dz=AT["dw"] + 64) == ERR_ALIAS
    assert route_backward(lib, M=0, z=None, ids=None, w=None, counts=None, dz=None) == 0


def test_route_workspace_size(lib):
    n = ctypes.c_uint64(7)
    assert lib.swiglu_route_workspace_size(64, 16, None) == ERR_NULL
    assert lib.swiglu_route_workspace_size(64, 513, ctypes.byref(n)) == ERR_SHAPE and n.value == 0
    assert lib.swiglu_route_workspace_size(-1, 8, ctypes.byref(n)) == ERR_SHAPE


def fused(lib, M=64, N=128, K=256, count=4, rank=16, slots=2, wsb=1 << 20, **kw):
    p = {**AT, **kw}
    return lib.swiglu_fused_gemm_lora(p["X"], p["W"], p["A"], p["B"], p["s"], count, rank, p["ids"],
                                      p["w"], p["Y"], M, N, K, slots, p["ws"], wsb, None)


def down(lib, M=64, N=128, K=256, count=4, rank=16, slots=2, wsb=1 << 20, **kw):
    p = {**AT, **kw}
    return lib.swiglu_down_proj_lora(p["X"], p["W3"], p["A"], p["B"], p["s"], count, rank, p["ids"],
                                     p["w"], p["Y"], M, K, N, slots, p["ws"], wsb, None)


def block(lib, M=64, N=128, K=256, count=4, rank=16, slots=2, wsb=1 << 20, count2=4, rank2=8, **kw):
    p = {**AT, **kw}
    return lib.swiglu_gated_mlp_lora(p["X"], p["W"], p["W3"], p["A"], p["B"], p["s"], count, rank,
                                     p["A2"], p["B2"], p["s2"], count2, rank2, p["ids"], p["w"],
                                     p["H"], p["Y"], M, N, K, slots, p["ws"], wsb, None)


CALLS = [fused, down, block]


@pytest.mark.parametrize("call", CALLS)
def test_lora_shapes(lib, call):
    for kw in (dict(M=-1), dict(K=20), dict(K=1 << 22), dict(N=12), dict(slots=0), dict(slots=9),
               dict(rank=0), dict(rank=12), dict(rank=264), dict(count=0), dict(count=8193)):
        assert call(lib, **kw) == ERR_SHAPE, kw
    assert call(lib, M=0, X=None, W=None, W3=None, A=None, B=None, Y=None, ws=None) == 0
    # T does not fit the workspace
    assert call(lib, wsb=64 * 2 * 16 * 2 - 1) == ERR_SHAPE


def test_lora_block_tables(lib):
    assert block(lib, rank2=12) == ERR_SHAPE
    assert block(lib, count2=0) == ERR_SHAPE
    # the larger of the two tables' T
    assert block(lib, rank=8, rank2=256, wsb=64 * 2 * 256 * 2 - 1) == ERR_SHAPE
    for name in ("A2", "B2", "s2", "H", "W3"):
        assert block(lib, **{name: None}) == ERR_NULL, name
    assert block(lib, A2=AT["A2"] + 8) == ERR_ALIGN
    assert block(lib, H=AT["B2"] + 64) == ERR_ALIAS
    assert block(lib, Y=AT["H"] + 64) == ERR_ALIAS


@pytest.mark.parametrize("call", CALLS)
def test_lora_pointers(lib, call):
    weight = {"down": "W3"}.get(call.__name__, "W")
    for name in ("X", weight, "A", "B", "s", "ids", "Y", "ws"):
        assert call(lib, **{name: None}) == ERR_NULL, name
    for name in ("X", weight, "A", "B", "Y"):
        assert call(lib, **{name: AT[name] + 8}) == ERR_ALIGN, name
    for name in ("s", "ids", "w"):
        assert call(lib, **{name: AT[name] + 2}) == ERR_ALIGN, name
    assert call(lib, ws=AT["ws"] + 16) == ERR_ALIGN
    for name in ("X", weight, "A", "B", "s", "ids", "w", "ws"):
        assert call(lib, Y=AT[name]) == ERR_ALIAS, name
    assert call(lib, ws=AT["ids"]) == ERR_ALIAS
    assert call(lib, ws=AT["A"]) == ERR_ALIAS


def test_lora_workspace_size(lib):
    n = ctypes.c_uint64(7)
    f = lib.swiglu_lora_workspace_size
    assert f(64, 128, 256, 2, 16, None) == ERR_NULL
    assert f(64, 12, 256, 2, 16, ctypes.byref(n)) == ERR_SHAPE and n.value == 0
    assert f(64, 128, 256, 9, 16, ctypes.byref(n)) == ERR_SHAPE
    assert f(64, 128, 256, 2, 20, ctypes.byref(n)) == ERR_SHAPE
    assert f(0, 128, 256, 2, 16, ctypes.byref(n)) == 0 and n.value == 0


def test_binding_refuses_what_the_calls_cannot_take():
    z = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="ROCm device"):
        sw.swiglu_route(z, 2)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        sw.swiglu_route(z.half(), 2)
    with pytest.raises(ValueError, match=r"\[M, E\]"):
        sw.swiglu_route(z[0], 2)
    with pytest.raises(TypeError):
        sw.swiglu_route([1.0], 2)
    with pytest.raises(ValueError):
        sw.swiglu_route_backward(z, torch.zeros(4, dtype=torch.int32), z, z)
    A, B = torch.zeros(2, 16, 32, dtype=torch.bfloat16), torch.zeros(2, 24, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="ROCm device"):
        sw.SwigluLora(A, B, torch.zeros(2))
    with pytest.raises(ValueError, match="three dimensions"):
        sw.SwigluLora(A[0], B, torch.zeros(2))
    with pytest.raises(TypeError):
        sw.SwigluLora(None, B, torch.zeros(2))
