"""Refusals of the training calls and of the calls on 4-bit weights (no GPU): invalid
arguments are rejected before any HIP call.  Fake device addresses are used;
validation fails before they could be dereferenced."""
import os

import pytest

from gated_mlp_gemm_amd import swiglu as sw

ERR_NULL, ERR_SHAPE, ERR_ALIGN = sw.SWIGLU_ERR_NULL, sw.SWIGLU_ERR_SHAPE, sw.SWIGLU_ERR_ALIGN
ERR_UNSUP, ERR_ALIAS = sw.SWIGLU_ERR_UNSUPPORTED, sw.SWIGLU_ERR_ALIAS

NAMES = ("A", "W", "W3", "H", "GU", "Out", "dOut", "dH", "dGU", "dA", "dW", "dW3", "addW", "addW3",
         "q", "s", "q3", "s3", "X", "ws")
AT = {n: 0x100_0000_0000 * (i + 1) for i, n in enumerate(NAMES)}


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sw.LIBRARY):
        pytest.fail("libswiglu.so is not built (python -m gated_mlp_gemm_amd.build)")
    return sw.load_library()


def fused_train(lib, M=64, N=72, K=136, wsb=1 << 20, **kw):
    p = {**AT, **kw}
    return lib.swiglu_fused_gemm_train(p["A"], p["W"], p["H"], p["GU"], M, N, K, p["ws"], wsb, None)


def mlp_train(lib, M=64, N=72, K=136, wsb=1 << 20, **kw):
    p = {**AT, **kw}
    return lib.swiglu_gated_mlp_train(p["A"], p["W"], p["W3"], p["H"], p["GU"], p["Out"], M, N, K,
                                      p["ws"], wsb, None)


def down_back(lib, M=64, N=72, K=136, kind=0, wsb=1 << 20, **kw):
    p = {**AT, **kw}
    return lib.swiglu_down_proj_backward(p["dOut"], p["H"], p["W3"], p["dH"], p["dW3"], p["addW3"],
                                         kind, M, N, K, p["ws"], wsb, None)


def fused_back(lib, M=64, N=72, K=136, kind=0, wsb=1 << 20, **kw):
    p = {**AT, **kw}
    return lib.swiglu_fused_gemm_backward(p["dH"], p["A"], p["W"], p["GU"], p["dGU"], p["dA"],
                                          p["dW"], p["addW"], kind, M, N, K, p["ws"], wsb, None)


def mlp_back(lib, M=64, N=72, K=136, kind=0, wsb=1 << 20, **kw):
    p = {**AT, **kw}
    return lib.swiglu_gated_mlp_backward(p["dOut"], p["A"], p["W"], p["W3"], p["H"], p["GU"],
                                         p["dGU"], p["dA"], p["dW"], p["addW"], p["dW3"], p["addW3"],
                                         kind, M, N, K, p["ws"], wsb, None)


def quantize(lib, M=64, K=96, **kw):
    p = {**AT, **kw}
    return lib.swiglu_quantize_mx4(p["X"], p["q"], p["s"], M, K, None)


def dequantize(lib, M=64, K=96, **kw):
    p = {**AT, **kw}
    return lib.swiglu_dequantize_mx4(p["q"], p["s"], p["X"], M, K, None)


def fused_mx4(lib, M=64, N=64, K=96, wsb=1 << 20, **kw):
    p = {**AT, **kw}
    return lib.swiglu_fused_gemm_mx4(p["A"], p["q"], p["s"], p["H"], M, N, K, p["ws"], wsb, None)


def down_mx4(lib, M=64, N=64, K=96, wsb=1 << 20, **kw):
    p = {**AT, **kw}
    return lib.swiglu_down_proj_mx4(p["H"], p["q3"], p["s3"], p["Out"], M, N, K, p["ws"], wsb, None)


def mlp_mx4(lib, M=64, N=64, K=96, wsb=1 << 20, **kw):
    p = {**AT, **kw}
    return lib.swiglu_gated_mlp_mx4(p["A"], p["q"], p["s"], p["q3"], p["s3"], p["H"], p["Out"], M, N,
                                    K, p["ws"], wsb, None)


READS = {fused_train: ("A", "W"), mlp_train: ("A", "W", "W3"), down_back: ("dOut", "H", "W3"),
         fused_back: ("dH", "A", "W", "GU"), mlp_back: ("dOut", "A", "W", "W3", "H", "GU"),
         fused_mx4: ("A", "q", "s"), down_mx4: ("H", "q3", "s3"), mlp_mx4: ("A", "q", "s", "q3", "s3")}
WRITES = {fused_train: ("H", "GU"), mlp_train: ("H", "GU", "Out"), down_back: ("dH", "dW3"),
          fused_back: ("dGU", "dA", "dW"), mlp_back: ("dGU", "dA", "dW", "dW3"), fused_mx4: ("H",),
          down_mx4: ("Out",), mlp_mx4: ("H", "Out")}
OPTIONAL = {"dH", "dA", "dW", "dW3"}


@pytest.mark.parametrize("call", list(READS))
def test_shapes(lib, call):
    assert call(lib, M=-1) == ERR_SHAPE
    assert call(lib, N=-8) == ERR_SHAPE
    assert call(lib, N=12) == ERR_SHAPE
    assert call(lib, K=12) == ERR_SHAPE
    assert call(lib, K=0) == (0 if call is down_mx4 else ERR_SHAPE)   # (D = 0: no columns)
    assert call(lib, K=(1 << 22) + 8) == ERR_SHAPE
    assert call(lib, N=(1 << 22) + 8) == ERR_SHAPE


@pytest.mark.parametrize("call", [fused_train, mlp_train, down_back, fused_back, mlp_back])
def test_limits_of_training(lib, call):
    if call is down_back:
        assert call(lib, N=(1 << 21) + 8) == ERR_SHAPE
        assert call(lib, K=(1 << 21) + 8) == ERR_SHAPE
    else:
        assert call(lib, N=(1 << 20) + 8) == ERR_SHAPE
    assert call(lib, M=(1 << 30) + 1) == ERR_SHAPE


@pytest.mark.parametrize("call", list(READS))
def test_pointers(lib, call):
    for name in READS[call]:
        assert call(lib, **{name: None}) == ERR_NULL, name
        assert call(lib, **{name: AT[name] + 2}) == ERR_ALIGN, name
        for out in WRITES[call]:
            if (name, out) != ("GU", "dGU"):
                assert call(lib, **{out: AT[name]}) == ERR_ALIAS, (name, out)
            assert call(lib, **{out: AT[name] + 16}) == ERR_ALIAS, (name, out)
    for name in WRITES[call]:
        assert call(lib, **{name: AT[name] + 8}) == ERR_ALIGN, name
        if name not in OPTIONAL:
            assert call(lib, **{name: None}) == ERR_NULL, name
        for other in WRITES[call]:
            if other != name:
                assert call(lib, **{name: AT[other]}) == ERR_ALIAS, (name, other)
    assert call(lib, ws=AT["ws"] + 128) == ERR_ALIGN
    assert call(lib, ws=AT[WRITES[call][0]]) == ERR_ALIAS
    assert call(lib, ws=AT[READS[call][0]]) == ERR_ALIAS


@pytest.mark.parametrize("call", [down_back, fused_back, mlp_back])
def test_gradient_arguments(lib, call):
    assert call(lib, kind=2) == ERR_UNSUP
    assert call(lib, kind=-1) == ERR_UNSUP
    weights = [("dW3", "addW3")] if call is down_back else [("dW", "addW")]
    if call is mlp_back:
        weights.append(("dW3", "addW3"))
    for dw, add in weights:
        assert call(lib, **{dw: None}) == ERR_NULL          # a sum without a gradient
        assert call(lib, **{add: AT[add] + 2}) == ERR_ALIGN
        assert call(lib, **{add: AT[dw] + 16}) == ERR_ALIAS  # neither apart nor the same
        assert call(lib, **{add: AT["ws"]}) == ERR_ALIAS
    if call is down_back:
        assert call(lib, dH=None, dW3=None, addW3=None) == ERR_NULL
    # fp32 gradients are twice as long
    dw, n = ("dW3", 72 * 136) if call is down_back else ("dW", 2 * 72 * 136)
    read = READS[call][0]
    at = AT[read] - 2 * n - 64
    assert call(lib, kind=0, **{dw: at}) == ERR_ALIAS


def test_dgu_may_be_gu_only_whole(lib):
    for call in (fused_back, mlp_back):
        assert call(lib, dGU=AT["GU"] + 32) == ERR_ALIAS
        assert call(lib, GU=AT["dGU"] + 32) == ERR_ALIAS


@pytest.mark.parametrize("call", [quantize, dequantize])
def test_quantizer(lib, call):
    assert call(lib, M=-1) == ERR_SHAPE
    assert call(lib, M=(1 << 23) + 1) == ERR_SHAPE
    for K in (0, 8, 40, -32, (1 << 21) + 32):
        assert call(lib, K=K) == ERR_SHAPE
    for name in ("X", "q", "s"):
        assert call(lib, **{name: None}) == ERR_NULL
    assert call(lib, X=AT["X"] + 8) == ERR_ALIGN
    assert call(lib, q=AT["q"] + 8) == ERR_ALIGN
    assert call(lib, M=0, X=None, q=None, s=None) == 0
    out = "q" if call is quantize else "X"
    assert call(lib, **{out: AT["s"] - 64}) == ERR_ALIAS
    assert call(lib, s=AT["q"] + 64 * 48 - 1) == ERR_ALIAS if call is quantize else True


def test_groups_are_whole(lib):
    for call in (fused_mx4, mlp_mx4):
        assert call(lib, K=72) == ERR_SHAPE
        assert call(lib, s=AT["s"] + 2) == ERR_ALIGN
    for call in (down_mx4, mlp_mx4):
        assert call(lib, N=72) == ERR_SHAPE
        assert call(lib, s3=AT["s3"] + 2) == ERR_ALIGN


def test_nothing_to_do(lib):
    none = dict.fromkeys(NAMES)
    assert fused_train(lib, M=0, **none) == 0
    assert mlp_train(lib, M=0, **none) == 0
    assert fused_train(lib, N=0, **none) == 0
    assert fused_mx4(lib, M=0, **none) == 0 and fused_mx4(lib, N=0, **none) == 0
    assert down_mx4(lib, M=0, **none) == 0 and mlp_mx4(lib, M=0, **none) == 0
    # no rows: a gradient's memory is still needed for its zeros, and dGU is not
    assert down_back(lib, M=0, **none) == ERR_NULL
