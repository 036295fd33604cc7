"""The block's training calls against their definition in 64 bits (needs an MI355X).

Bounds.  Operands are bf16, so products are exact in fp32, and the definition is
computed from the values that the call was given (GU, H) or stored itself (dGU).
With |X||W| the product of the magnitudes:
 - sums: fp32 over n terms, in at least 32-term MFMA blocks of several partial
   sums: n / 16 + 32 roundings of half a step (2^-24) of a partial sum, which is
   at most |X||W|;
 - s(g) = 1 / (1 + e^-g) by the hardware exp2 and reciprocal: the exponent is
   rounded to 2^-24 of |g| log2 e, exp2, sum and reciprocal to 2^-22 each, so s is
   off by less than (1 + |g|) 2^-20, s (1 + g (1 - s)) by (1 + |g|)^2 2^-20, and
   g s by (1 + |g|) |g| 2^-20;
 - |s (1 + g (1 - s))| <= 1.1, |g s| <= |g|;
 - one rounding at the end: bf16 2^-8, fp32 2^-24 relative.
"""
from __future__ import annotations

import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
GUARD = 4096   # elements on both sides of an output


@pytest.fixture(autouse=True)
def _default_dispatch(monkeypatch):
    monkeypatch.delenv("SWIGLU_I_TILE", raising=False)
    monkeypatch.delenv("SWIGLU_TAIL", raising=False)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    sw.load_library()
    return torch.device("cuda:0")


class Guarded:
    """Outputs with guards on both sides, and the check that they are whole."""

    def __init__(self, dev):
        self.dev, self.made = dev, []

    def __call__(self, shape, dtype=BF, fill=float("nan")):
        n = 1
        for d in shape:
            n *= d
        whole = torch.full((n + 2 * GUARD,), 7.0, dtype=dtype, device=self.dev)
        view = whole[GUARD:GUARD + n].view(shape)
        view.fill_(fill)
        self.made.append((whole, n))
        return view

    def check(self):
        for whole, n in self.made:
            assert bool((whole[:GUARD] == 7).all()) and bool((whole[GUARD + n:] == 7).all())


def roundings(n):
    return (n / 16 + 32) * 2.0 ** -24


def product(x, w):
    """(x w, a bound of its error) in 64 bits."""
    x, w = x.double(), w.double()
    return x @ w, roundings(x.shape[1]) * (x.abs() @ w.abs()) + 2.0 ** -126


def rounded(v, err, dtype):
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    return v, err * (1 + half) + v.abs() * half + 2.0 ** -126


def within(got, want, what):
    value, tol = want
    off = (got.double().cpu() - value).abs()
    worst = float((off / tol).max()) if off.numel() else 0.0
    print(f"  {what}: worst error {worst:.3f} of its bound", flush=True)
    assert got.shape == value.shape and bool((off <= tol).all()), f"{what}: {worst}"


def sigmoid(g):
    return torch.sigmoid(g)


def want_forward(a, w, w3):
    g, ge = product(a, w[0::2].t())
    u, ue = product(a, w[1::2].t())
    s = g * sigmoid(g)
    se = 1.1 * ge + (1 + g.abs()) * g.abs() * 2.0 ** -20
    h = rounded(s * u, se * u.abs() + s.abs() * ue + se * ue, BF)
    gu = torch.stack((g, u), 2).flatten(1), torch.stack((ge, ue), 2).flatten(1)
    return h, rounded(*gu, BF)


def want_dgu(dh, dhe, gu):
    g, u = gu[:, 0::2].double(), gu[:, 1::2].double()
    s = sigmoid(g)
    slope = s * (1 + g * (1 - s))
    big = (1 + g.abs())
    dg, du = dh * u * slope, dh * g * s
    dge = u.abs() * (1.1 * dhe + (dh.abs() + dhe) * big * big * 2.0 ** -20)
    due = g.abs() * (dhe + (dh.abs() + dhe) * big * 2.0 ** -20)
    return rounded(torch.stack((dg, du), 2).flatten(1), torch.stack((dge, due), 2).flatten(1), BF)


def want_dw(dy, x, dtype, add=None):
    v, e = product(dy.t(), x)
    if add is not None:
        # the sum with `add` is one more fp32 rounding
        e = e + (v.abs() + e + add.double().abs()) * 2.0 ** -24
        v = v + add.double()
    return rounded(v, e, dtype)


def inputs_of(M, K, N, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF)  # noqa: E731
    return {"A": r(M, K), "W": r(2 * N, K, std=K ** -0.5), "W3": r(K, N, std=N ** -0.5),
            "dOut": r(M, K), "dH": r(M, N), "GU": r(M, 2 * N, std=2.0), "H": r(M, N),
            "addW": torch.randn(2 * N, K, generator=g), "addW3": torch.randn(K, N, generator=g)}


def on(dev, d):
    return {k: v.to(dev) for k, v in d.items()}


def workspace_of(dev, M, N, K):
    n = sw.swiglu_workspace_size(max(M, 1), N, K, "ablation")
    return torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device=dev)


SHAPES = [(1, 8, 8), (1, 520, 264), (2, 72, 1032), (33, 136, 24), (64, 64, 64), (65, 200, 136),
          (127, 264, 520), (129, 72, 72), (130, 1000, 264), (257, 264, 8), (300, 520, 136),
          (513, 136, 1064)]


def check_forward(dev, M, K, N, ws, seed):
    c = inputs_of(M, K, N, seed)
    d, out = on(dev, c), Guarded(dev)
    H, GU, Out = out((M, N)), out((M, 2 * N)), out((M, K))
    got = sw.swiglu_gated_mlp_train(d["A"], d["W"], d["W3"], H, GU, Out, workspace=ws)
    torch.cuda.synchronize()
    assert got == (Out, H, GU) or [t.data_ptr() for t in got] == [t.data_ptr() for t in (Out, H, GU)]
    out.check()
    h, gu = want_forward(c["A"], c["W"], c["W3"])
    within(H, h, "H")
    within(GU, gu, "GU")
    within(Out, rounded(*product(H.cpu(), c["W3"].t()), BF), "Out")
    H2, GU2 = sw.swiglu_fused_gemm_train(d["A"], d["W"], workspace=ws)
    assert torch.equal(H2, H) and torch.equal(GU2, GU)


def check_backward(dev, M, K, N, ws, seed, dtype=BF, add=False, in_place=False):
    c = inputs_of(M, K, N, seed)
    d, out = on(dev, c), Guarded(dev)
    addW, addW3 = c["addW"].to(dtype), c["addW3"].to(dtype)
    dGU = d["GU"].clone() if in_place else out((M, 2 * N))
    GU = dGU if in_place else d["GU"]
    dA, dW, dW3 = out((M, K)), out((2 * N, K), dtype), out((K, N), dtype)
    kw = {"dGU": dGU, "dA": dA, "dW_fused": dW, "dW3t": dW3, "workspace": ws}
    if add and in_place:
        dW.copy_(addW.to(dev))
        dW3.copy_(addW3.to(dev))
        kw |= {"dW_fused_add": dW, "dW3t_add": dW3}
    elif add:
        kw |= {"dW_fused_add": addW.to(dev), "dW3t_add": addW3.to(dev)}
    sw.swiglu_gated_mlp_backward(d["dOut"], d["A"], d["W"], d["W3"], d["H"], GU, **kw)
    torch.cuda.synchronize()
    out.check()
    within(dGU, want_dgu(*product(c["dOut"], c["W3"]), c["GU"]), "dGU")
    own = dGU.cpu()
    within(dA, rounded(*product(own, c["W"]), BF), "dA")
    within(dW, want_dw(own, c["A"], dtype, addW if add else None), "dW_fused")
    within(dW3, want_dw(c["dOut"], c["H"], dtype, addW3 if add else None), "dW3t")
    return d, dGU, dA, dW, dW3


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_forward(dev, M, K, N):
    check_forward(dev, M, K, N, None, 100 + M)
    check_forward(dev, M, K, N, workspace_of(dev, M, N, K), 200 + M)


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_backward(dev, M, K, N):
    check_backward(dev, M, K, N, None, 300 + M)
    check_backward(dev, M, K, N, workspace_of(dev, M, N, K), 400 + M, F32, add=True)


@pytest.mark.parametrize("tile,tail", [("256", "whole"), ("256", "split"), ("128", "whole"),
                                       ("128", "split")])
def test_every_schedule(dev, monkeypatch, tile, tail):
    monkeypatch.setenv("SWIGLU_I_TILE", tile)
    monkeypatch.setenv("SWIGLU_TAIL", tail)
    ws = workspace_of(dev, 300, 520, 264)
    check_forward(dev, 300, 264, 520, ws, 1)
    check_forward(dev, 385, 200, 264, ws, 2)
    check_backward(dev, 300, 264, 520, ws, 3, F32)
    check_backward(dev, 385, 200, 264, ws, 4, BF, add=True)
    check_backward(dev, 513, 328, 136, ws, 5, F32, add=True, in_place=True)


def test_many_tiles(dev):
    """More tiles than compute units, whole rounds and a split last one."""
    M, K, N = 1500, 1096, 2824
    ws = workspace_of(dev, M, N, K)
    check_forward(dev, M, K, N, ws, 11)
    check_backward(dev, M, K, N, ws, 12, F32, add=True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sums_in_place(dev, dtype):
    for M, K, N in ((5, 72, 136), (200, 264, 72), (700, 520, 520)):
        check_backward(dev, M, K, N, workspace_of(dev, M, N, K), 20 + M, dtype, add=True, in_place=True)
        check_backward(dev, M, K, N, None, 30 + M, dtype, add=True)


@pytest.mark.parametrize("M,N,D", [(1, 8, 8), (3, 264, 136), (129, 72, 520), (700, 1032, 264)])
def test_down_proj_backward(dev, M, N, D):
    c = inputs_of(M, D, N, 40 + M)
    d = on(dev, c)
    ws = workspace_of(dev, M, N, D)
    dh = rounded(*product(c["dOut"], c["W3"]), BF)
    for dtype in (BF, F32):
        out = Guarded(dev)
        dH, dW = out((M, N)), out((D, N), dtype)
        sw.swiglu_down_proj_backward(d["dOut"], d["H"], d["W3"], dH, dW, workspace=ws)
        torch.cuda.synchronize()
        out.check()
        within(dH, dh, "dH")
        within(dW, want_dw(c["dOut"], c["H"], dtype), "dW3t")
    # one without the other (their schedules may be others), and the types that are chosen
    only, none = sw.swiglu_down_proj_backward(d["dOut"], d["H"], d["W3"], need_dW=False, workspace=ws)
    assert none is None
    within(only, dh, "dH alone")
    none, only = sw.swiglu_down_proj_backward(d["dOut"], d["H"], d["W3"], need_dH=False, workspace=ws,
                                              grad_dtype=F32)
    assert none is None and only.dtype == F32
    within(only, want_dw(c["dOut"], c["H"], F32), "dW3t alone")
    add = d["addW3"]
    got = sw.swiglu_down_proj_backward(d["dOut"], d["H"], d["W3"], dW3t_add=add)[1]
    assert got.dtype == F32
    within(got, want_dw(c["dOut"], c["H"], F32, c["addW3"]), "dW3t + add")
    assert torch.equal(add.cpu(), c["addW3"])
    assert sw.swiglu_down_proj_backward(d["dOut"], d["H"], d["W3"], need_dH=False,
                                        need_dW=False) == (None, None)


@pytest.mark.parametrize("M,K,N", [(1, 8, 8), (17, 136, 264), (129, 72, 520), (700, 264, 1032)])
def test_fused_gemm_backward(dev, M, K, N):
    c = inputs_of(M, K, N, 50 + M)
    d, out = on(dev, c), Guarded(dev)
    ws = workspace_of(dev, M, N, K)
    dGU, dA, dW = out((M, 2 * N)), out((M, K)), out((2 * N, K), F32)
    sw.swiglu_fused_gemm_backward(d["dH"], d["A"], d["W"], d["GU"], dGU, dA, dW, workspace=ws)
    torch.cuda.synchronize()
    out.check()
    dh = c["dH"].double()
    within(dGU, want_dgu(dh, torch.zeros_like(dh), c["GU"]), "dGU")
    own = dGU.cpu()
    within(dA, rounded(*product(own, c["W"]), BF), "dA")
    within(dW, want_dw(own, c["A"], F32), "dW_fused")
    GU = d["GU"].clone()
    dA2, dW2, dGU2 = sw.swiglu_fused_gemm_backward(d["dH"], d["A"], d["W"], GU, dGU=GU, workspace=ws,
                                                   grad_dtype=F32)
    assert dGU2 is GU and torch.equal(GU, dGU) and torch.equal(dA2, dA) and torch.equal(dW2, dW)
    dA2, none, dGU2 = sw.swiglu_fused_gemm_backward(d["dH"], d["A"], d["W"], d["GU"], need_dW=False,
                                                    workspace=ws)
    assert none is None and torch.equal(dGU2, dGU)
    within(dA2, rounded(*product(own, c["W"]), BF), "dA alone")


def test_frozen_weights_and_first_layer(dev):
    M, K, N = 200, 136, 264
    d, dGU, dA, dW, dW3 = check_backward(dev, M, K, N, None, 60)
    args = (d["dOut"], d["A"], d["W"], d["W3"], d["H"], d["GU"])
    a, w, w3, gu = sw.swiglu_gated_mlp_backward(*args, need_dW=False)
    assert w is None and w3 is None and torch.equal(a, dA) and torch.equal(gu, dGU)
    a, w, w3, gu = sw.swiglu_gated_mlp_backward(*args, need_dA=False)
    assert a is None and torch.equal(w, dW) and torch.equal(w3, dW3) and torch.equal(gu, dGU)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_rows(dev, dtype):
    K, N = 72, 136
    e = lambda *s: torch.empty(*s, dtype=BF, device=dev)  # noqa: E731
    A, W, W3 = e(0, K), torch.ones(2 * N, K, dtype=BF, device=dev), torch.ones(K, N, dtype=BF, device=dev)
    ws = workspace_of(dev, 1, N, K)
    Out, H, GU = sw.swiglu_gated_mlp_train(A, W, W3)
    assert Out.shape == (0, K) and H.shape == (0, N) and GU.shape == (0, 2 * N)
    out = Guarded(dev)
    dW, dW3 = out((2 * N, K), dtype), out((K, N), dtype)
    sw.swiglu_gated_mlp_backward(e(0, K), A, W, W3, H, GU, dW_fused=dW, dW3t=dW3, workspace=ws)
    assert bool((dW == 0).all()) and bool((dW3 == 0).all())
    add = torch.randn(2 * N, K, device=dev).to(dtype)
    sw.swiglu_fused_gemm_backward(H, A, W, GU, dW_fused=dW, dW_fused_add=add, workspace=ws)
    assert torch.equal(dW, add)
    dW3.fill_(3.0)
    sw.swiglu_down_proj_backward(e(0, K), H, W3, dW3t=dW3, dW3t_add=dW3, workspace=ws)
    assert bool((dW3 == 3).all())
    torch.cuda.synchronize()
    out.check()


def test_extreme_gates(dev):
    """Saturated and huge Gates: finite gradients, as the limits of the formula."""
    M, K, N = 40, 64, 72
    c = inputs_of(M, K, N, 70)
    big = torch.tensor([0.0, -0.0, 90.0, -90.0, 200.0, -200.0, 3e38, -3e38, 1e-38, -1e-38], dtype=BF)
    c["GU"][:, 0::2] = big[torch.arange(M * N).view(M, N) % 10]
    d = on(dev, c)
    dA, dW, dGU = sw.swiglu_fused_gemm_backward(d["dH"], d["A"], d["W"], d["GU"])
    torch.cuda.synchronize()
    g, u, dh = c["GU"][:, 0::2].double(), c["GU"][:, 1::2].double(), c["dH"].double()
    up = g > 50
    down = g < -50
    got = dGU.cpu().double()
    dg, du = got[:, 0::2], got[:, 1::2]
    # far to the right the unit passes (H = g u), far to the left it is shut
    assert torch.allclose(dg[up], (dh * u)[up], rtol=2.0 ** -7, atol=0)
    assert bool((dg[down] == 0).all()) and bool((du[down] == 0).all())
    near = ~(up | down)
    assert torch.allclose(dg[near], 0.5 * (dh * u)[near], rtol=2.0 ** -7, atol=1e-37)
    fine = up & ((dh * g).abs() < 3e38)
    assert torch.allclose(du[fine], (dh * g)[fine], rtol=2.0 ** -7, atol=0)


def test_broken_row_stays_its_own(dev):
    """NaN in one row of dOut: that row of dGU and dA, and the weights' gradients."""
    M, K, N = 300, 136, 264
    c = inputs_of(M, K, N, 80)
    d = on(dev, c)
    args = lambda x: (x, d["A"], d["W"], d["W3"], d["H"], d["GU"])  # noqa: E731
    clean = sw.swiglu_gated_mlp_backward(*args(d["dOut"]))
    bad = d["dOut"].clone()
    bad[77, 5] = float("nan")
    dA, dW, dW3, dGU = sw.swiglu_gated_mlp_backward(*args(bad))
    keep = torch.arange(M, device=dev) != 77
    assert torch.equal(dA[keep], clean[0][keep]) and torch.equal(dGU[keep], clean[3][keep])
    assert bool(dA[77].isnan().all()) and bool(dGU[77].isnan().all()) and bool(dW.isnan().all())
    rows = torch.arange(K, device=dev) != 5
    assert torch.equal(dW3[rows], clean[2][rows]) and bool(dW3[5].isnan().all())


def test_differences(dev):
    """The gradients along a direction against differences of the block in 64 bits.

    The kernels' gradients take GU and H rounded to bf16.  With e = 2^-8: G off by
    e |G| changes s (1 + G (1 - s)), whose slope is at most 0.5, by 0.5 e |G|; U off
    by e |U|; G s by 1.1 e |G|; dGU is rounded by e of itself, and so are the
    gradients; H by e |H| in dW3t."""
    M, K, N = 24, 72, 136
    c = inputs_of(M, K, N, 90)
    d = on(dev, c)
    A, W, W3, dOut = (c[n].double() for n in ("A", "W", "W3", "dOut"))
    Out, H, GU = sw.swiglu_gated_mlp_train(d["A"], d["W"], d["W3"])
    dA, dW, dW3, _ = sw.swiglu_gated_mlp_backward(d["dOut"], d["A"], d["W"], d["W3"], H, GU,
                                                  grad_dtype=F32)

    def loss(a, w, w3):
        g, u = a @ w[0::2].t(), a @ w[1::2].t()
        return float(((g * torch.sigmoid(g) * u) @ w3.t() * dOut).sum())

    e = 2.0 ** -8
    g, u = A @ W[0::2].t(), A @ W[1::2].t()
    dh = (dOut @ W3).abs()
    dg_tol = dh * u.abs() * (1.1 * e + 0.5 * e * g.abs() + 1.1 * e) * 1.1
    du_tol = dh * g.abs() * (1.1 * e + e) * 1.1
    dgu_tol = torch.stack((dg_tol, du_tol), 2).flatten(1)
    h = (g * torch.sigmoid(g) * u).abs()
    tols = {"A": dgu_tol @ W.abs() + dA.double().cpu().abs() * e,
            "W": dgu_tol.t() @ A.abs(),
            "W3": dOut.abs().t() @ h * e * 1.1}
    gen = torch.Generator().manual_seed(91)
    for name, got in (("A", dA), ("W", dW), ("W3", dW3)):
        base = {"A": A, "W": W, "W3": W3}
        for _ in range(4):
            v = torch.randn(base[name].shape, generator=gen, dtype=torch.float64)
            step = 1e-4
            lo, hi = ({**base, name: base[name] + s * step * v} for s in (-1, 1))
            slope = (loss(*hi.values()) - loss(*lo.values())) / (2 * step)
            mine = float((got.double().cpu() * v).sum())
            # independent roundings: the bound of their sum is the sum of the bounds
            tol = float((tols[name] * v.abs()).sum())
            print(f"  {name}: {mine:.5f} against {slope:.5f}, bound {tol:.5f}", flush=True)
            assert abs(mine - slope) <= tol + 1e-4 * abs(slope)


def test_same_call_same_bits_and_other_streams(dev):
    M, K, N = 385, 520, 1032
    d = on(dev, inputs_of(M, K, N, 95))
    ws = [workspace_of(dev, M, N, K) for _ in range(2)]

    def both(w):
        Out, H, GU = sw.swiglu_gated_mlp_train(d["A"], d["W"], d["W3"], workspace=w)
        return (Out, H, GU) + sw.swiglu_gated_mlp_backward(d["dOut"], d["A"], d["W"], d["W3"], H, GU,
                                                           grad_dtype=F32, workspace=w)

    first = both(ws[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    got = []
    for s, w in zip(streams, ws):
        with torch.cuda.stream(s):
            got.append(both(w))
    torch.cuda.synchronize()
    for other in got:
        assert all(torch.equal(a, b) for a, b in zip(first, other))


def test_captured_step(dev):
    """Forward and backward in a graph, replayed beside eager calls, on new inputs."""
    M, K, N = 200, 264, 520
    d = on(dev, inputs_of(M, K, N, 96))
    ws, eager_ws = (workspace_of(dev, M, N, K) for _ in range(2))
    outs = {n: torch.empty(s, dtype=t, device=dev) for n, s, t in (
        ("H", (M, N), BF), ("GU", (M, 2 * N), BF), ("Out", (M, K), BF), ("dGU", (M, 2 * N), BF),
        ("dA", (M, K), BF), ("dW", (2 * N, K), F32), ("dW3", (K, N), F32))}

    def step(w, o):
        sw.swiglu_gated_mlp_train(d["A"], d["W"], d["W3"], o["H"], o["GU"], o["Out"], workspace=w)
        sw.swiglu_gated_mlp_backward(d["dOut"], d["A"], d["W"], d["W3"], o["H"], o["GU"],
                                     dGU=o["dGU"], dA=o["dA"], dW_fused=o["dW"], dW3t=o["dW3"],
                                     workspace=w)

    step(ws, outs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step(ws, outs)
    for seed in (97, 98, 99):
        for k, v in inputs_of(M, K, N, seed).items():
            d[k].copy_(v)
        for t in outs.values():
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        mine = {k: torch.empty_like(v) for k, v in outs.items()}
        step(eager_ws, mine)
        torch.cuda.synchronize()
        assert all(torch.equal(outs[k], mine[k]) for k in outs)


def test_binding_refuses(dev):
    M, K, N = 16, 64, 72
    d = on(dev, inputs_of(M, K, N, 5))
    args = [d[n] for n in ("dOut", "A", "W", "W3", "H", "GU")]
    with pytest.raises(TypeError):
        sw.swiglu_gated_mlp_backward(*args, grad_dtype=torch.float16)
    with pytest.raises(TypeError):
        sw.swiglu_gated_mlp_backward(*args, dW_fused=torch.empty(2 * N, K, dtype=F32, device=dev),
                                     dW3t=torch.empty(K, N, dtype=BF, device=dev))
    with pytest.raises(ValueError):
        sw.swiglu_gated_mlp_backward(*args, need_dW=False, dW3t_add=d["addW3"])
    with pytest.raises(ValueError):
        sw.swiglu_gated_mlp_backward(*args, need_dA=False, dA=torch.empty(M, K, dtype=BF, device=dev))
    with pytest.raises(ValueError):
        sw.swiglu_gated_mlp_backward(d["dOut"][:8], *args[1:])
    with pytest.raises(ValueError):
        sw.swiglu_gated_mlp_backward(*args[:5], d["GU"][:, :N].contiguous())
    with pytest.raises(ValueError):
        sw.swiglu_gated_mlp_backward(d["dOut"].t().contiguous().t(), *args[1:])
    with pytest.raises(sw.SwigluError) as e:
        sw.swiglu_gated_mlp_backward(*args, dA=d["A"])
    assert e.value.status == sw.SWIGLU_ERR_ALIAS
