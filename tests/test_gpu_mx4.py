"""4-bit weights against their definition in 64 bits (needs an MI355X).

Bounds.  The numbers that codes and scales stand for are exact in bf16, so products
are exact in fp32.  With |X||W| the product of the magnitudes:
 - sums: fp32 over K terms, in at least 32-term MFMA blocks of several partial
   sums: K / 16 + 32 roundings of half a step (2^-24) of a partial sum, which is
   at most |X||W|;
 - SiLU: |SiLU'| <= 1.1, the hardware exp2 and reciprocal (1 + |g|) 2^-20 of |g|;
 - one rounding to bf16 (2^-8 relative).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
LADDER = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


@pytest.fixture(autouse=True)
def _default_dispatch(monkeypatch):
    monkeypatch.delenv("SWIGLU_I_TILE", raising=False)
    monkeypatch.delenv("SWIGLU_TAIL", raising=False)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    sw.load_library()
    return torch.device("cuda:0")


# --- the format, number by number -------------------------------------------
def values_of(q, s):
    """[rows, K] in 64 bits of codes and scales (uint8 CPU tensors)."""
    q, s = q.numpy(), s.numpy().astype(np.int64)
    code = np.empty((q.shape[0], 2 * q.shape[1]), dtype=np.int64)
    code[:, 0::2], code[:, 1::2] = q & 15, q >> 4
    v = LADDER[code & 7] * np.where(code & 8, -1.0, 1.0)
    size = np.where(s == 255, np.nan, np.ldexp(1.0, (s - 127).astype(np.int32)))
    return torch.from_numpy(v * np.repeat(size, 32, axis=1))


def quantized(x):
    """(numbers, scales) of bf16 x: every code's distance compared, ties to the even code."""
    v = x.double().numpy().reshape(x.shape[0], -1, 32)
    bits = x.view(torch.int16).numpy().astype(np.int64).reshape(v.shape) & 0x7FFF
    e = bits.max(axis=2) >> 7
    s = np.where(e == 255, 255, np.maximum(e - 2, 0))
    size = np.ldexp(1.0, (s - 127).astype(np.int32))
    with np.errstate(invalid="ignore"):
        u = np.abs(v) / size[..., None]
        far = np.abs(u[..., None] - LADDER)
        best = far.min(axis=-1, keepdims=True)
        near = far == best                       # one code, or two neighbours
        even = near & (np.arange(8) % 2 == 0)
        pick = np.where((near.sum(-1) > 1), even.argmax(-1), near.argmax(-1))
    code = LADDER[pick] * np.where(v < 0, -1.0, 1.0) * size[..., None]
    code[s == 255] = np.nan
    return torch.from_numpy(code.reshape(x.shape)), torch.from_numpy(s.astype(np.uint8))


def check_quantizer(dev, x):
    q, s = sw.swiglu_quantize_mx4(x.to(dev))
    back = sw.swiglu_dequantize_mx4(q, s)
    torch.cuda.synchronize()
    want, want_s = quantized(x)
    assert torch.equal(s.cpu(), want_s)
    assert torch.allclose(values_of(q.cpu(), s.cpu()), want, rtol=0, atol=0, equal_nan=True)
    assert torch.allclose(back.cpu().double(), want, rtol=0, atol=0, equal_nan=True)


def test_every_bf16_number(dev):
    """Each of the 65536 patterns beside each of some largest magnitudes of its group."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF).view(-1, 1)
    rows = []
    for top in (0.0, 1.0, -6.0, 7.96875, 2.0 ** 120, 2.0 ** -120, 2.0 ** -126, 2.0 ** -133, 3e38):
        rows.append(torch.cat([every, torch.full_like(every, top).expand(-1, 31)], 1))
    check_quantizer(dev, torch.cat(rows))
    # borders between codes, below and above by a bf16 step, in every size of group
    steps = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    near = torch.cat([steps * (1 + d) for d in (-2.0 ** -7, 0.0, 2.0 ** -7)])
    base = torch.cat([near, -near[:10], torch.tensor([4.0])]).repeat(250, 1)[:, :32]
    check_quantizer(dev, (base * torch.pow(2.0, torch.arange(-125.0, 125.0).double())[:, None]).to(BF))


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (1, 8192), (257, 3616), (1000, 64)])
def test_quantizer_shapes(dev, rows, K):
    g = torch.Generator().manual_seed(rows + K)
    x = (torch.randn(rows, K, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))).to(BF)
    check_quantizer(dev, x)
    q = torch.full((rows * K // 2 + 64,), 0xA5, dtype=torch.uint8, device=dev)
    s = torch.full((rows * K // 32 + 64,), 0xA5, dtype=torch.uint8, device=dev)
    nq, ns = rows * K // 2, rows * K // 32
    sw.swiglu_quantize_mx4(x.to(dev), q[:nq].view(rows, -1), s[1:1 + ns].view(rows, -1))
    torch.cuda.synchronize()
    assert bool((q[nq:] == 0xA5).all()) and bool((s[1 + ns:] == 0xA5).all()) and int(s[0]) == 0xA5
    assert torch.equal(s[1:1 + ns].cpu().view(rows, -1), quantized(x)[1])
    e = torch.empty(0, K, dtype=BF, device=dev)
    q0, s0 = sw.swiglu_quantize_mx4(e)
    assert q0.shape == (0, K // 2) and s0.shape == (0, K // 32)
    assert sw.swiglu_dequantize_mx4(q0, s0).shape == (0, K)


# --- the products -------------------------------------------------------------
def roundings(n):
    return (n / 16 + 32) * 2.0 ** -24


def product(x, w):
    x = x.double()
    return x @ w.t(), roundings(x.shape[1]) * (x.abs() @ w.abs().t()) + 2.0 ** -126


def rounded(v, err):
    return v, err * (1 + 2.0 ** -8) + v.abs() * 2.0 ** -8 + 2.0 ** -126


def gated(x, w):
    g, ge = product(x, w[0::2])
    u, ue = product(x, w[1::2])
    s = g * torch.sigmoid(g)
    se = 1.1 * ge + (1 + g.abs()) * g.abs() * 2.0 ** -20
    return rounded(s * u, se * u.abs() + s.abs() * ue + se * ue)


def within(got, want, what):
    value, tol = want
    off = (got.double().cpu() - value).abs()
    worst = float((off / tol).max()) if off.numel() else 0.0
    print(f"  {what}: worst error {worst:.3f} of its bound", flush=True)
    assert got.shape == value.shape and bool((off <= tol).all()), f"{what}: {worst}"


def codes_of(g, rows, K):
    """Any codes, scales about those of a weight of K inputs."""
    q = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8)
    s = 125 - int(np.log2(K) / 2) + torch.randint(-3, 3, (rows, K // 32), generator=g)
    return q, s.to(torch.uint8)


def workspace_of(dev, M, N, K):
    n = sw.swiglu_workspace_size(max(M, 1), N, K, "ablation")
    return torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device=dev)


class Guarded:
    def __init__(self, dev):
        self.dev, self.made = dev, []

    def __call__(self, shape):
        n = shape[0] * shape[1]
        whole = torch.full((n + 8192,), 7.0, dtype=BF, device=self.dev)
        view = whole[4096:4096 + n].view(shape)
        view.fill_(float("nan"))
        self.made.append((whole, n))
        return view

    def check(self):
        for whole, n in self.made:
            assert bool((whole[:4096] == 7).all()) and bool((whole[4096 + n:] == 7).all())


def check_block(dev, M, K, N, ws, seed):
    g = torch.Generator().manual_seed(seed)
    A = torch.randn(M, K, generator=g).to(BF)
    (wq, wsc), (vq, vsc) = codes_of(g, 2 * N, K), codes_of(g, K, N)
    d = [t.to(dev) for t in (A, wq, wsc, vq, vsc)]
    out = Guarded(dev)
    H, Out = out((M, N)), out((M, K))
    sw.swiglu_gated_mlp_mx4(*d, H=H, Out=Out, workspace=ws)
    torch.cuda.synchronize()
    out.check()
    within(H, gated(A, values_of(wq, wsc)), f"H M={M} K={K} N={N}")
    within(Out, rounded(*product(H.cpu(), values_of(vq, vsc))), "Out")
    Y = sw.swiglu_fused_gemm_mx4(d[0], d[1], d[2], workspace=ws)
    Z = sw.swiglu_down_proj_mx4(H, d[3], d[4], workspace=ws)
    assert torch.equal(Y, H) and torch.equal(Z, Out)


SHAPES = [(1, 32, 32), (1, 544, 288), (2, 96, 1056), (3, 1056, 96), (5, 2080, 160), (8, 64, 64),
          (9, 320, 544), (16, 1024, 256), (17, 288, 96), (31, 160, 2080), (33, 608, 32),
          (64, 64, 1056), (65, 224, 160), (127, 288, 544), (129, 96, 96), (130, 1056, 288),
          (257, 288, 32), (300, 544, 160), (513, 160, 1056)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_block(dev, M, K, N):
    check_block(dev, M, K, N, None, M)
    check_block(dev, M, K, N, workspace_of(dev, M, N, K), 1000 + M)


@pytest.mark.parametrize("M", [1, 4, 16, 24, 48, 64, 100, 128])
def test_wide_and_long(dev, M):
    """More tiles than compute units, and a long contraction of few columns."""
    K, N = 544, 16480
    check_block(dev, M, K, N, workspace_of(dev, M, N, K), 30 + M)
    check_block(dev, M, 8224, 64, workspace_of(dev, M, 64, 8224), 60 + M)


@pytest.mark.parametrize("tile,tail", [("256", "whole"), ("256", "split"), ("128", "whole"),
                                       ("128", "split")])
def test_every_schedule(dev, monkeypatch, tile, tail):
    monkeypatch.setenv("SWIGLU_I_TILE", tile)
    monkeypatch.setenv("SWIGLU_TAIL", tail)
    for M, K, N in ((300, 544, 288), (385, 224, 288), (140, 32, 544), (60, 544, 160)):
        check_block(dev, M, K, N, workspace_of(dev, M, N, K), M)


def test_many_tiles(dev):
    M, K, N = 1500, 1120, 2848
    check_block(dev, M, K, N, workspace_of(dev, M, N, K), 5)


@pytest.mark.parametrize("M", [1, 7, 24, 70, 200])
def test_columns_of_any_multiple_of_eight(dev, M):
    g = torch.Generator().manual_seed(M)
    for N, K in ((8, 64), (24, 320), (136, 96)):
        x = torch.randn(M, K, generator=g).to(BF)
        q, s = codes_of(g, 2 * N, K)
        y = sw.swiglu_fused_gemm_mx4(x.to(dev), q.to(dev), s.to(dev))
        within(y, gated(x, values_of(q, s)), "Y")
        q, s = codes_of(g, N, K)
        y = sw.swiglu_down_proj_mx4(x.to(dev), q.to(dev), s.to(dev))
        within(y, rounded(*product(x, values_of(q, s))), "Out")


@pytest.mark.parametrize("M", [1, 5, 16, 24, 60, 128, 300])
def test_like_the_bf16_calls(dev, M):
    """What the calls on bf16 weights compute of the numbers that the codes stand for."""
    K, N = 544, 1056
    g = torch.Generator().manual_seed(M)
    A = torch.randn(M, K, generator=g).to(BF).to(dev)
    W = (torch.randn(2 * N, K, generator=g) / K ** 0.5).to(BF).to(dev)
    q, s = sw.swiglu_quantize_mx4(W)
    y = sw.swiglu_fused_gemm_mx4(A, q, s)
    z = sw.swiglu_fused_gemm(A, sw.swiglu_dequantize_mx4(q, s))
    rel = float((y.double() - z.double()).norm() / z.double().norm())
    # two roundings of nearly the same sums: they differ where a sum lies at a border
    assert rel < 2.0 ** -10, rel


@pytest.mark.parametrize("M", [1, 3, 20, 70, 200])
def test_broken_groups_and_rows_stay_their_own(dev, M):
    K, N = 320, 288
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=g).to(BF)
    q, s = codes_of(g, N, K)
    clean = sw.swiglu_down_proj_mx4(x.to(dev), q.to(dev), s.to(dev))
    s2 = s.clone()
    s2[77, 4] = 255                                  # a group that is NaN
    s2[N - 1, K // 32 - 1] = 255
    s2[5, 0] = 0                                     # and tiny ones: 2^-127
    y = sw.swiglu_down_proj_mx4(x.to(dev), q.to(dev), s2.to(dev))
    hit = torch.zeros(N, dtype=torch.bool, device=dev)
    hit[[77, N - 1]] = True
    assert bool(y[:, hit].isnan().all())
    hit[5] = True
    assert torch.equal(y[:, ~hit], clean[:, ~hit])
    v = values_of(q, s2)
    within(y[:, 5:6], rounded(*product(x, v[5:6])), "tiny group")
    bad = x.clone()
    bad[M // 2, 33] = float("nan")
    y = sw.swiglu_down_proj_mx4(bad.to(dev), q.to(dev), s.to(dev))
    keep = torch.arange(M, device=dev) != M // 2
    assert bool(y[M // 2].isnan().all()) and torch.equal(y[keep], clean[keep])
    # an infinity: infinite where its weight is not zero, NaN where it is
    bad[M // 2, 33] = float("inf")
    y = sw.swiglu_down_proj_mx4(bad.to(dev), q.to(dev), s.to(dev))[M // 2].cpu().double()
    w = values_of(q, s)[:, 33]
    assert bool(y[w == 0].isnan().all()) and torch.equal(y[w != 0], w[w != 0].sign() * float("inf"))


# Weights of less than four groups a row, where a group's neighbours are other rows'.
@pytest.mark.parametrize("M", [1, 6, 20, 40, 64, 100, 300])
@pytest.mark.parametrize("K", [32, 64, 96, 160])
def test_broken_groups_of_short_rows(dev, M, K):
    N = 312
    g = torch.Generator().manual_seed(M * K)
    x = torch.randn(M, K, generator=g).to(BF).to(dev)
    q, s = (t.to(dev) for t in codes_of(g, N, K))
    hit = torch.arange(N, device=dev) % 3 == 1
    clean = sw.swiglu_down_proj_mx4(x, q, s)
    for group in range(K // 32):
        s2 = s.clone()
        s2[hit, group] = 255
        y = sw.swiglu_down_proj_mx4(x, q, s2)
        assert bool(y[:, hit].isnan().all()) and torch.equal(y[:, ~hit], clean[:, ~hit])


# Rows too long for a compute unit's LDS beside the activations of the few-row kernel.
@pytest.mark.parametrize("M,K", [(1, 1 << 18), (4, 1 << 17), (24, 96 * 1024), (64, 131072 + 32)])
def test_very_long_rows(dev, M, K):
    N = 24
    g = torch.Generator(device=dev).manual_seed(M)
    x = torch.randn(M, K, generator=g, device=dev).to(BF)
    q = torch.randint(0, 256, (N, K // 2), generator=g, device=dev, dtype=torch.uint8)
    s = torch.randint(115, 119, (N, K // 32), generator=g, device=dev).to(torch.uint8)
    v = sw.swiglu_dequantize_mx4(q, s)
    assert torch.equal(v.cpu().double(), values_of(q.cpu(), s.cpu()))
    y = sw.swiglu_down_proj_mx4(x, q, s)
    within(y, rounded(*product(x.cpu(), v.cpu().double())), f"M={M} K={K}")


def test_other_streams_and_graphs(dev):
    K, N = 544, 1056
    g = torch.Generator().manual_seed(9)
    codes = [t.to(dev) for t in (*codes_of(g, 2 * N, K), *codes_of(g, K, N))]
    for M in (1, 12, 40, 200):
        A = torch.randn(M, K, generator=g).to(BF).to(dev)
        ws = [workspace_of(dev, M, N, K) for _ in range(3)]
        first = sw.swiglu_gated_mlp_mx4(A, *codes, workspace=ws[0])
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(dev) for _ in range(2)]
        got = []
        for st, w in zip(streams, ws):
            with torch.cuda.stream(st):
                got.append(sw.swiglu_gated_mlp_mx4(A, *codes, workspace=w))
        torch.cuda.synchronize()
        for o in got:
            assert torch.equal(o[0], first[0]) and torch.equal(o[1], first[1])
        H, Out = torch.empty_like(first[1]), torch.empty_like(first[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(streams[0]):
            with torch.cuda.graph(graph, stream=streams[0]):
                sw.swiglu_gated_mlp_mx4(A, *codes, H=H, Out=Out, workspace=ws[0])
        for _ in range(3):
            A.copy_(torch.randn(M, K, generator=g).to(BF))
            H.fill_(float("nan"))
            Out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            want = sw.swiglu_gated_mlp_mx4(A, *codes, workspace=ws[2])
            torch.cuda.synchronize()
            assert torch.equal(Out, want[0]) and torch.equal(H, want[1])


def test_trained_then_served(dev):
    """A training step of the block, then the block with its weights in 4 bits: both
    close to the same numbers as far as 4 bits allow (scales of powers of two: a weight
    is off by at most an eighth of its group's largest, or a quarter above 6)."""
    M, K, N = 48, 256, 544
    g = torch.Generator().manual_seed(3)
    A = torch.randn(M, K, generator=g).to(BF).to(dev)
    W = (torch.randn(2 * N, K, generator=g) / K ** 0.5).to(BF).to(dev)
    W3 = (torch.randn(K, N, generator=g) / N ** 0.5).to(BF).to(dev)
    Out, H, GU = sw.swiglu_gated_mlp_train(A, W, W3)
    dA, dW, dW3, _ = sw.swiglu_gated_mlp_backward(Out, A, W, W3, H, GU, grad_dtype=torch.float32)
    W2, W32 = (W.float() - 1e-3 * dW).to(BF), (W3.float() - 1e-3 * dW3).to(BF)
    served, h = sw.swiglu_gated_mlp_mx4(A, *sw.swiglu_quantize_mx4(W2), *sw.swiglu_quantize_mx4(W32))
    W4, W34 = (sw.swiglu_dequantize_mx4(*sw.swiglu_quantize_mx4(w)) for w in (W2, W32))
    within(h, gated(A.cpu(), W4.cpu().double()), "H served")
    within(served, rounded(*product(h.cpu(), W34.cpu().double())), "Out served")


def test_binding_refuses(dev):
    g = torch.Generator().manual_seed(1)
    A = torch.randn(4, 64, generator=g).to(BF).to(dev)
    q, s = (t.to(dev) for t in codes_of(g, 32, 64))
    with pytest.raises(TypeError):
        sw.swiglu_fused_gemm_mx4(A, q.to(torch.int8), s)
    with pytest.raises(ValueError):
        sw.swiglu_fused_gemm_mx4(A, q, s[:, :1].contiguous())
    with pytest.raises(ValueError):
        sw.swiglu_fused_gemm_mx4(A, q[:, ::2], s)
    with pytest.raises(sw.SwigluError) as e:
        sw.swiglu_quantize_mx4(A[:, :40].contiguous())
    assert e.value.status == sw.SWIGLU_ERR_SHAPE
