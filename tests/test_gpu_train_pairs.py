"""The two products of a backward pass in one launch (needs an MI355X): sizes at which a
compute unit's share of both is long enough for it, with tiles whole and split, ragged in
every direction, against 64-bit products (bounds as in test_gpu_train.py)."""
from __future__ import annotations

import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _default_dispatch(monkeypatch):
    monkeypatch.delenv("SWIGLU_I_TILE", raising=False)
    monkeypatch.delenv("SWIGLU_TAIL", raising=False)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    sw.load_library()
    return torch.device("cuda:0")


def inputs_of(dev, M, K, N, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=dev) * std).to(BF)  # noqa: E731
    return {"A": r(M, K), "W": r(2 * N, K, std=K ** -0.5), "W3": r(K, N, std=N ** -0.5),
            "dOut": r(M, K), "GU": r(M, 2 * N, std=2.0), "H": r(M, N), "dH": r(M, N),
            "addW": torch.randn(2 * N, K, generator=g, device=dev),
            "addW3": torch.randn(K, N, generator=g, device=dev)}


def near(got, x, w, what, add=None):
    """got = x w (+ add), rounded to its type, within the bound."""
    x, w = x.double(), w.double()
    v = x @ w
    tol = (x.shape[1] / 16 + 32) * 2.0 ** -24 * (x.abs() @ w.abs())
    if add is not None:
        tol += (v.abs() + tol + add.double().abs()) * 2.0 ** -24
        v = v + add.double()
    half = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
    tol = tol * (1 + half) + v.abs() * half + 2.0 ** -126
    worst = float(((got.double() - v).abs() / tol).max())
    print(f"  {what}: worst error {worst:.3f} of its bound", flush=True)
    assert worst <= 1, what


def near_dgu(got, d, what):
    dh = d["dOut"].double() @ d["W3"].double()
    dhe = (d["W3"].shape[0] / 16 + 32) * 2.0 ** -24 * (d["dOut"].double().abs() @ d["W3"].double().abs())
    g, u = d["GU"][:, 0::2].double(), d["GU"][:, 1::2].double()
    s = torch.sigmoid(g)
    big = 1 + g.abs()
    v = torch.stack((dh * u * s * (1 + g * (1 - s)), dh * g * s), 2).flatten(1)
    e = torch.stack((u.abs() * (1.1 * dhe + (dh.abs() + dhe) * big * big * 2.0 ** -20),
                     g.abs() * (dhe + (dh.abs() + dhe) * big * 2.0 ** -20)), 2).flatten(1)
    tol = e * (1 + 2.0 ** -8) + v.abs() * 2.0 ** -8 + 2.0 ** -126
    worst = float(((got.double() - v).abs() / tol).max())
    print(f"  {what}: worst error {worst:.3f} of its bound", flush=True)
    assert worst <= 1, what


def workspace_of(dev, M, N, K):
    return torch.full((sw.swiglu_workspace_size(M, N, K, "ablation"),), 0xFF, dtype=torch.uint8,
                      device=dev)


# (the weight's products longer, shorter and as long as the activation's; contractions
# that end inside a K step; one long and narrow, whose tiles are all split)
SHAPES = [(2100, 1544, 4104), (1000, 3592, 6152), (4099, 1032, 4872), (260, 4104, 9224),
          (5003, 520, 5000), (2048, 2048, 2048), (3100, 1288, 1800)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_block(dev, M, K, N):
    d = inputs_of(dev, M, K, N, M)
    ws = workspace_of(dev, M, N, K)
    args = [d[n] for n in ("dOut", "A", "W", "W3", "H", "GU")]
    for dtype, add in ((BF, False), (F32, True)):
        kw = {"dW_fused_add": d["addW"], "dW3t_add": d["addW3"]} if add else {}
        dA, dW, dW3, dGU = sw.swiglu_gated_mlp_backward(*args, grad_dtype=dtype, workspace=ws, **kw)
        torch.cuda.synchronize()
        near_dgu(dGU, d, "dGU")
        near(dA, dGU, d["W"], "dA")
        near(dW, dGU.t(), d["A"], "dW_fused", kw.get("dW_fused_add"))
        near(dW3, d["dOut"].t(), d["H"], "dW3t", kw.get("dW3t_add"))


@pytest.mark.parametrize("M,K,N", SHAPES[:4])
def test_down_projection(dev, M, K, N):
    d = inputs_of(dev, M, K, N, 7 + M)
    ws = workspace_of(dev, M, N, K)
    for dtype in (BF, F32):
        dH, dW3 = sw.swiglu_down_proj_backward(d["dOut"], d["H"], d["W3"], grad_dtype=dtype, workspace=ws)
        near(dH, d["dOut"], d["W3"], "dH")
        near(dW3, d["dOut"].t(), d["H"], "dW3t")
    sums = d["addW3"].clone()
    sw.swiglu_down_proj_backward(d["dOut"], d["H"], d["W3"], dW3t=sums, dW3t_add=sums, workspace=ws)
    near(sums, d["dOut"].t(), d["H"], "dW3t in place", d["addW3"])


def test_same_bits_on_streams_and_replays(dev):
    """Two streams at once, each with its workspace; a captured pass replayed on other
    inputs beside eager ones: which workgroup ran a tile shows nowhere."""
    M, K, N = 2100, 1544, 4104
    d = inputs_of(dev, M, K, N, 5)
    ws = [workspace_of(dev, M, N, K) for _ in range(3)]
    args = [d[n] for n in ("dOut", "A", "W", "W3", "H", "GU")]
    first = sw.swiglu_gated_mlp_backward(*args, grad_dtype=F32, workspace=ws[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    got = []
    for _ in range(3):
        for s, w in zip(streams, ws):
            with torch.cuda.stream(s):
                got.append(sw.swiglu_gated_mlp_backward(*args, grad_dtype=F32, workspace=w))
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(first, o))
    outs = [torch.empty_like(t) for t in first]
    kw = dict(zip(("dA", "dW_fused", "dW3t", "dGU"), outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(streams[0]):
        with torch.cuda.graph(graph, stream=streams[0]):
            sw.swiglu_gated_mlp_backward(*args, workspace=ws[0], **kw)
    for seed in (6, 7, 8, 9):
        for k, v in inputs_of(dev, M, K, N, seed).items():
            d[k].copy_(v)
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = sw.swiglu_gated_mlp_backward(*args, grad_dtype=F32, workspace=ws[2])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
