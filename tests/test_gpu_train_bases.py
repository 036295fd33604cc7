"""The training calls on operands that begin at any multiple of 16 bytes, gradients written
over what they are made of in one launch of two products, captured passes that take turns on
one workspace, and weights' gradients of more than 4 GiB (needs an MI355X); bounds as in
test_gpu_train.py."""
from __future__ import annotations

import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw
from test_gpu_train_large import near as near_bound
from test_gpu_train_pairs import inputs_of, near, near_dgu, workspace_of

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


def moved(t, by):
    """A copy that begins `by` bytes past a multiple of 256, NaN around it."""
    whole = torch.full((t.numel() + 1024,), float("nan"), dtype=t.dtype, device=t.device)
    first = 512 + by // t.element_size()
    view = whole[first:first + t.numel()].view(t.shape)
    view.copy_(t)
    assert view.data_ptr() % 256 == by
    return view


@pytest.mark.parametrize("M,K,N", [(1, 72, 136), (100, 264, 136), (300, 136, 520), (1000, 520, 1096),
                                   (5003, 520, 5000)])
def test_bases(dev, M, K, N):
    d = inputs_of(dev, M, K, N, M)
    ws = workspace_of(dev, M, N, K)
    names = ("dOut", "A", "W", "W3", "H", "GU")

    def all_of(d, fresh):
        out = sw.swiglu_gated_mlp_train(d["A"], d["W"], d["W3"], workspace=ws)
        kw = {n: fresh(shape, dtype) for n, shape, dtype in
              (("dA", (M, K), BF), ("dW_fused", (2 * N, K), F32), ("dW3t", (K, N), F32),
               ("dGU", (M, 2 * N), BF))}
        grads = sw.swiglu_gated_mlp_backward(*(d[n] for n in names), dW_fused_add=d["addW"],
                                             dW3t_add=d["addW3"], workspace=ws, **kw)
        return out + grads

    want = all_of(d, lambda shape, dtype: torch.empty(shape, dtype=dtype, device=dev))
    for by in (16, 48, 80, 240):
        m = {n: moved(t, by + 16 * (i % 2) if by < 240 else by) for i, (n, t) in enumerate(d.items())}
        got = all_of(m, lambda shape, dtype: moved(torch.zeros(shape, dtype=dtype, device=dev), by))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("M,K,N", [(5003, 520, 5000), (1000, 3592, 6152), (7409, 2824, 752)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_all_in_place(dev, M, K, N, dtype):
    """dGU over GU, the weights' gradients over their sums, in the pair kernel."""
    d = inputs_of(dev, M, K, N, 21)
    ws = workspace_of(dev, M, N, K)
    text = sw.swiglu_describe_backward(M, N, K, "gated_mlp", dtype, True, ws.numel())
    assert text.count("gemm_pair_kernel") == 2, text
    gu = d["GU"].clone()
    sums = d["addW"].to(dtype), d["addW3"].to(dtype)
    dW, dW3 = (t.clone() for t in sums)
    dA, *_ = sw.swiglu_gated_mlp_backward(d["dOut"], d["A"], d["W"], d["W3"], d["H"], gu, dGU=gu,
                                          dW_fused=dW, dW_fused_add=dW, dW3t=dW3, dW3t_add=dW3,
                                          workspace=ws)
    near_dgu(gu, d, "dGU")
    near(dA, gu, d["W"], "dA")
    near(dW, gu.t(), d["A"], "dW_fused", sums[0])
    near(dW3, d["dOut"].t(), d["H"], "dW3t", sums[1])


def test_passes_that_share_a_workspace(dev):
    """Two captured passes of different sizes and an eager one, one after the other on one
    workspace, whose counts lie at the same words for all of them."""
    shapes = [(5003, 520, 5000), (1000, 3592, 6152)]
    ws = workspace_of(dev, 5003, 5000, 520)
    assert ws.numel() == workspace_of(dev, 1000, 6152, 3592).numel()
    stream = torch.cuda.Stream(dev)
    runs = []
    for i, (M, K, N) in enumerate(shapes):
        d = inputs_of(dev, M, K, N, 31 + i)
        args = [d[n] for n in ("dOut", "A", "W", "W3", "H", "GU")]
        want = sw.swiglu_gated_mlp_backward(*args, grad_dtype=F32,
                                            workspace=workspace_of(dev, M, N, K))
        outs = [torch.empty_like(t) for t in want]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            with torch.cuda.graph(graph, stream=stream):
                sw.swiglu_gated_mlp_backward(*args, workspace=ws, **dict(
                    zip(("dA", "dW_fused", "dW3t", "dGU"), outs)))
        runs.append((graph, outs, want, args))
    for order in ((0, 1, 0), (1, 1, 0), (0, 0, 1)):
        for _, outs, _, _ in runs:
            for t in outs:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for i in order:
                runs[i][0].replay()
            eager = sw.swiglu_gated_mlp_backward(*runs[order[0]][3], grad_dtype=F32, workspace=ws)
            runs[order[1]][0].replay()
        torch.cuda.synchronize()
        for i in set(order):
            assert all(torch.equal(a, b) for a, b in zip(runs[i][1], runs[i][2]))
        assert all(torch.equal(a, b) for a, b in zip(eager, runs[order[0]][2]))


@pytest.mark.parametrize("M", [40, 700])
def test_gradients_beyond_4_gib(dev, M):
    """dW_fused of 4.3 GB and dW3t of 2.2, in 32 bits and added to sums in place."""
    K, N = 28680, 18944
    assert 2 * N * K * 4 > 1 << 32
    d = {}
    g = torch.Generator(device=dev).manual_seed(M)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=dev) * std).to(BF)  # noqa: E731
    d = {"A": r(M, K), "W": r(2 * N, K, std=K ** -0.5), "W3": r(K, N, std=N ** -0.5), "dOut": r(M, K),
         "GU": r(M, 2 * N), "H": r(M, N)}
    dW = torch.full((2 * N, K), 0.5, dtype=F32, device=dev)
    dW3 = torch.full((K, N), -0.25, dtype=F32, device=dev)
    ws = workspace_of(dev, M, N, K)
    dA, _, _, dGU = sw.swiglu_gated_mlp_backward(d["dOut"], d["A"], d["W"], d["W3"], d["H"], d["GU"],
                                                 dW_fused=dW, dW_fused_add=dW, dW3t=dW3,
                                                 dW3t_add=dW3, workspace=ws)
    torch.cuda.synchronize()
    near_dgu(dGU, d, "dGU")
    near(dA, dGU, d["W"], "dA")
    half = (M / 16 + 32) * 2.0 ** -24
    for got, dy, x, was in ((dW, dGU, d["A"], 0.5), (dW3, d["dOut"], d["H"], -0.25)):
        for i in range(0, got.shape[0], 8192):
            a, b = dy[:, i:i + 8192].double().t().contiguous(), x.double()
            v, e = a @ b, half * (a.abs() @ b.abs())
            e += (v.abs() + e + abs(was)) * 2.0 ** -24
            near_bound(got[i:i + 8192], v + was, e, f"rows {i} on")
    del dW, dW3
    torch.cuda.empty_cache()
