"""The two products of a backward pass in one launch, at sizes whose plan is checked first
(needs an MI355X): swiglu_describe_backward() names the launches, so a size that stops
reaching the pair kernel fails here.  Bounds as in test_gpu_train.py."""
from __future__ import annotations

import re

import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw
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


def plan(M, K, N, call, dtype, add, ws):
    """For each stage of the call: how the tiles of the activation's and of the weight's
    gradient run in the pair kernel ('whole' or 'split'), or None for launches apart."""
    text = sw.swiglu_describe_backward(M, N, K, call, dtype, add, ws.numel())
    print(f"  {text}", flush=True)
    stages = []
    for stage in text.split(", then "):
        m = re.match(r"gemm_pair_kernel<\w+> \((\d+ whole tiles|\d+ tiles split \d+ ways along K) of"
                     r" the activation's gradient, (\d+ whole tiles|\d+ tiles split \d+ ways along K)"
                     r" of the weight's; \d+ workgroups\)", stage)
        stages.append(m and tuple("whole" if "whole" in t else "split" for t in m.groups()))
        if m:
            assert stage.count("split_reduce_kernel") == stages[-1].count("split")
    return stages


WHOLE, X, W, BOTH = ("whole", "whole"), ("split", "whole"), ("whole", "split"), ("split", "split")
# dOut's and GU's stage.  Contractions that end inside a K step, rows and columns inside a
# tile; the last one even in all of them.
PLANS = [(1000, 3592, 6152, [X, X]), (5003, 520, 5000, [W, X]), (7409, 2824, 752, [BOTH, W]),
         (3000, 2056, 4104, [WHOLE, X]), (6007, 3080, 712, [X, W]), (2048, 1536, 8960, [WHOLE, X])]


def check_block(dev, M, K, N, dtype, add, d, ws):
    kw = {"dW_fused_add": d["addW"].to(dtype), "dW3t_add": d["addW3"].to(dtype)} if add else {}
    args = [d[n] for n in ("dOut", "A", "W", "W3", "H", "GU")]
    dA, dW, dW3, dGU = sw.swiglu_gated_mlp_backward(*args, grad_dtype=dtype, workspace=ws, **kw)
    torch.cuda.synchronize()
    near_dgu(dGU, d, "dGU")
    near(dA, dGU, d["W"], "dA")
    near(dW, dGU.t(), d["A"], "dW_fused", kw.get("dW_fused_add"))
    near(dW3, d["dOut"].t(), d["H"], "dW3t", kw.get("dW3t_add"))


@pytest.mark.parametrize("M,K,N,stages", PLANS)
def test_block(dev, M, K, N, stages):
    ws = workspace_of(dev, M, N, K)
    d = inputs_of(dev, M, K, N, M)
    for dtype, add in ((BF, False), (BF, True), (F32, False), (F32, True)):
        assert plan(M, K, N, "gated_mlp", dtype, add, ws) == stages
        check_block(dev, M, K, N, dtype, add, d, ws)


@pytest.mark.parametrize("M,K,N,stages", [(260, 4104, 9224, [X, X]), (9001, 1544, 1032, [W, None]),
                                          (16384, 520, 1032, [W, None])])
def test_block_in_32_bits(dev, M, K, N, stages):
    """Few rows and many; a weight's tiles split seven and more ways."""
    ws = workspace_of(dev, M, N, K)
    assert plan(M, K, N, "gated_mlp", F32, False, ws) == stages
    check_block(dev, M, K, N, F32, False, inputs_of(dev, M, K, N, M), ws)


@pytest.mark.parametrize("M,K,N,stage", [(1000, 3592, 6152, X), (5003, 520, 5000, W),
                                         (7409, 2824, 752, BOTH), (3000, 2056, 4104, WHOLE),
                                         (4100, 4104, 520, X)])
def test_down_projection(dev, M, K, N, stage):
    ws = workspace_of(dev, M, N, K)
    d = inputs_of(dev, M, K, N, 7 + M)
    for dtype in (BF, F32):
        assert plan(M, K, N, "down_proj", dtype, False, ws) == [stage]
        dH, dW3 = sw.swiglu_down_proj_backward(d["dOut"], d["H"], d["W3"], grad_dtype=dtype,
                                               workspace=ws)
        near(dH, d["dOut"], d["W3"], "dH")
        near(dW3, d["dOut"].t(), d["H"], "dW3t")
    sums = d["addW3"].clone()
    assert plan(M, K, N, "down_proj", F32, True, ws) == [stage]
    sw.swiglu_down_proj_backward(d["dOut"], d["H"], d["W3"], dW3t=sums, dW3t_add=sums, workspace=ws)
    near(sums, d["dOut"].t(), d["H"], "dW3t in place", d["addW3"])


def test_swiglu_stage(dev):
    M, K, N = 7409, 2824, 752
    ws = workspace_of(dev, M, N, K)
    d = inputs_of(dev, M, K, N, 3)
    assert plan(M, K, N, "fused_gemm", F32, False, ws) == [None, W]   # (dGU first, by elements)
    dA, dW, dGU = sw.swiglu_fused_gemm_backward(d["dH"], d["A"], d["W"], d["GU"], grad_dtype=F32,
                                                workspace=ws)
    near(dA, dGU, d["W"], "dA")
    near(dW, dGU.t(), d["A"], "dW_fused")


def test_no_pair_without_its_workspace(dev):
    """Nor for few rows, nor where a tile is forced."""
    M, K, N = 5003, 520, 5000
    full = workspace_of(dev, M, N, K)
    small = full[:full.numel() // 2]
    assert plan(M, K, N, "gated_mlp", F32, False, small) == [None, None]
    assert plan(64, 3592, 6152, "gated_mlp", F32, False, full) == [None, None]
    check_block(dev, M, K, N, F32, False, inputs_of(dev, M, K, N, 9), small)


def _call(d, w, **kw):
    args = [d[n] for n in ("dOut", "A", "W", "W3", "H", "GU")]
    return sw.swiglu_gated_mlp_backward(*args, grad_dtype=F32, workspace=w, **kw)


@pytest.mark.parametrize("M,K,N", [(5003, 520, 5000), (1000, 3592, 6152), (7409, 2824, 752)])
def test_same_bits_on_streams(dev, M, K, N):
    """Two streams at once, each with its workspace: which workgroup drew a tile shows
    nowhere."""
    d = inputs_of(dev, M, K, N, 5)
    ws = [workspace_of(dev, M, N, K) for _ in range(2)]
    assert None not in plan(M, K, N, "gated_mlp", F32, False, ws[0])
    first = _call(d, ws[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    got = []
    for _ in range(4):
        for s, w in zip(streams, ws):
            with torch.cuda.stream(s):
                got.append(_call(d, w))
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(first, o))


@pytest.mark.parametrize("M,K,N", [(5003, 520, 5000), (1000, 3592, 6152)])
def test_replays(dev, M, K, N):
    """Two captured passes, each with a workspace of its own, replayed at the same time on
    two streams beside eager calls, on other inputs every time: the counts start anew at
    every replay, whatever the call before left in a workspace."""
    d = inputs_of(dev, M, K, N, 5)
    ws = [workspace_of(dev, M, N, K) for _ in range(3)]
    assert None not in plan(M, K, N, "gated_mlp", F32, False, ws[0])
    first = _call(d, ws[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    outs, graphs = [], []
    for s, w in zip(streams, ws):
        outs.append([torch.empty_like(t) for t in first])
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.stream(s):
            with torch.cuda.graph(graphs[-1], stream=s):
                _call(d, w, **dict(zip(("dA", "dW_fused", "dW3t", "dGU"), outs[-1])))
    for seed in (6, 7, 8):
        for k, v in inputs_of(dev, M, K, N, seed).items():
            d[k].copy_(v)
        for w in ws[:2]:
            w.fill_(seed)          # whatever is there
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(2):
            for s, graph in zip(streams, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
        want = _call(d, ws[2])
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, want))
        # an eager call on a replayed call's workspace
        assert all(torch.equal(a, b) for a, b in zip(_call(d, ws[0]), want))
        torch.cuda.synchronize()
