"""4-bit weights whose scales begin at any multiple of 4 bytes (needs an MI355X), with bytes
around them that would make a neighbour read as a scale NaN: the same bits as with scales at
the start of an allocation."""
from __future__ import annotations

import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw
from test_gpu_mx4 import codes_of, workspace_of

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    sw.load_library()
    return torch.device("cuda:0")


def shifted(s, by):
    whole = torch.full((s.numel() + 4096,), 255, dtype=torch.uint8, device=s.device)
    view = whole[1024 + by:1024 + by + s.numel()].view(s.shape)
    view.copy_(s)
    assert view.data_ptr() % 16 == by
    return view


# one group a row, an odd number of them, one more than a whole number of 16 bytes of them
@pytest.mark.parametrize("K", [32, 96, 544, 1056])
@pytest.mark.parametrize("M", [1, 7, 24, 33, 64, 100, 130, 300])
def test_scales_at_multiples_of_four(dev, M, K):
    g = torch.Generator().manual_seed(M * K)
    # (columns that end inside a tile of 16 rows of the weight, and N = 544 of the contraction)
    N = 544 if K == 96 else 32 * 13
    A = torch.randn(M, K, generator=g).to(BF).to(dev)
    (wq, ws), (vq, vs) = codes_of(g, 2 * N, K), codes_of(g, K, N)
    wq, ws, vq, vs = (t.to(dev) for t in (wq, ws, vq, vs))
    dq, ds = (t.to(dev) for t in codes_of(g, 40, K))
    fq, fs = (t.to(dev) for t in codes_of(g, 48, K))
    space = workspace_of(dev, M, N, K)
    want = sw.swiglu_gated_mlp_mx4(A, wq, ws, vq, vs, workspace=space)
    down = sw.swiglu_down_proj_mx4(A, dq, ds)
    fused = sw.swiglu_fused_gemm_mx4(A, fq, fs)
    assert not any(bool(t.isnan().any()) for t in (*want, down, fused))
    for by in (4, 8, 12):
        got = sw.swiglu_gated_mlp_mx4(A, wq, shifted(ws, by), vq, shifted(vs, 16 - by), workspace=space)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(sw.swiglu_down_proj_mx4(A, dq, shifted(ds, by)), down)
        assert torch.equal(sw.swiglu_fused_gemm_mx4(A, fq, shifted(fs, by)), fused)
