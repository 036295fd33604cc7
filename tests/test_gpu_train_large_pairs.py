"""Two products in one launch on matrices whose offsets pass 31 and 32 bits (needs an MI355X):
GU and dGU of 4.3 GB, H of 2.2.  Rows about each border, and the weights' gradients over all
rows, against 64-bit products; bounds as in test_gpu_train.py."""
from __future__ import annotations

import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw
from test_gpu_train_large import contracted, near, product

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
M, K, N = 57000, 520, 18944


def test_offsets(monkeypatch):
    monkeypatch.delenv("SWIGLU_I_TILE", raising=False)
    monkeypatch.delenv("SWIGLU_TAIL", raising=False)
    dev = torch.device("cuda:0")
    assert M * 2 * N * 2 > 1 << 32 and M * N * 2 > 1 << 31
    g = torch.Generator(device=dev).manual_seed(11)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=dev) * std).to(BF)  # noqa: E731
    A, W, W3, dOut = r(M, K), r(2 * N, K, std=K ** -0.5), r(K, N, std=N ** -0.5), r(M, K)
    GU, H = r(M, 2 * N), r(M, N)
    ws = torch.full((sw.swiglu_workspace_size(M, N, K, "ablation"),), 0xFF, dtype=torch.uint8,
                    device=dev)
    text = sw.swiglu_describe_backward(M, N, K, "gated_mlp", F32, False, ws.numel())
    assert text.count("gemm_pair_kernel") == 2, text
    dA, dW, dW3, dGU = sw.swiglu_gated_mlp_backward(dOut, A, W, W3, H, GU, grad_dtype=F32,
                                                    workspace=ws)
    torch.cuda.synchronize()
    border = (1 << 31) // (4 * N)
    rows = torch.cat([torch.arange(a, a + 300, device=dev)
                      for a in (0, border - 150, 2 * border - 150, M - 300)])
    dh, dhe = product(dOut[rows], W3)
    gate, up = GU[rows][:, 0::2].double(), GU[rows][:, 1::2].double()
    sig, big = torch.sigmoid(gate), 1 + gate.abs()
    near(dGU[rows][:, 0::2], dh * up * sig * (1 + gate * (1 - sig)),
         up.abs() * (1.1 * dhe + (dh.abs() + dhe) * big * big * 2.0 ** -20), "dG")
    near(dGU[rows][:, 1::2], dh * gate * sig,
         gate.abs() * (dhe + (dh.abs() + dhe) * big * 2.0 ** -20), "dU")
    near(dA[rows], *product(dGU[rows], W), "dA")
    near(dW, *contracted(dGU, A), "dW_fused")
    near(dW3, *contracted(dOut, H), "dW3t")
    text = sw.swiglu_describe_backward(M, N, K, "down_proj", F32, False, ws.numel())
    assert text.startswith("gemm_pair_kernel"), text
    dH, dW3b = sw.swiglu_down_proj_backward(dOut, H, W3, grad_dtype=F32, workspace=ws)
    near(dH[rows], dh, dhe, "dH")
    assert torch.equal(dW3b, dW3)     # (the same tiles of the same contraction)
