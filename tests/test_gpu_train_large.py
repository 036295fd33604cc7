"""The training calls on matrices whose offsets pass 31 and 32 bits (needs an MI355X): GU and
dGU of 4.3 GB, H and dH of 2.2, and the weights' gradients contracted over all their rows.
Rows about each border against 64-bit products; bounds as in test_gpu_train.py."""
from __future__ import annotations

import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
M, K, N = 57000, 24, 18944
CHUNK = 4096


def bound(n, mags):
    return (n / 16 + 32) * 2.0 ** -24 * mags


def near(got, v, e, what):
    half = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
    tol = e * (1 + half) + v.abs() * half + 2.0 ** -126
    worst = float(((got.double() - v).abs() / tol).max())
    print(f"  {what}: worst error {worst:.3f} of its bound", flush=True)
    assert worst <= 1, what


def product(x, w):
    x, w = x.double(), w.double()
    return x @ w, bound(x.shape[1], x.abs() @ w.abs())


def contracted(dy, x):
    """dy^T x over all rows."""
    v = e = 0.0
    for i in range(0, dy.shape[0], CHUNK):
        a, b = dy[i:i + CHUNK].double().t().contiguous(), x[i:i + CHUNK].double()
        v, e = v + a @ b, e + a.abs() @ b.abs()
    return v, bound(dy.shape[0], e)


@pytest.mark.parametrize("with_workspace", [True, False])
def test_offsets(monkeypatch, with_workspace):
    monkeypatch.delenv("SWIGLU_I_TILE", raising=False)
    monkeypatch.delenv("SWIGLU_TAIL", raising=False)
    dev = torch.device("cuda:0")
    assert M * 2 * N * 2 > 1 << 32 and M * N * 2 > 1 << 31
    g = torch.Generator(device=dev).manual_seed(7)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=dev) * std).to(BF)  # noqa: E731
    A, W, W3, dOut = r(M, K), r(2 * N, K, std=K ** -0.5), r(K, N, std=N ** -0.5), r(M, K)
    ws = None
    if with_workspace:
        ws = torch.full((sw.swiglu_workspace_size(M, N, K, "ablation"),), 0xFF, dtype=torch.uint8,
                        device=dev)
    Out, H, GU = sw.swiglu_gated_mlp_train(A, W, W3, workspace=ws)
    dA, dW, dW3, dGU = sw.swiglu_gated_mlp_backward(dOut, A, W, W3, H, GU, grad_dtype=F32,
                                                    workspace=ws)
    torch.cuda.synchronize()
    border = (1 << 31) // (4 * N)
    rows = torch.cat([torch.arange(a, a + 300, device=dev)
                      for a in (0, border - 150, 2 * border - 150, M - 300)])
    gate, ge = product(A[rows], W[0::2].t())
    up, ue = product(A[rows], W[1::2].t())
    near(GU[rows][:, 0::2], gate, ge, "G")
    near(GU[rows][:, 1::2], up, ue, "U")
    s = gate * torch.sigmoid(gate)
    se = 1.1 * ge + (1 + gate.abs()) * gate.abs() * 2.0 ** -20
    near(H[rows], s * up, se * up.abs() + s.abs() * ue + se * ue, "H")
    near(Out[rows], *product(H[rows], W3.t()), "Out")
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
    dH, dW3b = sw.swiglu_down_proj_backward(dOut, H, W3, grad_dtype=F32, workspace=ws)
    near(dH[rows], dh, dhe, "dH")
    near(dW3b, *contracted(dOut, H), "dW3t alone")
