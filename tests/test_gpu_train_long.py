"""Weights' gradients over as many rows as the calls take (needs an MI355X): contractions of
2^22 to 2^24 K steps, one tile split along K into hundreds of pieces.

Operands are +1 and -1, so every product is one of them too, every partial sum is a whole
number that stays far below 2^24 in magnitude (sums of n random signs: some sqrt(n), n at most
2^30), and fp32 holds all of them exactly: results have to be equal."""
from __future__ import annotations

import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
CHUNK = 1 << 24


def signs(g, dev, rows, cols):
    """+1 and -1, drawn in chunks."""
    out = torch.empty(rows, cols, dtype=BF, device=dev)
    for i in range(0, rows, CHUNK):
        n = min(CHUNK, rows - i)
        out[i:i + n] = torch.randint(0, 2, (n, cols), generator=g, device=dev, dtype=torch.int8) * 2 - 1
    return out


@pytest.mark.parametrize("M", [(1 << 28) + 37, (1 << 29) - 100, 1 << 30])
def test_long_contractions(monkeypatch, M):
    monkeypatch.delenv("SWIGLU_I_TILE", raising=False)
    monkeypatch.delenv("SWIGLU_TAIL", raising=False)
    dev = torch.device("cuda:0")
    N, D = 8, 16
    g = torch.Generator(device=dev).manual_seed(M)
    dOut, H = signs(g, dev, M, D), signs(g, dev, M, N)
    W3t = torch.randint(-3, 4, (D, N), generator=g, device=dev).to(BF)
    ws = torch.full((sw.swiglu_workspace_size(M, N, D, "ablation"),), 0xFF, dtype=torch.uint8,
                    device=dev)
    print(f"  M={M}: {M * D * 2 / 1e9:.1f} and {M * N * 2 / 1e9:.1f} GB", flush=True)
    dH, dW = sw.swiglu_down_proj_backward(dOut, H, W3t, grad_dtype=F32, workspace=ws)
    torch.cuda.synchronize()
    print("  called", flush=True)
    want = torch.zeros(D, N, dtype=torch.float64, device=dev)
    for i in range(0, M, CHUNK):
        d, h = dOut[i:i + CHUNK].float(), H[i:i + CHUNK].float()
        want += (d.t().contiguous() @ h).double()          # (whole numbers below 2^24: exact)
        assert torch.equal(dH[i:i + CHUNK].float(), d @ W3t.float())
    assert torch.equal(dW.double(), want), float((dW.double() - want).abs().max())
    del dOut, H, dH
    torch.cuda.empty_cache()
