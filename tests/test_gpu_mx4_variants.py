"""Every form of the few-row kernel of the 4-bit weights, which is chosen by the activations'
rows and by how many 16-row tiles of the weight there are for a compute unit, and weights of
more than 4 GiB of codes (needs an MI355X); bounds as in test_gpu_mx4.py."""
from __future__ import annotations

import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw
from test_gpu_mx4 import codes_of, gated, product, rounded, values_of, within

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    sw.load_library()
    return torch.device("cuda:0")


# 16-row tiles of the weight: at most one for each of 256 compute units, up to four, more
ROWS = [168, 4096, 4104, 9000, 16360, 16400, 24008]


@pytest.mark.parametrize("M", [1, 3, 4, 5, 8, 9, 16, 17, 24, 32, 33, 48, 49, 64])
def test_every_form(dev, M):
    g = torch.Generator().manual_seed(M)
    # (short of a wave's blocks of 128, past them by a group, and several rounds of the rings)
    for K in (96, 544, 1184):
        x = torch.randn(M, K, generator=g).to(BF)
        q, s = codes_of(g, 2 * max(ROWS), K)
        xd, qd, sd = x.to(dev), q.to(dev), s.to(dev)
        v = values_of(q, s)
        sums, h = rounded(*product(x, v)), gated(x, v)
        for rows in ROWS:
            y = sw.swiglu_down_proj_mx4(xd, qd[:rows], sd[:rows])
            within(y, tuple(t[:, :rows] for t in sums), f"M={M} K={K} rows={rows}")
            n = rows // 8 * 4
            n -= n % 8
            y = sw.swiglu_fused_gemm_mx4(xd, qd[:2 * n], sd[:2 * n])
            within(y, tuple(t[:, :n] for t in h), f"M={M} K={K} gated {n}")


@pytest.mark.parametrize("M", [1, 2, 4])
def test_long_rows_of_a_wide_weight(dev, M):
    """Few rows beside K >= 8192 and more than four tiles a compute unit."""
    g = torch.Generator().manual_seed(70 + M)
    for K, rows in ((8192, 16400), (8224, 16656), (8160, 16400)):
        x = torch.randn(M, K, generator=g).to(BF)
        q, s = codes_of(g, rows, K)
        v = sw.swiglu_dequantize_mx4(q.to(dev), s.to(dev)).double()
        xd = x.to(dev).double()
        value, err = product(xd, v)
        y = sw.swiglu_down_proj_mx4(x.to(dev), q.to(dev), s.to(dev))
        within(y, tuple(t.cpu() for t in rounded(value, err)), f"M={M} K={K} rows={rows}")
        y = sw.swiglu_fused_gemm_mx4(x.to(dev), q.to(dev), s.to(dev))
        within(y, tuple(t.cpu() for t in gated(xd, v)), f"M={M} K={K} gated")


def test_codes_beyond_4_gib(dev):
    """A weight of 4.3 GB of codes (17 GB as bf16), quantized, read back and multiplied."""
    K, rows = 8192, (1 << 20) + 32
    assert rows * K // 2 > 1 << 32
    g = torch.Generator(device=dev).manual_seed(1)
    w = torch.empty(rows, K, dtype=BF, device=dev)
    step = 1 << 16
    for i in range(0, rows, step):
        n = min(step, rows - i)
        w[i:i + n] = torch.randn(n, K, generator=g, device=dev) / K ** 0.5
    q, s = sw.swiglu_quantize_mx4(w)
    back = sw.swiglu_dequantize_mx4(q, s)
    torch.cuda.synchronize()
    print("  quantized", flush=True)
    # the same rows laid out alone: about 2^31 and 2^32 numbers and bytes, and the last ones
    spots = torch.cat([torch.arange(a, a + 64, device=dev)
                       for a in (0, (1 << 18) - 32, (1 << 19) - 32, (1 << 20) - 32, rows - 64)])
    q1, s1 = sw.swiglu_quantize_mx4(w[spots].contiguous())
    assert torch.equal(q[spots], q1) and torch.equal(s[spots], s1)
    v = values_of(q1.cpu(), s1.cpu())
    assert torch.equal(back[spots].cpu().double(), v)
    del w, back
    for M in (1, 3, 40, 70, 200):
        x = torch.randn(M, K, generator=g, device=dev).to(BF)
        y = sw.swiglu_down_proj_mx4(x, q, s)
        within(y[:, spots], rounded(*product(x.cpu(), v)), f"M={M}")
        y = sw.swiglu_fused_gemm_mx4(x, q, s)
        pairs = spots[0::2] // 2
        within(y[:, pairs], gated(x.cpu(), v), f"M={M} gated")
    del q, s, y
    torch.cuda.empty_cache()
