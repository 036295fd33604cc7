"""swiglu_route and swiglu_route_backward at the ends of their ranges, against the
definition in 64 bits (needs an MI355X).

The gradient's bound is that of its formula: p (G - sum p G) with a relative error of
2^-17 of the magnitudes of both terms (a softmax of fp32 logits under 40, 62 roundings
of 2^-24, and two products), as p and G are each off by at most 2^-18 of themselves.
"""
from __future__ import annotations

import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    sw.load_library()
    return torch.device("cuda:0")


@pytest.mark.parametrize("normalize", [True, False], ids=["normalized", "raw"])
@pytest.mark.parametrize("each", [(1 << 27) - 1, 1 << 27, 1 << 28, (1 << 30) + 12345, (1 << 31) - 1])
def test_gradient_with_picks_past_31_bits(dev, each, normalize):
    """Counts of a batch whose picks together pass 2^31 (each expert's own does not)."""
    M, E, k = 9, 16, 4
    print(f"\n[case] route gradient, {E} experts of about {each} picks, normalize={normalize}",
          flush=True)
    g = torch.Generator().manual_seed(each % 1000)
    z = torch.randn(M, E, generator=g)
    counts = torch.tensor([max(0, each - 1000003 * e * e) for e in range(E)] + [1 << 29],
                          dtype=torch.int32)
    counts[3] = 0
    d_loss = torch.tensor(float(1 << 29))
    ids, w, _, _ = sw.swiglu_route(z.to(dev), k, normalize=normalize)
    dz = sw.swiglu_route_backward(z.to(dev), ids, w, counts.to(dev), d_loss=d_loss.to(dev),
                                  normalize=normalize)
    torch.cuda.synchronize()
    p = torch.softmax(z.double(), 1)
    c = counts.double()
    G = (d_loss.double() * E * c[:E] / (c[:E].sum() * c[E])).expand(M, E)
    want = p * (G - (p * G).sum(1, keepdim=True))
    size = p * (G + (p * G).sum(1, keepdim=True))
    off = (dz.cpu().double() - want).abs()
    assert (off <= 2.0 ** -17 * size).all(), float((off / size).max())
