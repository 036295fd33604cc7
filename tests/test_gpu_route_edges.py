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
BF = torch.bfloat16
INF = float("inf")


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


def nan_rows(E, dtype, sign):
    """A NaN of the sign alone, beside -inf, and beside numbers, at several places."""
    word = {torch.float32: (torch.int32, 0x7FC00001, -0x400000),
            BF: (torch.int16, 0x7FC0, -0x40)}[dtype]
    nan = torch.tensor([word[1] if sign > 0 else word[2]], dtype=word[0]).view(dtype)
    assert torch.isnan(nan).all()
    rows = []
    for at in sorted({0, E // 2, E - 1}):
        for rest in (-INF, 0.5, 3.0e38):
            row = torch.full((E,), rest).to(dtype)
            row[at] = nan
            rows.append(row)
    rows.append(nan.expand(E).clone())
    return torch.stack(rows)


@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("sign", [1, -1], ids=["positive", "negative"])
def test_a_nan_of_either_sign_makes_its_rows_picks_nan(dev, sign, dtype):
    for E, k in ((1, 1), (5, 1), (5, 3), (64, 4), (300, 16)):
        z = nan_rows(E, dtype, sign)
        M = z.shape[0]
        z = torch.cat([z, torch.linspace(-1, 1, E).to(dtype)[None]])   # and a row without
        for normalize in (True, False):
            print(f"\n[case] route NaN {dtype} sign={sign} E={E} k={k} normalize={normalize}",
                  flush=True)
            ids, w, counts, loss = sw.swiglu_route(z.to(dev), k, normalize=normalize)
            torch.cuda.synchronize()
            ids, w = ids.cpu(), w.cpu()
            assert int(ids.min()) >= -1 and int(ids.max()) < E
            assert (ids[:M, 0] >= 0).all()
            assert torch.isnan(w[:M][ids[:M] >= 0]).all(), w[:M]
            assert (w[ids < 0] == 0).all()
            assert not torch.isnan(w[M]).any()
            assert torch.isnan(loss)
            assert int(counts[E]) == M + 1


@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("E,k", [(1, 1), (6, 3), (64, 8), (200, 16)])
def test_an_infinite_logit_makes_its_rows_weights_nan(dev, E, k, dtype):
    """softmax takes inf - inf: NaN, for every pick; the picks are what they are."""
    z = torch.linspace(-2, 2, E).flip(0).repeat(4, 1)
    z[0, E // 2] = INF
    z[1, 0] = z[1, E - 1] = INF
    z[2] = -INF
    z[2, E - 1] = INF
    z = z.to(dtype)
    for normalize in (True, False):
        print(f"\n[case] route inf {dtype} E={E} k={k} normalize={normalize}", flush=True)
        ids, w, counts, loss = sw.swiglu_route(z.to(dev), k, normalize=normalize)
        torch.cuda.synchronize()
        order = torch.sort(z.float(), dim=1, descending=True, stable=True)
        want = torch.where(order.values[:, :k] > -INF, order.indices[:, :k], -1)
        assert torch.equal(ids.cpu().long(), want)
        w = w.cpu()
        assert torch.isnan(w[:3][want[:3] >= 0]).all(), w[:3]
        assert (w[want < 0] == 0).all()
        assert not torch.isnan(w[3]).any()
        assert torch.isnan(loss)
