"""The binding of the calls with low-rank adapters (needs an MI355X): what a table
holds at the time of the call counts, and the sizes that the C calls take."""
from __future__ import annotations

import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    sw.load_library()
    return torch.device("cuda:0")


def tensors(dev, L, D, N, r, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    new = lambda *shape: torch.randn(*shape, generator=g, device=dev).mul_(0.3).to(BF)  # noqa: E731
    return new(L, r, N), new(L, D, r), torch.rand(L, generator=g, device=dev) + 0.5


@pytest.mark.parametrize("how", ["assigned", "data"])
@pytest.mark.parametrize("name", ["A", "B", "scale"])
def test_a_tables_tensors_are_those_of_the_call(dev, name, how):
    print(f"\n[case] table {name} {how}", flush=True)
    M, N, D, L, r = 20, 64, 72, 3, 8
    g = torch.Generator(device=dev).manual_seed(1)
    h = torch.randn(M, N, generator=g, device=dev).to(BF)
    w = torch.randn(D, N, generator=g, device=dev).to(BF)
    ids = torch.randint(0, L, (M, 1), generator=g, device=dev, dtype=torch.int32)
    first, second = tensors(dev, L, D, N, r, 2), tensors(dev, L, D, N, r, 3)
    table = sw.SwigluLora(*first)
    before = sw.swiglu_down_proj_lora(h, w, table, ids)
    i = ("A", "B", "scale").index(name)
    mixed = list(first)
    mixed[i] = second[i]
    kept = getattr(table, name).detach()      # (the old storage stays)
    if how == "assigned":
        setattr(table, name, second[i])
    else:
        getattr(table, name).data = second[i]
    got = sw.swiglu_down_proj_lora(h, w, table, ids)
    want = sw.swiglu_down_proj_lora(h, w, sw.SwigluLora(*mixed), ids)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and not torch.equal(got, before)
    del kept


def test_a_tables_tensors_are_checked_at_the_call(dev):
    M, N, D, L, r = 4, 64, 72, 3, 8
    h, w = torch.zeros(M, N, dtype=BF, device=dev), torch.zeros(D, N, dtype=BF, device=dev)
    ids = torch.zeros(M, 1, dtype=torch.int32, device=dev)
    A, B, scale = tensors(dev, L, D, N, r, 4)
    for name, bad, error in (
            ("A", A[:2], ValueError), ("A", A.float(), TypeError), ("A", A.cpu(), ValueError),
            ("A", A.transpose(1, 2), ValueError), ("A", A[:, :, :56].contiguous(), ValueError),
            ("B", B[:, :, :4], ValueError), ("B", B[:, :64].contiguous(), ValueError),
            ("B", B[0], ValueError), ("scale", scale[:2], ValueError),
            ("scale", scale.double(), TypeError), ("scale", None, TypeError)):
        table = sw.SwigluLora(A, B, scale)
        setattr(table, name, bad)
        with pytest.raises(error):
            sw.swiglu_down_proj_lora(h, w, table, ids)
    grown = sw.SwigluLora(A, B, scale)
    grown.A, grown.B = torch.cat([A, A], 1), torch.cat([B, B], 2)
    assert (grown.rank, grown.count, grown.columns, grown.K) == (2 * r, L, D, N)
    assert not sw.swiglu_down_proj_lora(h, w, grown, ids).any()


@pytest.mark.parametrize("D", [0, (1 << 21) + 8, 1 << 22])
def test_down_projection_columns_without_a_workspace(dev, D):
    """The binding sizes its own workspace for every D that the C call takes."""
    print(f"\n[case] down projection D={D}", flush=True)
    M, N, L, r = 3, 16, 2, 8
    g = torch.Generator(device=dev).manual_seed(5)
    h = torch.randn(M, N, generator=g, device=dev).to(BF)
    w = torch.randn(D, N, generator=g, device=dev).to(BF)
    A, B, scale = tensors(dev, L, D, N, r, 6)
    ids = torch.tensor([[0], [-1], [1]], dtype=torch.int32, device=dev)
    out = sw.swiglu_down_proj_lora(h, w, sw.SwigluLora(A, B, scale), ids)
    torch.cuda.synchronize()
    assert out.shape == (M, D)
    x = h.double()
    want, size = x @ w.double().t(), x.abs() @ w.double().abs().t()
    for m, n in ((0, 0), (2, 1)):
        t = (A[n].double() @ x[m]) * scale[n].double()
        want[m] += B[n].double() @ t
        size[m] += B[n].double().abs() @ (A[n].double().abs() @ x[m].abs()) * scale[n].double()
    # sums of 16 and 8 terms in fp32 and T in 16 bits: 2^-15 of the magnitudes; one bf16 rounding
    assert ((out.double() - want).abs() <= 2.0 ** -14 * size + 2.0 ** -8 * want.abs()).all()
