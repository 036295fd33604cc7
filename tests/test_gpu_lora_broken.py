"""Calls with an adapter that holds infinities or NaN (needs an MI355X).

Every row of a tile is multiplied with every adapter of its plan, those that it does not
name with zeros.  A tile that meets an infinity or NaN is done again, with zeros in their
place and what they are added to the rows that name their adapter.  So

 - the rows that do not name it get, bit for bit, what they get beside an adapter with
   zeros in those places;
 - the rows that name it get what the formula gives: classes (finite, either infinity,
   NaN) are compared, finite values within the bounds of the sums;
 - the call takes a few times as long, not a thousand times.
"""
from __future__ import annotations

import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    sw.load_library()
    return torch.device("cuda:0")


def make(dev, kind, M, K, N, L, r, J, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    parts = 2 if kind == "gated" else 1
    new = lambda std, *shape: torch.randn(*shape, generator=g, device=dev).mul_(std).to(BF)  # noqa: E731
    x, w = new(1.0, M, K), new(K ** -0.5, parts * N, K)
    A, B = new(K ** -0.5, L, parts * r, K), new(0.7 * r ** -0.5, L, parts * N, r)
    scale = torch.rand(L, generator=g, device=dev) + 0.5
    ids = torch.randint(0, L, (M, J), generator=g, device=dev, dtype=torch.int32)
    ids[ids == 1] = 0
    ids[3::7, J - 1] = 1                # some rows name the broken adapter
    weights = torch.rand(M, J, generator=g, device=dev) + 0.25
    return x, w, A, B, scale, ids, weights


def call(kind, x, w, A, B, scale, ids, weights):
    run = sw.swiglu_fused_gemm_lora if kind == "gated" else sw.swiglu_down_proj_lora
    return run(x, w, sw.SwigluLora(A, B, scale), ids, weights)


SCHEDULES = [(5, 200, 264, 8, 2, None, None), (30, 1096, 264, 40, 1, None, None),
             (60, 520, 32776, 16, 1, None, None), (100, 520, 1400, 24, 3, "256", "fixup"),
             (128, 3584, 4864, 16, 2, None, None), (128, 520, 1400, 16, 2, "128", "split"),
             (300, 328, 1400, 16, 2, "256", "split"), (300, 328, 1400, 128, 8, "256", "quarter"),
             (520, 136, 1400, 64, 1, "256", "whole"), (520, 136, 1400, 8, 4, "128", "whole"),
             (700, 520, 520, 256, 2, "128", "split"), (2600, 264, 5000, 16, 1, "256", "quarter")]


@pytest.mark.parametrize("kind", ["gated", "down"])
@pytest.mark.parametrize("M,K,N,r,J,tile,tail", SCHEDULES)
def test_other_rows_as_beside_zeros(dev, kind, M, K, N, r, J, tile, tail, monkeypatch):
    print(f"\n[case] broken adapter {kind} M={M} K={K} N={N} r={r} J={J} {tile} {tail}", flush=True)
    if tile:
        monkeypatch.setenv("SWIGLU_I_TILE", tile)
        monkeypatch.setenv("SWIGLU_TAIL", tail)
    x, w, A, B, scale, ids, weights = make(dev, kind, M, K, N, 5, r, J, M + r)
    g = torch.Generator(device=dev).manual_seed(7)
    for share in (0.002, 1.0):
        at = torch.rand(B[1].shape, generator=g, device=dev) < share
        at[0, 0] = True
        what = torch.tensor([NAN, INF, -INF], device=dev).to(BF)[
            torch.randint(0, 3, B[1].shape, generator=g, device=dev)]
        bad, zero = B.clone(), B.clone()
        bad[1] = torch.where(at, what, B[1])
        zero[1] = torch.where(at, torch.zeros_like(what), B[1])
        got = call(kind, x, w, A, bad, scale, ids, weights)
        want = call(kind, x, w, A, zero, scale, ids, weights)
        torch.cuda.synchronize()
        others = ~(ids == 1).any(1)
        assert others.any() and not others.all()
        assert torch.equal(got[others].view(torch.int16), want[others].view(torch.int16)), share
        # and in the columns without, the rows that name it
        parts = 2 if kind == "gated" else 1
        whole = ~at.any(1).view(N, parts).any(1)
        assert torch.equal(got[:, whole].view(torch.int16), want[:, whole].view(torch.int16)), share


@pytest.mark.parametrize("M,K,N,r,J,tile,tail", SCHEDULES)
def test_the_rows_that_name_it_get_what_the_formula_gives(dev, M, K, N, r, J, tile, tail, monkeypatch):
    """The down projection: infinities and NaN in B, and infinite weights (T infinite)
    beside finite and infinite B."""
    print(f"\n[case] broken values M={M} K={K} N={N} r={r} J={J} {tile} {tail}", flush=True)
    if tile:
        monkeypatch.setenv("SWIGLU_I_TILE", tile)
        monkeypatch.setenv("SWIGLU_TAIL", tail)
    x, w, A, B, scale, ids, weights = make(dev, "down", M, K, N, 5, r, J, M + r + 1)
    g = torch.Generator(device=dev).manual_seed(8)
    rows, elements = torch.arange(0, N, 3, device=dev), torch.randint(0, r, (N,), generator=g, device=dev)
    B[1, rows, elements[rows]] = torch.tensor([INF, -INF, NAN], device=dev).to(BF)[rows % 3 * 0 + rows // 3 % 3]
    weights[4::9, 0] = INF
    weights[3, J - 1] = -INF                         # T infinite and B infinite
    got = call("down", x, w, A, B, scale, ids, weights).cpu()
    x, w, A, B, scale, ids, weights = (t.cpu() for t in (x, w, A, B, scale, ids, weights))
    D = x.double() @ w.double().t()
    size = x.double().abs() @ w.double().abs().t()
    for n in range(A.shape[0]):
        share = torch.where(ids == n, weights.double(), 0.0).sum(1) * scale[n].double()
        take = (ids == n).any(1).nonzero()[:, 0]
        T = (x[take].double() @ A[n].double().t()) * share[take, None]
        T_size = (x[take].double().abs() @ A[n].double().abs().t()) * share[take, None].abs()
        b = B[n].double()
        # (products one by one: a matrix product's blocks may add zeros times infinities)
        D[take] += sum(T[:, i, None] * b[None, :, i] for i in range(r))
        size[take] += sum(T_size[:, i, None] * b[None, :, i].abs() for i in range(r))
    for kind in (torch.isnan, lambda t: t == INF, lambda t: t == -INF):
        assert torch.equal(kind(got.double()), kind(D))
    finite = torch.isfinite(D)
    # sums in fp32 (K / 16 + 32 roundings of 2^-24, J r one after the other), T in 16 bits
    tol = (K / 16 + 64 + J * r) * 2.0 ** -24 + 2.0 ** -15
    off = (got.double() - D).abs()[finite]
    assert (off <= (tol * size.abs() + 2.0 ** -8 * D.abs())[finite] + 2.0 ** -126).all()


@pytest.mark.parametrize("kind", ["gated", "down"])
@pytest.mark.parametrize("M", [64, 2048])
def test_a_broken_adapter_does_not_stall_the_call(dev, kind, M):
    """One request's adapter all NaN in 4096 columns of K = 4096, against the same call
    without: some times as long, where recomputing its columns' results one by one from K
    products took about a thousand times."""
    print(f"\n[case] broken adapter's time {kind} M={M}", flush=True)
    K = N = 4096
    x, w, A, B, scale, ids, weights = make(dev, kind, M, K, N, 8, 64, 1, 3)
    bad = B.clone()
    bad[1] = NAN
    times = []
    for table in (B, bad):
        for _ in range(2):
            call(kind, x, w, A, table, scale, ids, weights)
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(3):
            call(kind, x, w, A, table, scale, ids, weights)
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end) / 3)
    print(f"  {times[0] * 1000:.0f} us, broken {times[1] * 1000:.0f} us", flush=True)
    assert times[1] < 40 * times[0]
