"""The projections with low-rank adapters against the definition in 64 bits
(needs an MI355X).

Bounds.  Operands are bf16, so products are exact in fp32 and the definition is
computed from the same values.  With |X||W| the product of the magnitudes:
 - sums: fp32 over K terms, in at least 32-term MFMA blocks of several partial
   sums: K / 16 + 32 roundings of half a step (2^-24) of a partial sum, which
   is at most |X||W| (the same for the shrink and for the expansion);
 - T = weight scale X A^T is held as two bf16 numbers (what the first rounding
   leaves is at most 2^-8 of T, and is rounded by 2^-8 of itself: 2^-16; its own
   sums and two products in fp32): 2^-16 of |T| |B|, summed over the adapters;
 - Y: silu' <= 1.1, the hardware exp2 and reciprocal 2^-21 relative, and the
   product of two uncertain numbers; one rounding to bf16 (2^-8 relative).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _default_dispatch(monkeypatch):
    monkeypatch.delenv("SWIGLU_I_TILE", raising=False)
    monkeypatch.delenv("SWIGLU_TAIL", raising=False)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    sw.load_library()
    return torch.device("cuda:0")


def table_of(g, L, parts, columns, K, r):
    return {"A": (torch.randn(L, parts * r, K, generator=g) / K ** 0.5).to(BF),
            "B": (torch.randn(L, columns, r, generator=g) * (0.7 / r ** 0.5)).to(BF),
            "scale": torch.rand(L, generator=g) * 3.0 - 1.0}


def on(dev, t):
    return sw.SwigluLora(*(t[n].to(dev) for n in ("A", "B", "scale")))


def ids_of(g, M, L, J, pattern):
    ids = torch.randint(0, L, (M, J), generator=g, dtype=torch.int32)
    if pattern == "mixed":
        ids[torch.rand(M, J, generator=g) < 0.2] = -1
    elif pattern == "none":
        ids[:] = -1
    elif pattern == "outside":
        far = torch.tensor([L, L + 1, -7, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
        pick = torch.rand(M, J, generator=g) < 0.5
        ids[pick] = far[torch.randint(0, 5, (M, J), generator=g)][pick]
    elif pattern == "runs":
        ids = (torch.arange(M, dtype=torch.int32)[:, None] // max(1, M // 3) + torch.arange(
            J, dtype=torch.int32)[None, :]) % L
    elif pattern == "twice":
        ids[:, -1] = ids[:, 0]
    elif pattern == "one":
        ids[:] = -1
        ids[M // 2, J - 1] = L - 1
    return ids.contiguous()


def projected(x, w, t, part, parts, ids, weights):
    """(D, a bound of its error) of columns part::parts, in 64 bits."""
    xd, wd = x.double(), w[part::parts].double()
    K, r = x.shape[1], t["B"].shape[2]
    D = xd @ wd.t()
    roundings = lambda n: (n / 16 + 32) * 2.0 ** -24  # noqa: E731
    err = roundings(K) * (xd.abs() @ wd.abs().t())
    for n in range(t["A"].shape[0]):
        take = ids == n
        rows = take.any(1).nonzero()[:, 0]
        if rows.numel() == 0:
            continue
        share = torch.where(take, torch.ones_like(ids, dtype=torch.float64) if weights is None
                            else weights.double(), 0.0).sum(1)[rows] * t["scale"][n].double()
        # (weights of an adapter named twice are added in fp32)
        share_abs = torch.where(take, torch.ones_like(ids, dtype=torch.float64) if weights is None
                                else weights.double().abs(), 0.0).sum(1)[rows] * t["scale"][n].abs().double()
        a = t["A"][n, part * r:(part + 1) * r].double()
        b = t["B"][n, part::parts].double()
        T = (xd[rows] @ a.t()) * share[:, None]
        T_err = (T.abs() * 2.0 ** -16 + share_abs[:, None] * (xd[rows].abs() @ a.abs().t()) *
                 (roundings(K) + 2.0 ** -20) * (1 + 2.0 ** -7))
        D[rows] += T @ b.t()
        J = ids.shape[1]
        err[rows] += T_err @ b.abs().t() + roundings(K + J * r) * (T.abs() @ b.abs().t())
    return D, err + 2.0 ** -126


def gated(x, w, t, ids, weights):
    g, ge = projected(x, w, t, 0, 2, ids, weights)
    u, ue = projected(x, w, t, 1, 2, ids, weights)
    s = g * torch.sigmoid(g)
    y = s * u
    se = 1.1 * ge + s.abs() * 2.0 ** -20
    err = se * u.abs() + s.abs() * ue + se * ue
    return y, err * (1 + 2.0 ** -8) + y.abs() * 2.0 ** -8 + 2.0 ** -126


def rounded(D, err):
    return D, err * (1 + 2.0 ** -8) + D.abs() * 2.0 ** -8


def within(got, want, tol, what):
    off = (got.double().cpu() - want).abs()
    worst = float((off / tol).max()) if off.numel() else 0.0
    print(f"  {what}: worst error {worst:.3f} of its bound", flush=True)
    assert (off <= tol).all(), f"{what}: {worst}"


def case_of(kind, M, K, N, L, r, J, pattern, weighted, seed):
    g = torch.Generator().manual_seed(seed)
    parts = 2 if kind == "gated" else 1
    x = torch.randn(M, K, generator=g).to(BF)
    w = (torch.randn(parts * N, K, generator=g) / K ** 0.5).to(BF)
    t = table_of(g, L, parts, parts * N, K, r)
    ids = ids_of(g, M, L, J, pattern)
    weights = torch.rand(M, J, generator=g) if weighted else None
    return x, w, t, ids, weights


def run(kind, dev, x, w, t, ids, weights, out=None, workspace=None, lora=None):
    lora = on(dev, t) if lora is None else lora
    wt = None if weights is None else weights.to(dev)
    call = sw.swiglu_fused_gemm_lora if kind == "gated" else sw.swiglu_down_proj_lora
    y = call(x.to(dev), w.to(dev), lora, ids.to(dev), wt, out, workspace)
    torch.cuda.synchronize()
    return y


def check(dev, kind, M, K, N, L, r, J, pattern, weighted, seed):
    print(f"\n[case] lora {kind} M={M} K={K} N={N} L={L} r={r} J={J} {pattern} "
          f"weighted={weighted} seed={seed}", flush=True)
    x, w, t, ids, weights = case_of(kind, M, K, N, L, r, J, pattern, weighted, seed)
    y = run(kind, dev, x, w, t, ids, weights)
    want, tol = (gated(x, w, t, ids, weights) if kind == "gated"
                 else rounded(*projected(x, w, t, 0, 1, ids, weights)))
    within(y, want, tol, kind)
    return x, w, t, ids, weights, y


# few rows: the kernels that stream the weight
@pytest.mark.parametrize("kind", ["gated", "down"])
@pytest.mark.parametrize("M,K,N,L,r,J,pattern,weighted", [
    (1, 8, 8, 1, 8, 1, "mixed", False), (1, 896, 264, 8, 16, 1, "mixed", False),
    (1, 1000, 4864, 3, 64, 2, "twice", True), (2, 72, 24, 2, 24, 1, "outside", False),
    (7, 200, 1000, 40, 8, 3, "mixed", True), (16, 520, 136, 5, 40, 2, "mixed", False),
    (17, 256, 40, 70, 16, 8, "mixed", True), (33, 1536, 512, 16, 8, 1, "mixed", False),
    (33, 136, 24, 4, 256, 4, "outside", True), (64, 896, 1528, 200, 16, 2, "mixed", True),
    (65, 64, 72, 8, 16, 1, "runs", False), (100, 320, 264, 9, 128, 1, "mixed", False),
    (128, 512, 1000, 8, 16, 2, "twice", True), (128, 88, 8, 1, 8, 8, "mixed", True),
    (50, 512, 64, 4, 32, 1, "none", False), (128, 64, 264, 300, 8, 5, "one", False)])
def test_few_rows(dev, kind, M, K, N, L, r, J, pattern, weighted):
    check(dev, kind, M, K, N, L, r, J, pattern, weighted, seed=M + K + N + r)


# more: the tile kernels
@pytest.mark.parametrize("kind", ["gated", "down"])
@pytest.mark.parametrize("M,K,N,L,r,J,pattern,weighted", [
    (129, 64, 64, 3, 8, 1, "mixed", False), (300, 200, 392, 8, 16, 2, "mixed", True),
    (513, 512, 1000, 70, 24, 1, "mixed", False), (257, 1000, 136, 12, 64, 3, "twice", True),
    (700, 256, 264, 5, 256, 1, "runs", False), (260, 72, 8, 2, 40, 8, "outside", True),
    (1024, 320, 2056, 8, 16, 2, "mixed", True), (131, 96, 520, 4, 8, 1, "none", False),
    (400, 64, 24, 600, 16, 4, "mixed", True), (2048, 136, 512, 16, 64, 1, "runs", False)])
def test_tiles(dev, kind, M, K, N, L, r, J, pattern, weighted):
    check(dev, kind, M, K, N, L, r, J, pattern, weighted, seed=M + K + N + r)


@pytest.mark.parametrize("kind", ["gated", "down"])
@pytest.mark.parametrize("tile,tail", [("256", "split"), ("256", "quarter"), ("256", "whole"),
                                       ("128", "split"), ("128", "whole")])
def test_every_schedule(dev, kind, tile, tail, monkeypatch):
    monkeypatch.setenv("SWIGLU_I_TILE", tile)
    monkeypatch.setenv("SWIGLU_TAIL", tail)
    check(dev, kind, 520, 520, 1400, 6, 16, 2, "mixed", True, seed=1)
    check(dev, kind, 300, 1024, 4600, 6, 40, 1, "runs", False, seed=2)


@pytest.mark.parametrize("M", [1, 40, 100, 300])
def test_block_with_the_router(dev, M):
    """swiglu_route's picks and weights straight into swiglu_gated_mlp_lora."""
    K, N, L, r, J = 192, 328, 8, 16, 2
    print(f"\n[case] lora block M={M}", flush=True)
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=g).to(BF)
    w = (torch.randn(2 * N, K, generator=g) / K ** 0.5).to(BF)
    w3 = (torch.randn(K, N, generator=g) / N ** 0.5).to(BF)
    up, down = table_of(g, L, 2, 2 * N, K, r), table_of(g, L, 1, K, N, 2 * r)
    z = torch.randn(M, L, generator=g)
    z[M // 2] = float("-inf")                     # a row that takes no adapter
    ids, weights, _, _ = sw.swiglu_route(z.to(dev), J)
    out, h = sw.swiglu_gated_mlp_lora(x.to(dev), w.to(dev), w3.to(dev), on(dev, up), on(dev, down),
                                      ids, weights)
    torch.cuda.synchronize()
    want, tol = gated(x, w, up, ids.cpu(), weights.cpu())
    within(h, want, tol, "H")
    want, tol = rounded(*projected(h.cpu(), w3, down, 0, 1, ids.cpu(), weights.cpu()))
    within(out, want, tol, "Out")


def test_without_adapters_it_is_the_plain_call(dev):
    """Rows that name none get what the call without adapters gives them, up to
    one rounding of the fp32 sums' different order."""
    for M in (64, 300):
        print(f"\n[case] lora none M={M}", flush=True)
        x, w, t, ids, _ = case_of("gated", M, 512, 264, 4, 16, 1, "none", False, 5)
        y = run("gated", dev, x, w, t, ids, None)
        plain = sw.swiglu_fused_gemm(x.to(dev), w.to(dev), variant="i")
        want, tol = gated(x, w, t, ids, None)
        within(y, want, tol, "with the table")
        within(plain, want, tol, "plain")


@pytest.mark.parametrize("kind", ["gated", "down"])
@pytest.mark.parametrize("M", [30, 300])
def test_values_that_no_row_takes_do_not_matter(dev, kind, M):
    """NaN and infinities in adapters that no row names, in the scratch, and in
    another row's X, weights and adapter."""
    print(f"\n[case] lora NaN {kind} M={M}", flush=True)
    x, w, t, ids, weights = case_of(kind, M, 200, 264, 6, 16, 2, "mixed", True, 6)
    ids[ids == 3] = -1
    weights[ids == -1] = 1.0
    ws = torch.full((sw.swiglu_lora_workspace_size(M, 264, 200, 2, 16),), 0xFF, dtype=torch.uint8,
                    device=dev)
    first = run(kind, dev, x, w, t, ids, weights, workspace=ws)
    bad = {n: v.clone() for n, v in t.items()}
    bad["A"][3], bad["B"][3], bad["scale"][3] = float("nan"), float("inf"), float("nan")
    wbad = weights.clone()
    wbad[ids == -1] = float("nan")
    again = run(kind, dev, x, w, bad, ids, wbad)
    assert torch.equal(first, again)
    xbad = x.clone()
    xbad[7] = float("nan")
    wbad[9, 0] = float("inf")
    ids[9, 0] = 2
    ref = run(kind, dev, x, w, t, ids, weights)
    got = run(kind, dev, xbad, w, bad, ids, wbad)
    keep = [m for m in range(M) if m not in (7, 9)]
    assert torch.equal(ref[keep], got[keep])
    assert torch.isnan(got[7]).all()


@pytest.mark.parametrize("M", [30, 300])
def test_same_bits_and_rows_of_their_own(dev, M):
    """The same call gives the same bits; a row's result does not depend on
    the adapters of the others."""
    for kind in ("gated", "down"):
        print(f"\n[case] lora repeat {kind} M={M}", flush=True)
        x, w, t, ids, weights = case_of(kind, M, 520, 1000, 9, 24, 2, "mixed", True, 7)
        first = run(kind, dev, x, w, t, ids, weights)
        assert torch.equal(first, run(kind, dev, x, w, t, ids, weights))
        want, tol = (gated(x, w, t, ids, weights) if kind == "gated"
                     else rounded(*projected(x, w, t, 0, 1, ids, weights)))
        other = ids.clone()
        other[::2] = -1
        got = run(kind, dev, x, w, t, other, weights)
        within(got[1::2], want[1::2], tol[1::2], "rows whose adapters stayed")


def test_smallest_workspace(dev):
    """The bytes that are required: no split of K, the same result within the bounds."""
    for kind, M in (("gated", 20), ("down", 20), ("gated", 600), ("down", 600)):
        print(f"\n[case] lora workspace {kind} M={M}", flush=True)
        x, w, t, ids, weights = case_of(kind, M, 1024, 264, 5, 16, 1, "mixed", True, 8)
        up = lambda n: (n + 255) // 256 * 256  # noqa: E731
        need = (up(M * 1 * (2 if kind == "gated" else 1) * 16 * 4) +
                up((M + 255) // 256 * (4112 + 2 * 8)))
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        y = run(kind, dev, x, w, t, ids, weights, workspace=ws)
        want, tol = (gated(x, w, t, ids, weights) if kind == "gated"
                     else rounded(*projected(x, w, t, 0, 1, ids, weights)))
        within(y, want, tol, kind)


def test_outputs_end_where_they_end(dev):
    """Guard values around the output stay."""
    for kind, M, N in (("gated", 3, 8), ("down", 35, 24), ("gated", 130, 72), ("down", 257, 264)):
        print(f"\n[case] lora guards {kind} M={M} N={N}", flush=True)
        x, w, t, ids, weights = case_of(kind, M, 136, N, 3, 8, 1, "mixed", False, 9)
        store = torch.full((M * N + 512,), 7.0, dtype=BF, device=dev)
        out = store[256:256 + M * N].view(M, N)
        y = run(kind, dev, x, w, t, ids, weights, out=out)
        assert y.data_ptr() == out.data_ptr()
        assert (store[:256] == 7.0).all() and (store[256 + M * N:] == 7.0).all()
        want, tol = (gated(x, w, t, ids, weights) if kind == "gated"
                     else rounded(*projected(x, w, t, 0, 1, ids, weights)))
        within(y, want, tol, kind)


def test_a_table_past_32_bits(dev):
    """Adapters whose A and B begin past 2^31 bytes and elements."""
    K, N, r, L, M = 4096, 4096, 128, 2100, 5
    print("\n[case] lora far table", flush=True)
    g = torch.Generator().manual_seed(10)
    A = torch.zeros(L, r, K, dtype=BF, device=dev)        # 2.2 GB
    B = torch.zeros(L, N, r, dtype=BF, device=dev)
    small = table_of(g, 3, 1, N, K, r)
    at = [0, 1100, L - 1]
    for i, n in enumerate(at):
        A[n], B[n] = small["A"][i].to(dev), small["B"][i].to(dev)
    scale = torch.zeros(L, device=dev)
    scale[at] = small["scale"].to(dev)
    x = torch.randn(M, K, generator=g).to(BF)
    w = (torch.randn(N, K, generator=g) / K ** 0.5).to(BF)
    ids = torch.tensor([[at[0]], [at[2]], [-1], [at[1]], [at[2]]], dtype=torch.int32)
    y = sw.swiglu_down_proj_lora(x.to(dev), w.to(dev), sw.SwigluLora(A, B, scale), ids.to(dev))
    torch.cuda.synchronize()
    near = torch.tensor([[0], [2], [-1], [1], [2]], dtype=torch.int32)
    want, tol = rounded(*projected(x, w, small, 0, 1, near, None))
    within(y, want, tol, "far table")


def test_no_rows(dev):
    print("\n[case] lora M=0", flush=True)
    x, w, t, ids, _ = case_of("gated", 4, 64, 64, 2, 8, 1, "mixed", False, 11)
    y = sw.swiglu_fused_gemm_lora(x[:0].to(dev), w.to(dev), on(dev, t), ids[:0].to(dev))
    torch.cuda.synchronize()
    assert y.shape == (0, 64)


@pytest.mark.parametrize("M", [24, 400])
def test_graph_and_side_stream(dev, M):
    K, N, L, r, J = 512, 1000, 6, 16, 2
    print(f"\n[case] lora graph M={M}", flush=True)
    g = torch.Generator().manual_seed(12)
    x = torch.randn(M, K, generator=g).to(BF).to(dev)
    w = (torch.randn(2 * N, K, generator=g) / K ** 0.5).to(BF).to(dev)
    w3 = (torch.randn(K, N, generator=g) / N ** 0.5).to(BF).to(dev)
    up, down = on(dev, table_of(g, L, 2, 2 * N, K, r)), on(dev, table_of(g, L, 1, K, N, r))
    z = torch.randn(M, L, generator=g).to(dev)
    ids, weights, _, _ = sw.swiglu_route(z, J)
    ws = sw.make_lora_workspace(M, N, K, J, r, dev)

    def call(o):
        sw.swiglu_gated_mlp_lora(x, w, w3, up, down, ids, weights, H=o[0], Out=o[1], workspace=ws)
    outs = [torch.empty(M, N, dtype=BF, device=dev), torch.empty(M, K, dtype=BF, device=dev)]
    call(outs)
    static = [torch.empty_like(o) for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(static)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(outs, static))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(static)
    for _ in range(3):
        x.mul_(-0.5)
        ids.copy_((ids + 1) % L)
        call(outs)
        for o in static:
            o.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, static))


@pytest.mark.parametrize("kind,M,K,N,L,r,J,pattern", [
    ("gated", 5, 72, 16400, 3, 16, 1, "mixed"), ("gated", 64, 128, 16392, 20, 8, 2, "mixed"),
    ("down", 33, 200, 32776, 6, 24, 1, "mixed"), ("down", 64, 64, 32800, 4, 256, 8, "mixed"),
    ("gated", 40, 64, 16384, 5, 136, 3, "twice"), ("down", 1, 8, 40000, 2, 8, 1, "mixed")])
def test_few_rows_of_a_wide_weight(dev, kind, M, K, N, L, r, J, pattern):
    """A tile for every compute unit: the 64-row tiles."""
    check(dev, kind, M, K, N, L, r, J, pattern, J > 1, seed=M + K + r)


@pytest.mark.parametrize("tile,tail,M,K,N,r,J", [
    ("256", "fixup", 100, 520, 1400, 16, 2), ("256", "fixup", 7, 1024, 264, 64, 1),
    ("256", "fixup", 128, 600, 4600, 24, 4), ("128", "split", 100, 520, 1400, 16, 2),
    ("128", "whole", 128, 320, 9000, 64, 8), ("256", "split", 90, 1024, 1400, 256, 1)])
def test_every_schedule_of_few_rows(dev, tile, tail, M, K, N, r, J, monkeypatch):
    monkeypatch.setenv("SWIGLU_I_TILE", tile)
    monkeypatch.setenv("SWIGLU_TAIL", tail)
    check(dev, "gated", M, K, N, 6, r, J, "mixed", True, seed=3)
    check(dev, "down", M, K, N, 6, r, J, "mixed", True, seed=4)


def test_reduced_in_the_kernel_by_its_own_choice(dev):
    check(dev, "gated", 100, 3584, 4864, 8, 16, 1, "mixed", False, seed=5)


def one_after_the_other(x, w, t, part, parts, ids, weights):
    """projected() with sums that go one after the other: K + J r roundings."""
    D, err = projected(x, w, t, part, parts, ids, weights)
    size = x.double().abs() @ w[part::parts].double().abs().t()
    T = (x.double().abs() @ t["A"].double().abs().flatten(0, 1).t()).max() * 8 * t["scale"].abs().max()
    size += T * t["B"][:, part::parts].double().abs().sum(2).max()
    return D, err + (x.shape[1] + ids.shape[1] * t["B"].shape[2]) * 2.0 ** -24 * size


@pytest.mark.parametrize("kind", ["gated", "down"])
@pytest.mark.parametrize("M,K,N,r,J,tile,tail", [
    (1, 200, 264, 8, 2, None, None), (30, 200, 264, 16, 2, None, None),
    (50, 72, 16400, 24, 1, None, None), (100, 520, 1400, 40, 3, "256", "fixup"),
    (128, 520, 1400, 16, 2, "128", "split"), (300, 328, 1400, 16, 2, "256", "split"),
    (300, 328, 1400, 128, 8, "256", "quarter"), (520, 136, 1400, 16, 1, "256", "whole"),
    (520, 136, 1400, 8, 4, "128", "whole"), (300, 520, 520, 24, 2, "128", "split")])
def test_a_broken_adapter_is_its_rows_own(dev, kind, M, K, N, r, J, tile, tail, monkeypatch):
    """Infinities and NaN in the B of an adapter stay in the rows that name it, and
    are there what the formula makes of them."""
    print(f"\n[case] lora broken {kind} M={M} K={K} N={N} r={r} J={J} {tile} {tail}", flush=True)
    if tile:
        monkeypatch.setenv("SWIGLU_I_TILE", tile)
        monkeypatch.setenv("SWIGLU_TAIL", tail)
    x, w, t, ids, weights = case_of(kind, M, K, N, 5, r, J, "mixed", True, seed=M + r)
    weights += 0.25
    if M > 1:
        ids[ids == 2] = 1
        ids[::7, J - 1] = 2
    else:
        ids[0, 0], ids[0, 1] = 2, 1
    parts = 2 if kind == "gated" else 1
    bad = {n: v.clone() for n, v in t.items()}
    cols = parts * N
    inf_at = sorted({0, cols // 3 // parts * parts, cols - parts})
    for c in inf_at:
        bad["B"][2, c, c % r] = float("-inf") if c else float("inf")
    nan_at = sorted({parts * 5, cols // 2 // parts * parts})
    for c in nan_at:
        bad["B"][2, c, r - 1] = float("nan")
    touched = torch.zeros(N, dtype=torch.bool)
    touched[[c // parts for c in inf_at + nan_at]] = True
    named = (ids == 2).any(1)

    ref = run(kind, dev, x, w, t, ids, weights).cpu()
    got = run(kind, dev, x, w, bad, ids, weights).cpu()
    assert torch.equal(ref[:, ~touched], got[:, ~touched])
    if kind == "gated":
        g, ge = one_after_the_other(x, w, t, 0, 2, ids, weights)
        u, ue = one_after_the_other(x, w, t, 1, 2, ids, weights)
        s = g * torch.sigmoid(g)
        want, se = s * u, 1.1 * ge + s.abs() * 2.0 ** -20
        tol = (se * u.abs() + s.abs() * ue + se * ue) * (1 + 2.0 ** -8) + want.abs() * 2.0 ** -8
    else:
        want, tol = rounded(*one_after_the_other(x, w, t, 0, 1, ids, weights))
    if not named.all():
        within(got[~named], want[~named], tol[~named] + 2.0 ** -126, "the other rows")
    assert torch.isnan(got[named][:, [c // parts for c in nan_at]]).all()
    if kind == "down":
        a = x.double() @ t["A"][2].double().t()
        share = torch.where(ids == 2, weights.double(), 0.0).sum(1) * t["scale"][2].double()
        for c in inf_at:
            toward = (a[:, c % r] * share * float(bad["B"][2, c, c % r]))[named]
            assert torch.equal(got[named][:, c].double(), toward)
