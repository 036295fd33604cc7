"""swiglu_route and swiglu_route_backward against the definition in 64 bits
(needs an MI355X).

Picks, counts and the rows that route have to be equal.  Bounds of the computed
numbers, with u = 2^-24 (half an fp32 step): a probability takes the rounding of
z - max (|z - max| u in the exponential's argument, at most 40 u for the logits
here), exp itself (2 steps = 4 u), a sum of at most 512 terms (8 in a lane one
after the other, 6 levels over the lanes: 14 u), a reciprocal and a product
(4 u): 62 u, 2^-18 relative with a margin of one.  Probabilities under 2^-126
may be flushed.  The loss is a sum of non-negative terms: the mean of p adds the
rows one thread sums one after the other (at most 64 here: 64 u), the tree over
lanes and waves (22 u) and the final rounding: 2^-16 relative.  The gradient is
p (G - sum p G): both terms carry the relative error of a few such quantities,
so the bound is 2^-17 of p (|G| + sum p |G|) (and of the picked part's like),
plus half a bf16 step (2^-8) where the logits are bf16.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw

pytestmark = pytest.mark.gpu
NEG = float("-inf")


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    sw.load_library()
    return torch.device("cuda:0")


def logits_of(M, E, dtype, seed, closed=0.0, spread=1.5, ties=False):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(M, E, generator=g) * spread
    if ties:
        z = torch.round(z * 2) / 2          # many equal logits, zeros of both signs among them
        z = torch.where(torch.rand(M, E, generator=g) < 0.2, -z, z)
    if closed:
        z = torch.where(torch.rand(M, E, generator=g) < closed, torch.full_like(z, NEG), z)
    return z.to(dtype)


def definition(z, k, valid, normalize):
    """Rows one by one, in 64 bits."""
    z = z.double().numpy()
    M, E = z.shape
    p = np.zeros((M, E))
    ids = np.full((M, k), -1, dtype=np.int64)
    w = np.zeros((M, k))
    live = np.zeros(M, dtype=bool)
    for m in range(M):
        if (valid is not None and not valid[m]) or np.all(z[m] == -np.inf):
            continue
        live[m] = True
        e = np.exp(z[m] - z[m].max())
        p[m] = e / e.sum()
        picks = [i for i in sorted(range(E), key=lambda i: (-z[m, i], i)) if z[m, i] > -np.inf][:k]
        ids[m, :len(picks)] = picks
        w[m, :len(picks)] = p[m, picks]
        if normalize:
            w[m] = np.pad(e[picks], (0, k - len(picks))) / e[picks].sum()
    counts = np.bincount(ids[ids >= 0], minlength=E)
    n, total = int(live.sum()), int(counts.sum())
    loss = E * float((counts / max(total, 1) * p.sum(0) / max(n, 1)).sum())
    return p, live, ids, w, counts, n, total, loss


def gradient(p, live, ids, w, counts, n, total, dw, d_loss, normalize):
    """(d_logits, the sum of the magnitudes of what it is the difference of)."""
    M, E = p.shape
    g = np.broadcast_to(d_loss * E * counts / (max(total, 1) * max(n, 1)), (M, E))
    pick = np.zeros((M, E))
    pick_abs = np.zeros((M, E))
    dw = np.where(ids >= 0, dw, 0.0)
    if normalize:
        wdw = (w * dw).sum(1, keepdims=True)
        part, part_abs = w * (dw - wdw), w * (abs(dw) + (w * abs(dw)).sum(1, keepdims=True))
    else:
        part, part_abs = dw, abs(dw)
    for m in range(M):
        for j in range(ids.shape[1]):
            if ids[m, j] >= 0:
                pick[m, ids[m, j]] += part[m, j]
                pick_abs[m, ids[m, j]] += part_abs[m, j]
    if normalize:
        dz = p * (g - (p * g).sum(1, keepdims=True)) + pick
        size = p * (abs(g) + (p * abs(g)).sum(1, keepdims=True)) + pick_abs
    else:
        G, Ga = g + pick, abs(g) + pick_abs
        dz = p * (G - (p * G).sum(1, keepdims=True))
        size = p * (Ga + (p * Ga).sum(1, keepdims=True))
    return np.where(live[:, None], dz, 0.0), np.where(live[:, None], size, 0.0)


def check(dev, M, E, k, dtype, normalize, seed, closed=0.0, valid_share=None, spread=1.5,
          ties=False, z=None, workspace=None):
    print(f"\n[case] route M={M} E={E} k={k} {dtype} normalize={normalize} closed={closed} "
          f"valid={valid_share} seed={seed}", flush=True)
    if z is None:
        z = logits_of(M, E, dtype, seed, closed, spread, ties)
    g = torch.Generator().manual_seed(seed + 1)
    valid = None
    if valid_share is not None:
        valid = (torch.rand(M, generator=g) < valid_share).to(torch.uint8)
    dw = torch.randn(M, k, generator=g)
    d_loss = torch.tensor(0.37)
    zd = z.to(dev)
    vd = None if valid is None else valid.to(dev)
    ids, w, counts, loss = sw.swiglu_route(zd, k, valid=vd, normalize=normalize,
                                           workspace=workspace)
    dz = sw.swiglu_route_backward(zd, ids, w, counts, d_weights=dw.to(dev),
                                  d_loss=d_loss.to(dev), valid=vd, normalize=normalize)
    torch.cuda.synchronize()
    p, live, r_ids, r_w, r_counts, n, total, r_loss = definition(
        z, k, None if valid is None else valid.numpy(), normalize)
    assert np.array_equal(ids.cpu().numpy(), r_ids)
    assert np.array_equal(counts.cpu().numpy(), np.append(r_counts, n))
    err = np.abs(w.cpu().double().numpy() - r_w)
    assert (err <= 2.0 ** -18 * r_w + 2.0 ** -126).all(), err.max()
    assert abs(float(loss) - r_loss) <= 2.0 ** -16 * r_loss, (float(loss), r_loss)
    r_dz, size = gradient(p, live, r_ids, r_w, r_counts, n, total, dw.double().numpy(),
                          float(d_loss.double()), normalize)
    err = np.abs(dz.cpu().double().numpy() - r_dz)
    tol = 2.0 ** -17 * size + 2.0 ** -120
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(r_dz) + tol)
    assert (err <= tol).all(), (err / tol).max()
    assert dz.dtype == dtype
    return ids, w, counts, loss, dz


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("normalize", [True, False], ids=["normalized", "raw"])
@pytest.mark.parametrize("M,E,k", [
    (1, 1, 1), (1, 8, 2), (3, 2, 2), (5, 7, 3), (17, 32, 4), (31, 33, 5), (64, 61, 3), (65, 64, 8),
    (33, 100, 16), (257, 128, 8), (40, 129, 6), (19, 256, 16), (9, 257, 1), (21, 500, 7),
    (13, 512, 16), (16, 16, 16)])
def test_sizes(dev, M, E, k, dtype, normalize):
    check(dev, M, E, k, dtype, normalize, seed=M * 1000 + E + k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("normalize", [True, False], ids=["normalized", "raw"])
@pytest.mark.parametrize("M,E,k,closed,share", [
    (50, 6, 4, 0.6, None), (200, 64, 8, 0.05, 0.9), (70, 61, 3, 0.95, 0.5), (30, 8, 8, 0.9, None),
    (12, 16, 2, 1.0, None), (25, 64, 4, 0.0, 0.0), (1100, 20, 2, 0.3, 0.7)])
def test_closed_experts_and_padding(dev, M, E, k, closed, share, dtype, normalize):
    check(dev, M, E, k, dtype, normalize, seed=M + E, closed=closed, valid_share=share)


@pytest.mark.parametrize("E,k", [(8, 3), (64, 8), (200, 16)])
def test_ties_go_to_the_lowest_index(dev, E, k):
    check(dev, 60, E, k, torch.float32, True, seed=E, ties=True)
    check(dev, 60, E, k, torch.bfloat16, False, seed=E + 1, ties=True)
    check(dev, 20, E, k, torch.float32, False, seed=2, z=torch.zeros(20, E))


def test_many_rows(dev):
    # several passes a workgroup, partial sums over all workgroups
    check(dev, 40007, 12, 2, torch.float32, True, seed=3, closed=0.1, valid_share=0.9)
    check(dev, 9001, 96, 4, torch.bfloat16, False, seed=4)


def test_far_apart_logits_and_the_types_lowest_value(dev):
    print("\n[case] route far apart", flush=True)
    z = logits_of(64, 16, torch.float32, 5)
    z[::2] *= 40.0                                  # probabilities that flush to zero
    z[1, 3] = torch.finfo(torch.float32).min        # finite: picked, with weight 0
    z[3] = torch.finfo(torch.float32).min
    z[5] = 3.0e38
    z[7, 0] = 3.0e38
    for normalize in (True, False):
        ids, w, counts, loss = sw.swiglu_route(z.to(dev), 16, normalize=normalize)
        p, live, r_ids, r_w, r_counts, n, total, r_loss = definition(z, 16, None, normalize)
        torch.cuda.synchronize()
        assert np.array_equal(ids.cpu().numpy(), r_ids)
        # |z - max| up to 500: its rounding reaches exp as 500 u; flushed under 2^-126
        err = np.abs(w.cpu().double().numpy() - r_w)
        assert (err <= 2.0 ** -14 * r_w + 2.0 ** -120).all()
        assert abs(float(loss) - r_loss) <= 2.0 ** -14 * r_loss


def test_one_workgroup_without_workspace_gives_the_same(dev):
    z = logits_of(3000, 40, torch.float32, 6, closed=0.1).to(dev)
    print("\n[case] route without workspace", flush=True)
    a = sw.swiglu_route(z, 4)
    b = [torch.empty_like(t) for t in a]
    st = sw.load_library().swiglu_route(z.data_ptr(), sw.SWIGLU_F32, None, *(t.data_ptr() for t in b),
                                        3000, 40, 4, 1, None, 0,
                                        torch.cuda.current_stream(dev).cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    for i in range(3):
        assert torch.equal(a[i], b[i])
    assert abs(float(a[3]) - float(b[3])) <= 2.0 ** -16 * float(a[3])


def test_same_bits_every_time(dev):
    z = logits_of(20000, 64, torch.float32, 7).to(dev)
    print("\n[case] route repeated", flush=True)
    first = sw.swiglu_route(z, 4)
    for _ in range(3):
        again = sw.swiglu_route(z, 4)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_no_rows(dev):
    print("\n[case] route M=0", flush=True)
    z = torch.empty(0, 5, device=dev)
    ids, w, counts, loss = sw.swiglu_route(z, 2)
    dz = sw.swiglu_route_backward(z, ids, w, counts)
    torch.cuda.synchronize()
    assert counts.tolist() == [0] * 6 and float(loss) == 0.0 and dz.shape == (0, 5)


def test_values_in_padding_and_nan_logits_stay_in_their_row(dev):
    print("\n[case] route NaN", flush=True)
    z = logits_of(40, 10, torch.float32, 8)
    valid = torch.ones(40, dtype=torch.bool)
    bad = z.clone()
    bad[4] = float("nan")
    bad[5] = float("inf")
    bad[6, 2] = float("nan")
    valid[4:7] = False
    args = dict(valid=valid.to(dev), normalize=False)
    x, y = sw.swiglu_route(z.to(dev), 3, **args), sw.swiglu_route(bad.to(dev), 3, **args)
    assert all(torch.equal(a, b) for a, b in zip(x, y))
    dw = torch.randn(40, 3, device=dev)
    a = sw.swiglu_route_backward(z.to(dev), *x[:3], d_weights=dw, **args)
    b = sw.swiglu_route_backward(bad.to(dev), *y[:3], d_weights=dw, **args)
    assert torch.equal(a, b) and not a[4:7].any()
    # in a row that routes: that row's weights only (and the loss)
    ids, w, _, loss = sw.swiglu_route(bad.to(dev), 3, normalize=False)
    assert torch.isnan(w[4]).all() and torch.isnan(w[6]).all() and torch.isnan(loss)
    assert not torch.isnan(w[[*range(4), *range(7, 40)]]).any()
    assert int(ids.min()) >= 0 and int(ids.max()) < 10


def test_gradient_against_differences(dev):
    """The definition's loss in 64 bits, moved by +-h along a direction: the
    second-order remainder is under h^2 times a constant of a few units, and
    the picks do not change at this h."""
    M, E, k, h = 24, 12, 3, 1e-4
    for normalize in (True, False):
        print(f"\n[case] route differences normalize={normalize}", flush=True)
        z = logits_of(M, E, torch.float32, 9)
        g = torch.Generator().manual_seed(10)
        dw, way = torch.randn(M, k, generator=g), torch.randn(M, E, generator=g).double()
        ids, w, counts, _ = sw.swiglu_route(z.to(dev), k, normalize=normalize)
        dz = sw.swiglu_route_backward(z.to(dev), ids, w, counts, d_weights=dw.to(dev),
                                      d_loss=torch.tensor(0.5, device=dev), normalize=normalize)

        def value(x):
            _, _, i, v, _, _, _, loss = definition(x, k, None, normalize)
            assert np.array_equal(i, ids.cpu().numpy())
            return float((v * dw.double().numpy()).sum() + 0.5 * loss)
        slope = (value(z.double() + h * way) - value(z.double() - h * way)) / (2 * h)
        got = float((dz.cpu().double() * way).sum())
        # third derivatives along `way` (|way| < 4 an element) of M rows: h^2 / 6 * M * 4^3 * 6
        assert abs(got - slope) <= h * h * M * 64 + 2.0 ** -17 * float(way.abs().sum()), (got, slope)


def test_gradient_without_one_of_the_two(dev):
    z = logits_of(50, 20, torch.float32, 11).to(dev)
    print("\n[case] route gradient parts", flush=True)
    for normalize in (True, False):
        ids, w, counts, _ = sw.swiglu_route(z, 4, normalize=normalize)
        dw, dl = torch.randn(50, 4, device=dev), torch.tensor(0.3, device=dev)
        kw = dict(normalize=normalize)
        zero = sw.swiglu_route_backward(z, ids, w, counts, **kw)
        a = sw.swiglu_route_backward(z, ids, w, counts, d_weights=dw, **kw)
        b = sw.swiglu_route_backward(z, ids, w, counts, d_loss=dl, **kw)
        c = sw.swiglu_route_backward(z, ids, w, counts, d_weights=dw, d_loss=dl, **kw)
        assert not zero.any()
        assert torch.equal(a, sw.swiglu_route_backward(z, ids, w, counts, d_weights=dw,
                                                       d_loss=torch.zeros((), device=dev), **kw))
        assert float((a + b - c).abs().max()) <= 2.0 ** -17 * float(dw.abs().max())


def test_unaligned_rows_and_outputs(dev):
    """Logits that begin at any element (rows not 16-byte aligned)."""
    print("\n[case] route unaligned", flush=True)
    for dtype in (torch.float32, torch.bfloat16):
        z = logits_of(30, 64, dtype, 12).to(dev)
        store = torch.empty(30 * 64 + 1, dtype=dtype, device=dev)
        off = store[1:].view(30, 64)
        off.copy_(z)
        grad = torch.empty(30 * 64 + 1, dtype=dtype, device=dev)[1:].view(30, 64)
        x, y = sw.swiglu_route(z, 4), sw.swiglu_route(off, 4)
        assert all(torch.equal(a, b) for a, b in zip(x, y))
        dw = torch.randn(30, 4, device=dev)
        a = sw.swiglu_route_backward(z, *x[:3], d_weights=dw)
        b = sw.swiglu_route_backward(off, *y[:3], d_weights=dw, d_logits=grad)
        assert b.data_ptr() == grad.data_ptr() and torch.equal(a, b)


def test_graph_and_side_stream(dev):
    print("\n[case] route graph", flush=True)
    z = logits_of(5000, 64, torch.float32, 13).to(dev)
    dw, dl = torch.randn(5000, 4, device=dev), torch.tensor(0.2, device=dev)
    ws = torch.empty(max(1, sw.swiglu_route_workspace_size(5000, 64)), dtype=torch.uint8, device=dev)
    outs = list(sw.swiglu_route(z, 4, workspace=ws)) + [torch.empty_like(z)]

    def call(o):
        sw.swiglu_route(z, 4, ids=o[0], weights=o[1], counts=o[2], loss=o[3], workspace=ws)
        sw.swiglu_route_backward(z, o[0], o[1], o[2], d_weights=dw, d_loss=dl, d_logits=o[4])
    call(outs)
    static = [torch.empty_like(o) for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(static)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(outs, static))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(static)
    for _ in range(3):
        z.add_(0.25 * torch.randn_like(z))
        call(outs)
        for o in static:
            o.fill_(0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, static))
