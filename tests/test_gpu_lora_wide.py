"""Low-rank adapters at the ends of their sizes (needs an MI355X): the 64-row tiles of a
wide weight with tiles split along K, and the largest table.  Definitions and bounds are
those of test_gpu_lora.
"""
from __future__ import annotations

import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw
from test_gpu_lora import case_of, check, gated, projected, rounded, run, within

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    sw.load_library()
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def split(monkeypatch):
    monkeypatch.delenv("SWIGLU_I_TILE", raising=False)
    monkeypatch.setenv("SWIGLU_TAIL", "split")


def width(dev, kind, extra):
    """Columns of the output that make a tile of 128 columns for every compute unit and
    `extra` more, the last one ragged: those are the split ones."""
    cus = torch.cuda.get_device_properties(dev).multi_processor_count
    cols = (cus + extra) * 128 - 112
    return cols // 2 if kind == "gated" else cols


# pieces: min(CUs / extra, K steps of 64): 4 of 256 CUs, each with a share of the adapters;
# one K step each
@pytest.mark.parametrize("kind", ["gated", "down"])
@pytest.mark.parametrize("M,K,extra,L,r,J,pattern", [
    (64, 1000, 57, 30, 16, 2, "mixed"), (64, 512, 57, 17, 40, 1, "mixed"), (5, 576, 1, 4, 8, 1, "mixed"),
    (33, 840, 100, 50, 64, 3, "twice"), (1, 2048, 30, 3, 24, 2, "mixed")])
def test_64_row_tiles_split_along_k(dev, kind, M, K, extra, L, r, J, pattern):
    check(dev, kind, M, K, width(dev, kind, extra), L, r, J, pattern, J > 1, seed=M + K + r)


@pytest.mark.parametrize("kind", ["gated", "down"])
def test_a_broken_adapter_in_64_row_tiles_split_along_k(dev, kind):
    M, K, L, r, J = 50, 712, 12, 16, 2
    N = width(dev, kind, 57)
    print(f"\n[case] lora broken {kind} M={M} K={K} N={N}", flush=True)
    x, w, t, ids, weights = case_of(kind, M, K, N, L, r, J, "mixed", True, 21)
    ids[ids == 9] = 8
    ids[::7, 0] = 9
    bad = {n: v.clone() for n, v in t.items()}
    bad["B"][9, :, 3] = float("nan")
    named = (ids == 9).any(1)
    got = run(kind, dev, x, w, bad, ids, weights).cpu()
    want, tol = (gated(x, w, t, ids, weights) if kind == "gated"
                 else rounded(*projected(x, w, t, 0, 1, ids, weights)))
    within(got[~named], want[~named], tol[~named], "the other rows")
    assert torch.isnan(got[named]).all()


def table_with(dev, L, parts, columns, K, r, small, at):
    """A table of zeros on the device with the small one's adapters at places `at`."""
    A = torch.zeros(L, parts * r, K, dtype=BF, device=dev)
    B = torch.zeros(L, columns, r, dtype=BF, device=dev)
    scale = torch.zeros(L, device=dev)
    for i, n in enumerate(at):
        A[n], B[n], scale[n] = small["A"][i].to(dev), small["B"][i].to(dev), small["scale"][i].to(dev)
    return sw.SwigluLora(A, B, scale)


@pytest.mark.parametrize("kind", ["gated", "down"])
@pytest.mark.parametrize("M", [5, 300])
def test_the_largest_table(dev, kind, M):
    """8192 adapters, the last of which begin at 2^33 bytes and 2^32 elements less one
    adapter (down projection), or twice as far (Gate and Up)."""
    K, N, r, L = 4096, 4096, 128, 8192
    print(f"\n[case] lora largest table {kind} M={M}", flush=True)
    at = [0, 2047, 4095, 8190, 8191]
    parts = 2 if kind == "gated" else 1
    assert (L - 1) * r * K >= 2 ** 32 - 2 ** 19
    x, w, t, ids, weights = case_of(kind, M, K, N, len(at), r, 1, "mixed", True, 31)
    ids[0, 0], ids[1, 0] = 4, 3
    table = table_with(dev, L, parts, parts * N, K, r, t, at)
    far = torch.where(ids >= 0, torch.tensor(at, dtype=torch.int32)[ids.clamp(min=0).long()], ids)
    got = run(kind, dev, x, w, None, far, weights, lora=table)
    want, tol = (gated(x, w, t, ids, weights) if kind == "gated"
                 else rounded(*projected(x, w, t, 0, 1, ids, weights)))
    within(got, want, tol, "largest table")
    # every adapter named at once: the zeros among them change nothing
    if M == 300:
        ids2 = torch.cat([far, torch.arange(M, dtype=torch.int32)[:, None] * 27 + 5], 1).contiguous()
        ids2[:, 1][torch.isin(ids2[:, 1], torch.tensor(at, dtype=torch.int32))] = 1
        more = run(kind, dev, x, w, None, ids2, torch.cat([weights, weights], 1), lora=table)
        within(more, want, tol, "with 300 more")
