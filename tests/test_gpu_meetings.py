"""Launches whose workgroups meet in the workspace (needs an MI355X): the router
of many rows, the adapters' shrink split along K, the fused product split along K
and reduced in the kernel.

Each call counts arrivals in words of its own workspace, whatever these hold
before, so calls with workspaces of their own may run at the same time: any number
of them in flight, on several streams, and captured ones replayed beside them.
"""
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


def bits(t):
    return t.reshape(-1).view(torch.uint8)


class Route:
    """Rows enough for a workgroup on every compute unit."""
    M, E, k = 20000, 64, 4

    def __init__(self, dev, seed):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.z = torch.randn(self.M, self.E, generator=g, device=dev)
        n = sw.swiglu_route_workspace_size(self.M, self.E)
        assert n > 0
        self.ws = torch.empty(n, dtype=torch.uint8, device=dev)

    def outputs(self):
        new = lambda shape, t: torch.empty(shape, dtype=t, device=self.z.device)  # noqa: E731
        return [new((self.M, self.k), torch.int32), new((self.M, self.k), torch.float32),
                new(self.E + 1, torch.int32), new((), torch.float32)]

    def call(self, o):
        sw.swiglu_route(self.z, self.k, ids=o[0], weights=o[1], counts=o[2], loss=o[3],
                        workspace=self.ws)


class Down:
    """A shrink whose K is split 16 ways."""
    M, N, D, L, r = 33, 8192, 512, 6, 8

    def __init__(self, dev, seed):
        g = torch.Generator(device=dev).manual_seed(seed)
        new = lambda *shape: torch.randn(*shape, generator=g, device=dev).mul_(0.05).to(BF)  # noqa: E731
        self.h, self.w = new(self.M, self.N), new(self.D, self.N)
        self.table = sw.SwigluLora(new(self.L, self.r, self.N), new(self.L, self.D, self.r),
                                   torch.rand(self.L, generator=g, device=dev))
        self.ids = torch.randint(0, self.L, (self.M, 1), generator=g, device=dev, dtype=torch.int32)
        self.ws = sw.make_lora_workspace(self.M, self.D, self.N, 1, self.r, dev)

    def outputs(self):
        return [torch.empty(self.M, self.D, dtype=BF, device=self.h.device)]

    def call(self, o):
        sw.swiglu_down_proj_lora(self.h, self.w, self.table, self.ids, Out=o[0], workspace=self.ws)


class Fused:
    """Tiles split three ways along K, reduced in the kernel."""
    M, N, K = 100, 4864, 3584

    def __init__(self, dev, seed):
        g = torch.Generator(device=dev).manual_seed(seed)
        new = lambda *shape: torch.randn(*shape, generator=g, device=dev).mul_(0.05).to(BF)  # noqa: E731
        self.x, self.w = new(self.M, self.K), new(2 * self.N, self.K)
        self.ws = sw.make_workspace(self.M, self.N, self.K, "i", dev)
        assert "reduced in the kernel" in sw.swiglu_describe_launch(self.M, self.N, self.K, "i",
                                                                     self.ws.numel())

    def outputs(self):
        return [torch.empty(self.M, self.N, dtype=BF, device=self.x.device)]

    def call(self, o):
        sw.swiglu_fused_gemm(self.x, self.w, Y=o[0], variant="i", workspace=self.ws)


class FusedLora(Fused):
    """The same with adapters (the shrink and the product both meet)."""

    def __init__(self, dev, seed):
        super().__init__(dev, seed)
        g = torch.Generator(device=dev).manual_seed(seed + 1)
        new = lambda *shape: torch.randn(*shape, generator=g, device=dev).mul_(0.05).to(BF)  # noqa: E731
        self.table = sw.SwigluLora(new(4, 32, self.K), new(4, 2 * self.N, 16),
                                   torch.rand(4, generator=g, device=dev))
        self.ids = torch.randint(0, 4, (self.M, 1), generator=g, device=dev, dtype=torch.int32)
        self.ws = sw.make_lora_workspace(self.M, self.N, self.K, 1, 16, dev)

    def call(self, o):
        sw.swiglu_fused_gemm_lora(self.x, self.w, self.table, self.ids, Y=o[0], workspace=self.ws)


KINDS = [Route, Down, Fused, FusedLora]


@pytest.mark.parametrize("kind", KINDS)
def test_whatever_the_workspace_holds(dev, kind):
    print(f"\n[case] workspace contents {kind.__name__}", flush=True)
    c = kind(dev, 1)
    want, got = c.outputs(), c.outputs()
    c.ws.zero_()
    c.call(want)
    g = torch.Generator(device=dev).manual_seed(2)
    for fill in ("ones", "twos", "noise", "left", "left"):
        if fill == "ones":
            c.ws.fill_(255)
        elif fill == "twos":
            c.ws.fill_(1)
        elif fill == "noise":
            c.ws.random_(0, 256, generator=g)
        for o in got:
            o.fill_(7)
        c.call(got)
        torch.cuda.synchronize()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(want, got)), fill


def test_many_in_flight_on_several_streams(dev):
    """Each stream with calls of all kinds, more of them queued than any table of the
    library's could hold, every call with results of its own."""
    print("\n[case] many in flight", flush=True)
    streams = [torch.cuda.Stream() for _ in range(3)]
    each = [[kind(dev, 10 * s + i) for i, kind in enumerate(KINDS)] for s in range(len(streams))]
    want = [[c.outputs() for c in cs] for cs in each]
    for cs, os_ in zip(each, want):
        for c, o in zip(cs, os_):
            c.call(o)
    torch.cuda.synchronize()
    rounds = 20
    got = [[[c.outputs() for c in cs] for _ in range(rounds)] for cs in each]
    torch.cuda.synchronize()
    # one stream's whole queue before the next one's, and then turn by turn
    for s, stream in enumerate(streams):
        with torch.cuda.stream(stream):
            for r in range(rounds // 2):
                for c, o in zip(each[s], got[s][r]):
                    c.call(o)
    for r in range(rounds // 2, rounds):
        for s, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                for c, o in zip(each[s], got[s][r]):
                    c.call(o)
    torch.cuda.synchronize()
    for s in range(len(streams)):
        for r in range(rounds):
            for i, kind in enumerate(KINDS):
                assert all(torch.equal(bits(a), bits(b)) for a, b in zip(want[s][i], got[s][r][i])), (
                    s, r, kind.__name__)


def test_captured_calls_beside_eager_ones(dev):
    """A graph of all kinds, replayed on one stream while eager calls, more than 64 of
    them a replay, run on another."""
    print("\n[case] graph beside eager", flush=True)
    inside = [kind(dev, 40 + i) for i, kind in enumerate(KINDS)]
    beside = [kind(dev, 50 + i) for i, kind in enumerate(KINDS)]
    want_in, want_out = [c.outputs() for c in inside], [c.outputs() for c in beside]
    for c, o in zip(inside + beside, want_in + want_out):
        c.call(o)
    torch.cuda.synchronize()
    got_in = [c.outputs() for c in inside]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(5):
            for c, o in zip(inside, got_in):
                c.call(o)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got_out = [[c.outputs() for c in beside] for _ in range(20)]
        for outs in got_in:
            for o in outs:
                o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(one):
            graph.replay()
        with torch.cuda.stream(two):
            for outs in got_out:
                for c, o in zip(beside, outs):
                    c.call(o)
        torch.cuda.synchronize()
        assert all(torch.equal(bits(a), bits(b)) for w, g in zip(want_in, got_in) for a, b in zip(w, g))
        for outs in got_out:
            assert all(torch.equal(bits(a), bits(b)) for w, g in zip(want_out, outs)
                       for a, b in zip(w, g))
