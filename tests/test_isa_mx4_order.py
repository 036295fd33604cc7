"""The order of the loads that the 4-bit tiles' counted waits rest on (CPU: the compiled
gfx950 code).

A K step of a tile with 4-bit weights waits for the activations' panel of the next step by
a count: all vector memory operations but the youngest
    (STAGES - 2) panels of A + one fetch of codes and scales
are done (IssueOrder::kWaitSteady).  That holds the panel back only if the fetch stays
behind it: the panels' loads write LDS and the fetch, which writes registers, is an ordinary
load that the compiler may place.  So, on every path into such a wait, at most STAGES - 2
panels' worth of LDS loads may be among the operations that it leaves in flight.
"""
from __future__ import annotations

import os
import re

import pytest

from gated_mlp_gemm_amd import build

SHAPE = re.compile(r"gemm_tiles_kernelINS_9TileShapeI" + r"Li(\d+)E" * 9 + "Lb0ELb0ELb1EEE")
VMEM = ("buffer_load", "buffer_store", "buffer_atomic", "global_load", "global_store",
        "global_atomic", "flat_")


def _to_lds(ins):
    return ins.startswith("buffer_load") and ins.endswith(" lds")


def flow(lines):
    """Instructions (labels dropped) and, for each, what can run right before it: (its
    index, a condition).  The condition is that of the flags the compiler keeps for arms of
    which exactly one runs,
        s_mov_b64 F, -1 / if: ... s_mov_b64 F, 0 / s_andn2_b64 vcc, exec, F / s_cbranch_vccz
    (F, its value) where the branch is such a one, else None."""
    ins, at, pending = [], {}, []
    for line in lines:
        if line.endswith(":"):
            pending.append(line[:-1])
            continue
        at.update((name, len(ins)) for name in pending)
        pending = []
        ins.append(line)
    preds = [[] for _ in ins]
    for i, line in enumerate(ins):
        op = line.split()[0]
        flag, j = None, i - 1
        if op in ("s_cbranch_vccz", "s_cbranch_vccnz"):
            while j >= 0 and not re.match(r"s_cbranch|s_branch|\S+ vcc\b|v_cmp", ins[j]):
                j -= 1
            m = re.fullmatch(r"s_andn2_b64 vcc, exec, (s\[\d+:\d+\])", ins[j]) if j >= 0 else None
            flag = m and m.group(1)
        # vcc = exec & ~F is zero where F is -1
        taken = (flag, -1 if op == "s_cbranch_vccz" else 0) if flag else None
        other = (flag, 0 if op == "s_cbranch_vccz" else -1) if flag else None
        if i + 1 < len(ins) and op not in ("s_branch", "s_endpgm", "s_setpc_b64"):
            preds[i + 1].append((i, other))
        if (op == "s_branch" or op.startswith("s_cbranch")) and line.split()[-1] in at:
            preds[at[line.split()[-1]]].append((i, taken))
    return ins, preds


def most_lds_loads(ins, preds, i, n):
    """The most LDS loads among the n youngest vector memory operations before instruction
    i, over all paths into it (but those on which a flag would have two values)."""
    most, seen = 0, set()
    stack = [(i, n, 0, frozenset())]
    while stack:
        state = stack.pop()
        if state in seen:
            continue
        seen.add(state)
        at, left, lds, flags = state
        for j, condition in preds[at]:
            known = dict(flags)
            if condition and known.setdefault(*condition) != condition[1]:
                continue
            l, d = left, lds
            if ins[j].startswith(VMEM):
                l, d = left - 1, lds + _to_lds(ins[j])
                most = max(most, d)
            written = re.match(r"s_\w+ (s\[\d+:\d+\])(?:, (-1|0)$)?", ins[j])
            if written and written.group(1) in known:
                value = known.pop(written.group(1))
                if ins[j].startswith("s_mov_b64") and written.group(2) and int(written.group(2)) != value:
                    continue
            if l:
                stack.append((j, l, d, frozenset(known.items())))
    return most


def steady_waits(ins, count):
    """The waits that leave `count` operations in flight, right before a barrier."""
    return [i for i in range(len(ins) - 1)
            if ins[i] == f"s_waitcnt vmcnt({count})" and ins[i + 1].startswith("s_barrier")]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    path = build.device_assembly(os.path.join(tmp_path_factory.mktemp("isa"), "kernels.s"))
    with open(path) as f:
        text = f.read()
    found = {}
    for m in re.finditer(r"^(_Z\w+):", text, re.M):
        shape = SHAPE.search(m.group(1))
        if not shape:
            continue
        body = text[m.end():text.find(".Lfunc_end", m.end())]
        lines = [raw.split(";")[0].strip() for raw in body.split("\n")]
        lines = [x for x in lines if x and (x.endswith(":") or not x.startswith("."))]
        found[m.group(1)] = ([int(x) for x in shape.groups()], lines)
    return found


def test_the_counter():
    dma, code, wait = "buffer_load_dwordx4 v1, s[0:3], 0 offen lds", \
        "buffer_load_dwordx4 v[4:7], v1, s[0:3], 0 offen", "s_waitcnt vmcnt(1)"

    def most(*lines):
        ins, preds = flow([*lines, wait, "s_barrier"])
        (i,) = steady_waits(ins, 1)
        return most_lds_loads(ins, preds, i, 1)

    assert most(dma, code) == 0
    assert most(code, "v_mov_b32 v0, 0", dma) == 1          # the fetch ahead of the panel
    assert most(dma, code, "s_cbranch_scc1 .LBB0_1", dma, ".LBB0_1:") == 1   # on one path
    assert most(dma, code, "buffer_store_dword v0, v1, s[0:3], 0 offen") == 0
    # one of two arms fetches, whichever: no path without a fetch
    arms = ("s_mov_b64 s[8:9], -1", "s_mov_b64 vcc, s[6:7]", "s_cbranch_vccz .LBB0_1", code,
            "s_mov_b64 s[8:9], 0", ".LBB0_1:", "s_andn2_b64 vcc, exec, s[8:9]",
            "s_cbranch_vccnz .LBB0_2")
    assert most(dma, *arms, code, ".LBB0_2:") == 0
    assert most(dma, *arms, "v_mov_b32 v0, 0", ".LBB0_2:") == 1   # the second arm does not
    assert most(dma, *(x for x in arms if x != code), code, ".LBB0_2:") == 1   # nor the first


def test_fetches_stay_behind_the_panels(kernels):
    assert len(kernels) == 6, list(kernels)
    for name, ((bm, bn, bk, wm, wn, stages, eb, bstages, mi), lines) in kernels.items():
        threads = 64 * wm * wn
        panel = bm * bk * eb // (threads * 16)                     # LDS loads of A, a step
        codes = bn * bk // 2 // threads                            # bytes a lane
        fetch = 2 * (codes // min(codes, 16))                      # loads: codes and scales
        allowed = (stages - 2) * panel
        ins, preds = flow(lines)
        waits = steady_waits(ins, allowed + fetch)
        # the generic step, the unrolled ones and the first step, of each of two bodies
        assert len(waits) >= 8, (name, len(waits))
        for i in waits:
            got = most_lds_loads(ins, preds, i, allowed + fetch)
            assert got <= allowed, (name, i, got, allowed)
