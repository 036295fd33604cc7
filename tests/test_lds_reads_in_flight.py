"""LDS reads in flight, in the compiled gfx950 code (CPU: hipcc cross-compiles).

The kernels' LDS reads are inline assembly, so the compiler takes their destination
registers as written at once, and as free where no later use of the value follows on a
path (the reads of the step behind the last one).  A register reused before the read's
data lands is overwritten by it: a wrong value, or an address that faults.  So no
instruction may touch the destination of an LDS read before a wait that covers the read,
on any path.  LDS accesses return in order: s_waitcnt lgkmcnt(N) covers a read with at
least N LDS accesses behind it (scalar loads, which return in any order, do not count)."""
from __future__ import annotations

import re

from test_isa_invariants import _flow, _operands, _regs, assembly  # noqa: F401

_LGKM = re.compile(r"lgkmcnt\((\d+)\)")
_MOST = 15   # lgkmcnt holds 4 bits


def touched_in_flight(lines):
    """(read, instruction) for each read whose destination an instruction touches before
    a wait that covers it (the first instruction found)."""
    ins, preds = _flow(lines)
    after = [[] for _ in ins]
    for i, ps in enumerate(preds):
        for p in ps:
            after[p].append(i)
    registers = {}
    found = []
    for i, read in enumerate(ins):
        if not read.startswith("ds_read"):
            continue
        destination = _regs(_operands(read)[0])
        fewest = {}                     # instruction -> fewest LDS accesses behind the read
        stack = [(j, 0) for j in after[i]]
        while stack:
            j, behind = stack.pop()
            if fewest.get(j, _MOST + 1) <= behind:
                continue
            fewest[j] = behind
            line = ins[j]
            if line.startswith("s_waitcnt"):
                wait = _LGKM.search(line)
                if wait and int(wait.group(1)) <= behind:
                    continue
            if not line.startswith("s_"):
                if j not in registers:
                    registers[j] = set().union(*(_regs(o) for o in _operands(line)))
                if registers[j] & destination:
                    found.append((read, line))
                    break
            behind = min(_MOST, behind + line.startswith("ds_"))
            stack.extend((n, behind) for n in after[j])
    return found


def test_the_check_sees_what_it_is_for():
    read, use = "ds_read_b128 v[2:5], v1", "v_add_u32_e32 v9, 1, v4"
    assert touched_in_flight([read, use, "s_endpgm"]) == [(read, use)]
    assert not touched_in_flight([read, "s_waitcnt lgkmcnt(0)", use])
    assert touched_in_flight([read, "s_waitcnt vmcnt(0)", use])
    assert touched_in_flight([read, "s_waitcnt lgkmcnt(1)", use])
    assert not touched_in_flight([read, "ds_read_b32 v7, v1", "s_waitcnt vmcnt(3) lgkmcnt(1)", use])
    # on the path round the loop only
    assert touched_in_flight(["v_mov_b32_e32 v2, 0", ".L1:", "v_mov_b32_e32 v3, v1", read,
                              "s_cbranch_scc1 .L1", "s_waitcnt lgkmcnt(0)", "s_endpgm"])


def test_nothing_touches_the_destination_of_a_read_in_flight(assembly):  # noqa: F811
    kernels, _ = assembly
    assert sum(line.startswith("ds_read") for lines in kernels.values() for line in lines) > 1000
    bad = {name: found[:3] for name, lines in kernels.items() if (found := touched_in_flight(lines))}
    assert not bad, "\n".join(f"{n[:140]}: {f}" for n, f in bad.items())
