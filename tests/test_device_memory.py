"""What device memory the library holds (CPU: hipcc cross-compiles).

Calls that run at the same time, on different streams or as a captured graph
replayed beside eager calls, share nothing but what the library itself holds.  So
the only device variable in its code is the scratch of the call that documents it as
shared (swiglu_fused_gemm_noalloc); the words at which workgroups of one launch meet
lie in the caller's workspace."""
from __future__ import annotations

import os
import re

from gated_mlp_gemm_amd import build


def test_the_only_device_variable_is_the_noalloc_scratch(tmp_path):
    with open(build.device_assembly(os.path.join(tmp_path, "kernels.s"))) as f:
        names = set(re.findall(r"\.type\s+(\w+),@object", f.read()))
    names = {n for n in names if not n.startswith("__hip_cuid")}
    assert len(names) == 1 and "scratch" in names.pop(), names
