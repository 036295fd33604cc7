"""The pieces of a contraction split along K (csrc/pieces.hpp), compiled for the host: for
every number of pieces that a launch takes they begin at 0, follow each other, end at the
contraction's last step and are as long as each other but for one step, up to the 2^24 steps
of a weight's gradient over 2^30 rows.  The helper's products are watched for overflow."""
from __future__ import annotations

import os
import re
import subprocess

from gated_mlp_gemm_amd import build

STUB = """
#pragma once
#define __device__
#define __forceinline__ inline
"""

MAIN = r"""
#include "pieces.hpp"
#include <cstdint>
#include <cstdio>

int main() {
    long checked = 0;
    const int steps[] = {1, 2, 3, 31, 511, 512, 513, 1000, 32768, 32767, (1 << 22) - 1, 1 << 22,
                         (1 << 22) + 1, (1 << 23) + 5, (1 << 24) - 511, (1 << 24) - 1, 1 << 24};
    for (int nk : steps)
        for (int pieces = 1; pieces <= 1024 && pieces <= nk; ++pieces, ++checked) {
            int at = 0;
            for (int p = 0; p < pieces; ++p) {
                const int kb = swiglu::piece_begin(p, nk, pieces);
                const int ke = swiglu::piece_begin(p + 1, nk, pieces);
                const int64_t want = int64_t{p} * nk / pieces;
                const int len = ke - kb;
                if (kb != at || kb != want || len < nk / pieces || len > nk / pieces + 1) {
                    std::printf("nk %d pieces %d piece %d: [%d, %d)\n", nk, pieces, p, kb, ke);
                    return 1;
                }
                at = ke;
            }
            if (at != nk) {
                std::printf("nk %d pieces %d end at %d\n", nk, pieces, at);
                return 1;
            }
        }
    std::printf("%ld schedules\n", checked);
    return 0;
}
"""


def test_pieces_cover_the_contraction(tmp_path):
    (tmp_path / "hip").mkdir()
    (tmp_path / "hip" / "hip_runtime.h").write_text(STUB)
    (tmp_path / "main.cpp").write_text(MAIN)
    exe = str(tmp_path / "pieces")
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-I", str(tmp_path), "-I",
                    build.CSRC, str(tmp_path / "main.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=300,
                         text=True)
    assert out.returncode == 0 and "schedules" in out.stdout, out.stdout


def test_no_kernel_multiplies_pieces_by_steps():
    """Every split's bounds come from the helper."""
    for name in sorted(os.listdir(build.CSRC)):
        with open(os.path.join(build.CSRC, name), encoding="utf-8") as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        found = re.findall(r"\*\s*(?:\w+\.)?nk\s*/\s*[\w.]+", code)
        assert not found, (name, found)
