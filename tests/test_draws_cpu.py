"""Work items drawn by workgroups (csrc/draws.hpp), compiled for the host and run by
threads: whatever the words hold before, every item is run by exactly one workgroup of its
XCD, and the words are zero behind the call, so that a replay with the same tag starts
anew."""
from __future__ import annotations

import os
import subprocess

from gated_mlp_gemm_amd import build
from test_arrivals_cpu import STUB

MAIN = r"""
#include "draws.hpp"
#include <cstdio>
#include <random>
#include <thread>
#include <vector>

static bool call(uint64_t *words, uint64_t tag, int workgroups, int total, std::mt19937 &g) {
    std::vector<int> ran(total, 0), by(total, -1);
    std::vector<unsigned> slow(workgroups);
    for (auto &s : slow) s = g() % 40;
    std::vector<std::thread> threads;
    for (int b = 0; b < workgroups; ++b)
        threads.emplace_back([&, b] {
            int item = b;
            if (item >= total) return;
            swiglu::Draws d;
            d.begin(words, tag, b, workgroups, total, true);
            int ahead = b + workgroups;
            while (item < total) {
                const unsigned ticket = d.ask();
                __atomic_fetch_add(&ran[item], 1, __ATOMIC_RELAXED);
                by[item] = b;
                for (unsigned n = 0; n < slow[b]; ++n) std::this_thread::yield();
                d.answered(ticket);
                item = ahead;
                ahead = d.item(ticket);
            }
        });
    for (auto &t : threads) t.join();
    for (int i = 0; i < total; ++i)
        if (ran[i] != 1 || by[i] % 8 != i % 8) return false;
    const int used = workgroups < total ? workgroups : total;
    for (int x = 0; x < 8 && x < used; ++x)
        if (words[x] != 0) return false;
    return true;
}

int main() {
    std::mt19937 g(7);
    uint64_t tag = uint64_t{0x1234567} << swiglu::kArrivalBits;
    int calls = 0;
    for (int workgroups : {8, 16, 24})
        for (int total : {1, 3, 7, 8, 9, 15, 16, 17, 31, 32, 33, 47, 48, 49, 100, 777}) {
            std::vector<uint64_t> words(8);
            for (auto &w : words) w = (uint64_t{g()} << 32) | g();
            tag += uint64_t{1} << swiglu::kArrivalBits;
            // a call on whatever is there, replays with the same tag, a call with another
            for (int k = 0; k < 3; ++k, ++calls)
                if (!call(words.data(), tag, workgroups, total, g)) {
                    std::printf("workgroups %d items %d call %d\n", workgroups, total, k);
                    return 1;
                }
        }
    std::printf("%d calls\n", calls);
    return 0;
}
"""


def test_every_item_once_and_the_words_cleared(tmp_path):
    (tmp_path / "hip").mkdir()
    (tmp_path / "hip" / "hip_runtime.h").write_text(STUB)
    (tmp_path / "main.cpp").write_text(MAIN)
    exe = str(tmp_path / "draws")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", str(tmp_path), "-I", build.CSRC,
                    str(tmp_path / "main.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], stdout=subprocess.PIPE, timeout=300, text=True)
    assert out.returncode == 0 and "144 calls" in out.stdout, out.stdout
    assert os.path.exists(exe)
