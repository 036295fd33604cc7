"""The counting of arrivals in a workspace word (csrc/arrivals.hpp), compiled for the host
and run by threads: whatever the word holds before, exactly one of a call's workgroups is
the last, it sees what the others stored, and it leaves zero for a replay with the same
tag."""
from __future__ import annotations

import os
import subprocess

from gated_mlp_gemm_amd import build

STUB = """
#pragma once
#define __device__
#define __forceinline__ inline
#define __HIP_MEMORY_SCOPE_AGENT 0
#define __hip_atomic_compare_exchange_strong(p, e, d, s, f, scope) \\
    __atomic_compare_exchange_n(p, e, d, false, __ATOMIC_ACQ_REL, __ATOMIC_ACQUIRE)
#define __hip_atomic_fetch_add(p, v, order, scope) __atomic_fetch_add(p, v, __ATOMIC_ACQ_REL)
#define __hip_atomic_store(p, v, order, scope) __atomic_store_n(p, v, __ATOMIC_RELEASE)
"""

MAIN = r"""
#include "arrivals.hpp"
#include <cstdio>
#include <random>
#include <thread>
#include <vector>

// One call of n workgroups: how many were the last, and whether the last saw all stores.
static bool call(uint64_t *word, uint64_t tag, int n, std::mt19937 &g) {
    std::vector<int> stored(n, 0);
    std::vector<unsigned> before(n, 0);
    std::vector<int> saw(n, -1), pause(n);
    for (int &p : pause) p = g() % 3;
    std::vector<std::thread> threads;
    for (int i = 0; i < n; ++i)
        threads.emplace_back([&, i] {
            swiglu::Arrival meeting{};
            if (pause[i] == 1) std::this_thread::yield();
            meeting.announce(word, tag);
            if (pause[i] == 2) std::this_thread::yield();
            meeting.settle(word, tag);
            stored[i] = i + 1;
            before[i] = swiglu::arrive(word);
            if (before[i] + 1 != static_cast<unsigned>(n)) return;
            swiglu::arrivals_done(word);
            int sum = 0;
            for (int s : stored) sum += s;
            saw[i] = sum;
        });
    for (auto &t : threads) t.join();
    int lasts = 0;
    std::vector<int> seen(n, 0);
    for (int i = 0; i < n; ++i) {
        if (before[i] >= static_cast<unsigned>(n)) return false;
        seen[before[i]]++;
        lasts += before[i] + 1 == static_cast<unsigned>(n);
        if (saw[i] >= 0 && saw[i] != n * (n + 1) / 2) return false;
    }
    for (int s : seen) if (s != 1) return false;
    return lasts == 1 && *word == 0;
}

int main() {
    std::mt19937 g(7);
    const uint64_t step = 0x9E3779B97F4A7C15u;
    uint64_t next = 12345;
    for (int round = 0; round < 1500; ++round) {
        const uint64_t tag = next << swiglu::kArrivalBits;
        const uint64_t older = (next - step) << swiglu::kArrivalBits;
        next += step;
        const uint64_t held[] = {0, ~uint64_t{0}, 1, older, older + 3, tag ^ (uint64_t{1} << 63),
                                 tag + (uint64_t{1} << swiglu::kArrivalBits), g(),
                                 (static_cast<uint64_t>(g()) << 32) | g()};
        uint64_t word = held[round % 9];
        const int n = 2 + g() % 7;
        for (int replay = 0; replay < 3; ++replay)
            if (!call(&word, tag, n, g)) {
                std::printf("round %d replay %d n %d\n", round, replay, n);
                return 1;
            }
    }
    return 0;
}
"""


def test_one_workgroup_is_the_last_whatever_the_word_holds(tmp_path):
    os.makedirs(tmp_path / "hip")
    (tmp_path / "hip" / "hip_runtime.h").write_text(STUB)
    (tmp_path / "main.cpp").write_text(MAIN)
    exe = str(tmp_path / "arrivals")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", str(tmp_path), "-I", build.CSRC,
                    str(tmp_path / "main.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout
