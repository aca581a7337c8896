"""A device's value is made once, whichever threads ask for it first (csrc/hs_once.h)."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hierarchical_kv_cache_swap_gb300", "csrc")

PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>
#include "hs_once.h"

struct Value { int a, b; };

int main() {
    hs::PerDevice<Value> values;
    std::atomic<int> made{0}, wrong{0}, waiting{0};
    const int n = 16;
    std::vector<std::thread> threads;
    for (int i = 0; i < n; ++i)
        threads.emplace_back([&, i] {
            ++waiting;
            while (waiting < n) std::this_thread::yield();  // all of them ask at once
            const Value* v = nullptr;
            const int rc = values.get(i % 2, [&](Value* to) {
                ++made;
                to->a = 7;
                std::this_thread::sleep_for(std::chrono::milliseconds(50));
                to->b = 8;
                return 0;
            }, &v);
            if (rc != 0 || !v || v->a != 7 || v->b != 8) ++wrong;
        });
    for (auto& t : threads) t.join();
    const Value* v = nullptr;
    const int failed = values.get(5, [](Value*) { return 3; }, &v);  // an error is not kept
    const int again = values.get(5, [](Value* to) { *to = Value{1, 2}; return 0; }, &v);
    std::printf("%d %d %d %d %d\n", made.load(), wrong.load(), failed, again, v ? v->b : -1);
}
"""


def test_made_once(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("g++")
    (tmp_path / "once.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "once")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-pthread", "-I", CSRC, str(tmp_path / "once.cpp"), "-o", exe])
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.stdout.split() == ["2", "0", "3", "0", "2"], out
