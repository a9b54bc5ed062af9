"""The launch code's shared per-device state under two host threads (plain C++,
no GPU): a limit on dynamic shared memory that calls of different sizes raise."""
import shutil
import subprocess
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parent.parent / "sparse_top_kv_gb300" / "csrc"
PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include "hs_shared.h"

int main() {
    // A call that wants little has checked the limit and is about to set it
    // when one that wants more comes along, and the other way round.
    const int wants[2][2] = {{100, 200}, {200, 100}};
    for (auto& w : wants) {
        int known = 0;
        std::atomic<int> in_force{0};
        auto call = [&](int want, int first_ms, int set_ms) {
            std::this_thread::sleep_for(std::chrono::milliseconds(first_ms));
            const int rc = hs_host::raise_limit(&known, want, [&](int n) {
                std::this_thread::sleep_for(std::chrono::milliseconds(set_ms));
                in_force = n;
                return 0;
            });
            if (rc != 0 || in_force < want) std::printf("launch of %d with %d\n", want, int(in_force));
        };
        std::thread a(call, w[0], 0, 60), b(call, w[1], 20, 5);
        a.join();
        b.join();
        if (in_force != 200 || known != 200) std::printf("left %d, known %d\n", int(in_force), known);
        if (hs_host::raise_limit(&known, 50, [](int) { return 1; }) != 0) std::printf("lowered\n");
        if (hs_host::raise_limit(&known, 300, [](int) { return 4; }) != 4 || known != 200)
            std::printf("a failure was kept\n");
    }
    int known = 0, asked = 0;
    auto ask = [&] { ++asked; return 7; };
    if (hs_host::ask_once(&known, ask) != 7 || hs_host::ask_once(&known, ask) != 7 || asked != 1)
        std::printf("asked %d times\n", asked);
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_limits_raised_by_two_threads(tmp_path):
    (tmp_path / "t.cpp").write_text("#include <atomic>\n" + PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", f"-I{CSRC}",
                    str(tmp_path / "t.cpp"), "-o", str(tmp_path / "t")], check=True)
    res = subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and res.stdout == "", res.stdout
