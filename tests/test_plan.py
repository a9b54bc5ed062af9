"""Integer arithmetic of how calls are cut into work, on the host (plain C++)."""
import shutil
import subprocess
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parent.parent / "sparse_top_kv_gb300" / "csrc"


def run(tmp_path, body):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "t.cpp").write_text('#include <cstdio>\n#include "hs_plan.h"\n' + body)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror",
                    "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover=all",
                    f"-I{CSRC}", str(tmp_path / "t.cpp"), "-o", str(tmp_path / "t")], check=True)
    res = subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0 and res.stdout == "", res.stdout + res.stderr


def test_sums_saturate(tmp_path):
    run(tmp_path, r"""
int main() {
    using hs_plan::kSatMax;
    using hs_plan::sat_add;
    const int v[] = {0, 1, 5, 1 << 26, 1 << 29, (1 << 29) + 1, (1 << 30) - 1, 1 << 30, kSatMax};
    for (int a : v)
        for (int b : v) {
            const int64_t exact = int64_t(a) + b;
            const int want = exact < kSatMax ? int(exact) : kSatMax;
            if (sat_add(a, b) != want) std::printf("%d + %d: %d\n", a, b, sat_add(a, b));
            for (int c : v)
                if (sat_add(sat_add(a, b), c) != sat_add(a, sat_add(b, c)))
                    std::printf("%d + %d + %d depends on the order\n", a, b, c);
        }
}
""")
