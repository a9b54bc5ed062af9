"""Integer arithmetic of how calls are cut into work, on the host (plain C++)."""
import shutil
import subprocess
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parent.parent / "sparse_top_kv_gb300" / "csrc"


def run(tmp_path, body):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "t.cpp").write_text('#include <algorithm>\n#include <cstdio>\n#include "hs_plan.h"\n' + body)
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


def test_places_of_blocks_add_up(tmp_path):
    """The closed form is the sum of the blocks', and a block's is what it sees."""
    run(tmp_path, r"""
int main() {
    for (int held : {0, 1, 63, 64, 65, 500, 1000, 70000})
        for (int n : {0, 1, 63, 64, 65, 500, 5000})
            for (int tb : {1, 3, 64, 256})
                for (int window : {0, 1, 64, 200, 5000, 1 << 30})
                    for (int extra : {0, 256, 512}) {
                        const hs_plan::Request x = hs_plan::request(0, n, held, n, 1 << 30);
                        int64_t sum = 0;
                        for (int b = 0; b * tb < x.n; ++b) {
                            if (hs_plan::places_of_blocks(x, tb, window, extra, b) != sum)
                                std::printf("held %d n %d tb %d window %d: %d blocks\n", held, n, tb, window, b);
                            const int64_t p = x.T - x.n + int64_t(b) * tb;
                            const int64_t from = window > 0 ? std::max<int64_t>(0, p + 1 - window) : 0;
                            const int own = hs_plan::places_of_block(x, tb, window, extra, b);
                            if (p < 0 || own <= 0 || own != extra + p + tb - from)
                                std::printf("held %d n %d tb %d window %d: block %d is %d\n", held, n, tb, window, b, own);
                            sum += own;
                        }
                        if (hs_plan::places_of_blocks(x, tb, window, extra, (x.n + tb - 1) / tb) != sum)
                            std::printf("held %d n %d tb %d window %d: all\n", held, n, tb, window);
                    }
    // The largest: 2^24 new tokens over 2^30.
    const hs_plan::Request far = hs_plan::request(0, 1 << 24, 1 << 30, 1 << 24, 1 << 30);
    if (hs_plan::places_of_blocks(far, 1, 1 << 29, 512, 1 << 24) != (int64_t(512) + (1 << 29)) << 24)
        std::printf("the largest\n");
}
""")


def test_queries_that_attend_to_nothing_are_no_work(tmp_path):
    """Rows stay inside, each request's are those of its cu_new, and queries before
    position 0 are apart from the rest.  (A refused prompt of 8192 tokens, counted as if
    it saw itself, had two thirds of the GPU beside 64 single tokens over 4096.)"""
    run(tmp_path, r"""
int main() {
    const int tokens = 100, max_len = 300, ends[] = {-(1 << 30), -1, 0, 1, 5, 60, 99, 100, 101, 1 << 30};
    for (int c0 : ends)
        for (int c1 : ends)
            for (int held : {-(1 << 30), -1, 0, 1, 4, 55, 60, 299, 300, 301, 1 << 30}) {
                const hs_plan::Request x = hs_plan::request(c0, c1, held, tokens, max_len);
                const int first = std::clamp(c0, 0, tokens), n = std::max(0, std::clamp(c1, 0, tokens) - first);
                const int T = std::clamp(held, 0, max_len), blind = std::max(0, n - T);
                if (x.T != T || x.blind != blind || x.n != n - blind || x.first != first + blind)
                    std::printf("%d %d %d: %d %d %d %d\n", c0, c1, held, x.first, x.n, x.T, x.blind);
            }
    if (hs_plan::request(0, 8192, 0, 8192, 8192).n != 0) std::printf("refused\n");
}
""")
