"""The few-row kernel's launches (csrc/mx_few_plan.hpp), on the host: a launch has less than 2^32 threads along a
dimension, and with more it would run on what is left of them modulo 2^32."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "mx_few_plan.hpp"
using namespace q4;
int main() {
    const int64_t top = int64_t(1) << 25, cus[] = {1, 32, 64, 80, 256, 304}, Ks[] = {32, 544, 4096, 8224, 14368, 16384, top};
    long seen = 0, bad = 0;
    for (int64_t c : cus)
        for (int64_t K : Ks)
            for (int64_t M : {1, 4, 5, 16, 33, 64, 65, 128, 700})
                for (int nmat = 1; nmat <= 2; nmat++)
                    for (int x = 0; x < 3; x++) {
                        auto look = [&](int64_t N) {
                            if (N < 1 || N > top || !few_takes(x, nmat, M, N, K, c)) return;
                            const MxFewPlan p = plan_few(nmat, M, N, K, c);
                            seen++;
                            const bool whole = p.r >= 1 && p.r <= 3 && p.kw >= 1 && p.rw >= 1 && p.kw * p.rw <= 8;
                            const bool covers = few_columns(p, M, N) * p.rw * p.r * (M <= 4 ? 4 : 16) >= N;
                            if (!whole || !covers || few_columns(p, M, N) * few_threads(p) >= int64_t(1) << 32 || few_chunks(M) > 65535) bad++;
                        };
                        for (int64_t N : {int64_t(1), int64_t(4095), int64_t(12288)}) look(N);
                        for (int64_t d = 0; d < 4000; d += 3) look(top - d);
                        for (int64_t d = 0; d < 64; d++) look(top - d * 4 * c), look(top - d * 16 * c);
                    }
    std::printf("%ld %ld\n", seen, bad);
    return 0;
}
"""


def test_every_launch_fits(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", os.path.join(ROOT, "gemv_q4_affine_amd", "csrc"), str(src),
                    "-o", str(exe)], check=True)
    seen, bad = map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True, timeout=60).stdout.split())
    assert seen > 100000 and bad == 0
