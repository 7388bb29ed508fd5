"""csrc/wave_exchange.hpp on the host: one thread a wave, a std::barrier as the
workgroup's, and in every call another wave held back between the barrier and its
reads, so that the others are as far ahead as their barriers let them.  Every
wave must get the sums of every call, whatever a row's number of calls."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <barrier>
#include <chrono>
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>
#define __device__
#define __forceinline__ inline
#include "wave_exchange.hpp"

int main(int argc, char** argv) {
    const int waves = std::atoi(argv[1]), calls = std::atoi(argv[2]);
    static float red[2][q4::kMaxWaves][2];
    std::barrier<> bar(waves);
    std::vector<int> bad(waves, 0);
    std::vector<std::thread> ts;
    for (int wave = 0; wave < waves; wave++)
        ts.emplace_back([&, wave] {
            int turn = 0;
            for (int c = 0; c < calls; c++) {
                float a = float(100 * c + wave), b = float(wave * (c + 1));
                q4::wave_sums(a, b, wave, waves, true, red, turn, [&] {
                    bar.arrive_and_wait();
                    if (c % waves == wave) std::this_thread::sleep_for(std::chrono::milliseconds(3));
                });
                const int below = waves * (waves - 1) / 2;
                if (a != float(100 * c * waves + below) || b != float(below * (c + 1))) bad[wave]++;
            }
        });
    for (auto& t : ts) t.join();
    int total = 0;
    for (int n : bad) total += n;
    std::printf("%d\n", total);
    return 0;
}
"""


@pytest.mark.parametrize("waves", [2, 3, 8])
def test_a_slow_wave_reads_its_own_call(tmp_path, waves):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "exchange.cpp", tmp_path / "exchange"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++20", "-O1", "-pthread", "-I", os.path.join(ROOT, "gemv_q4_affine_amd", "csrc"), str(src),
                    "-o", str(exe)], check=True)
    out = subprocess.run([str(exe), str(waves), "40"], capture_output=True, text=True, check=True, timeout=60).stdout
    assert int(out) == 0, f"{out.strip()} sums of a call held another call's values"
