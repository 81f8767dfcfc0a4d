"""The attention kernels divide by numbers the host knows through a multiplication
(csrc/attn.h, Divisor): the host part compiled alone against plain division, at the quotients'
edges and up to 2^31 - 1."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

MAIN = r"""
#include <cstdint>
#include <cstdio>
#include <random>
#define __host__
#define __device__
#define __forceinline__ inline
%s
int main()
{
    std::mt19937_64 g(7);
    for (int64_t i = 0; i < 60000; ++i) {
        const uint32_t top = 2147483647u, d = i < 3000 ? i + 1 : 1 + static_cast<uint32_t>(g() %% top) / (1u << (g() %% 31));
        const Divisor by(d);
        for (int j = 0; j < 64; ++j) {
            const uint64_t edge = static_cast<uint64_t>(d) * (g() %% (top / d + 1));
            const uint64_t n64 = j == 0 ? top : j == 1 ? 0 : j %% 2 ? edge : edge + d - 1;
            const int n = static_cast<int>(n64 > top ? top : n64);
            if (by(n) != static_cast<int>(n / d) || by.rest(n) != static_cast<int>(n %% d)) {
                std::printf("%%d / %%u\n", n, d);
                return 1;
            }
        }
    }
    std::puts("ok");
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
def test_divisor(tmp_path):
    text = open(os.path.join(ROOT, "bidirectional_mamba_state_amd", "csrc", "attn.h")).read()
    struct = re.search(r"^struct Divisor \{.*?^\};", text, re.S | re.M).group(0)
    src, exe = tmp_path / "d.cc", tmp_path / "d"
    src.write_text(MAIN % struct)
    subprocess.run(["g++", "-O1", "-std=c++17", "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout
