"""The rotary embedding's rates, from the header that the library takes them
from, compiled with the host compiler, against 60-digit arithmetic: each within
6 units of 2^-64 of a turn a position, which with the fraction's own rounding
keeps an angle within 2^-30 of a turn at every int32 position."""
import os
import shutil
import subprocess
from decimal import Decimal, getcontext

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "rope_rates.h"
#include <cinttypes>
#include <cstdio>
#include <cstdlib>
int main(int argc, char **argv) {
  uint64_t freq[256];
  uint8_t axis[256];
  for (int a = 1; a + 1 < argc; a += 2) {
    const int dims[3] = {0, atoi(argv[a + 1]), 8};
    oq::rope_rates(atof(argv[a]), 3, dims, freq, axis);
    for (int j = 0; j < dims[1] / 2; j++) std::printf("%" PRIu64 " %d ", freq[j], axis[j]);
    std::printf("%d\n", axis[dims[1] / 2]);
  }
}
"""


def test_rates(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "rates.cpp", tmp_path / "rates"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "quantization_dit_linear_amd", "csrc")
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-I", csrc, str(src), "-o", str(exe)], check=True)
    cases = [(t, d) for t in (1.0, 1.001, 1.5, 2.0, 100.0, 500.0, 10000.0, 1e6, 1e12)
             for d in (2, 16, 20, 42, 44, 56, 64, 96, 128, 200, 256, 504)]
    out = subprocess.run([str(exe), *(str(v) for c in cases for v in c)], capture_output=True, text=True,
                         check=True, timeout=60).stdout.splitlines()
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    worst = 0
    for (theta, d), line in zip(cases, out, strict=True):
        v = [int(n) for n in line.split()]
        assert len(v) == d + 1 and v[-1] == 2 and set(v[1:-1:2]) == {1}
        log = Decimal(theta).ln()
        for i in range(d // 2):
            want = (-2 * i * log / d).exp() / (2 * pi) * 2 ** 64
            worst = max(worst, abs(v[2 * i] - want))
    assert worst <= 6, worst
    assert worst * 2 ** 31 / 2 ** 64 + Decimal(2) ** -33 <= Decimal(2) ** -30
