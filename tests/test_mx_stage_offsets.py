"""Where the MX tile kernel's requests go, checked on the host: the header that
the kernel takes its offsets from, compiled with the host compiler, and every
request of every stage of full and of ragged tiles followed.  A request for a
valid row's piece has to lie inside the buffer, at that piece; every other one
(rows past the last, pieces past K, stages past the last) past its end."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "mx_stage.h"
#include <cstdio>
#include <vector>

// a tile of `rows` rows, `valid` of them inside the matrix, rows of rowb bytes
template <int RB, int TH>
int check(int rows, int valid, int rowb) {
  using P = oq::MxPieces<RB, TH>;
  const int stages = (rowb + RB - 1) / RB, rounds = rows * P::C / TH;
  if (rows * P::C % TH != 0) return 1;
  for (int t = 0; t < stages + 3; t++) {
    std::vector<int> seen(valid * P::C, 0);
    for (int k = 0; k < rounds; k++)
      for (int tid = 0; tid < TH; tid++) {
        const int row = P::row(tid) + k * P::ROWS, col = t * RB + P::byte(tid);
        const uint32_t at = P::row(tid) * rowb + P::byte(tid);
        const uint64_t off = P::offset(at, P::byte(tid), rowb, t), size = P::size(valid, rowb, k);
        if (P::base(rowb, k) + size > (uint64_t)valid * rowb && size) return 5;
        if (row < valid && col < rowb) {
          if (P::base(rowb, k) + off != (uint64_t)row * rowb + col || off + 16 > size) return 2;
        } else if (off < size || off + 16 > 0xffffffffull) {
          return 3;
        }
        if (row < valid) seen[row * P::C + P::byte(tid) / 16]++;
      }
    for (int n : seen)
      if (n != 1) return 4;
  }
  return 0;
}

template <int RB, int TH>
int all(int rows) {
  for (int valid : {1, 2, 31, 32, 33, 63, 64, 65, 84, 127, 128, 129, 200, 255, 256})
    for (int rowb : {16, 32, 48, 64, 80, 112, 128, 144, 240, 256, 272, 1296, 2560, 8192, 16384}) {
      if (valid > rows) continue;
      const int rc = check<RB, TH>(rows, valid, rowb);
      if (rc) {
        std::printf("RB %d TH %d rows %d valid %d row bytes %d: %d\n", RB, TH, rows, valid, rowb, rc);
        return rc;
      }
    }
  return 0;
}

int main() {
  // 64 and 128 tiles: 256 threads; 256 tiles: 512
  return all<128, 256>(64) || all<64, 256>(64) || all<128, 256>(128) || all<64, 256>(128) ||
         all<128, 512>(256) || all<64, 512>(256);
}
"""


def test_requests_stay_inside_their_rows(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "offsets.cpp", tmp_path / "offsets"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "quantization_dit_linear_amd", "csrc")
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-I", csrc, str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stdout
