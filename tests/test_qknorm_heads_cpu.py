"""The walk over heads of the norm of queries and keys, enumerated on the host:
the header that the kernel uses is compiled with g++.  For every number of heads
and every share of them, each step's heads exist and are of one tensor, and all
steps together take each head once, in order."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SRC = r"""
#include <cstdio>
#include "qknorm_heads.h"
using namespace mhla;
int main() {
  long bad = 0, steps = 0;
  for (int rows = 1; rows <= 5; ++rows)
    for (int q = 0; q <= 12; ++q)
      for (int k = 0; k <= 12; ++k)
        for (int per = 1; per <= q + k; ++per) {
          int next = 0;  // the head that has to come
          for (int part = 0; part * per < q + k; ++part) {
            const HeadShare s(part, per, q, q + k);
            for (int h = s.first; h < s.last;) {
              const int end = s.step_end(h, rows);
              ++steps;
              const bool ok = h == next && end > h && end - h <= rows && end <= q + k && end <= s.last &&
                              (h < q) == (end - 1 < q) && (h < s.split) == (h < q);
              if (!ok && ++bad < 6) std::printf("rows %d heads %d + %d per %d: %d .. %d\n", rows, q, k, per, h, end);
              h = next = end;
            }
          }
          if (next != q + k) ++bad;
        }
  std::printf("steps %ld bad %ld\n", steps, bad);
  return bad != 0;
}
"""


def test_every_fetched_head_exists_and_is_taken_once(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "heads.cpp", tmp_path / "heads"
    src.write_text(SRC)
    subprocess.run([gxx, "-O2", "-std=c++17", f"-I{ROOT}/token_level_head_phi_gb300/csrc", str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and " bad 0" in out.stdout, out.stdout
