"""The ring backward's copies of row windows stay inside the arrays they are given: a host program
walks every row of many small arrays with the rule that the kernel uses (slm_norm_rows.h)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "lm_head_loss_streaming_b200", "csrc")

# For each piece width, row width, number of rows, distance between rows, distance of the first
# row from a 16-byte boundary, and number of blocks that share a row: every whole piece lies in the
# array, and the whole pieces and the single elements together cover each column of the row once.
PROGRAM = r"""
#include <stdio.h>
#include <vector>
#include "slm_norm_rows.h"
int main() {
  long cases = 0;
  for (int elems : {4, 8})
    for (int64_t d = 1; d <= 5 * elems + 1; ++d) {
      if (!slm::norm_ring_takes(d, elems)) continue;
      for (int64_t N = 1; N <= 2 * elems + 2; ++N)
        for (int64_t ld : {d, d + elems, d + 5 * elems})
          for (int shift0 = 0; shift0 < elems; ++shift0)
            for (int blocks : {1, 2, 4}) {
              const int64_t extent = (N - 1) * ld + d;
              const int most = static_cast<int>((d + 2 * elems - 2) / elems);
              const int seg = (most + blocks - 1) / blocks;
              for (int64_t row = 0; row < N; ++row, ++cases) {
                const int shift = static_cast<int>((shift0 + row * d) % elems);
                const int nvec = static_cast<int>((d + shift + elems - 1) / elems);
                std::vector<int> seen(d, 0);
                for (int rank = 0; rank < blocks; ++rank) {
                  const int piece0 = rank * seg;
                  int mine = nvec - piece0 < seg ? nvec - piece0 : seg;
                  if (mine < 0) mine = 0;
                  const slm::NormWindow w =
                      slm::norm_window(row, N, d, shift, elems, piece0, mine);
                  if (w.lo < w.hi) {
                    const int64_t a = row * ld - shift + static_cast<int64_t>(w.lo) * elems;
                    const int64_t b = row * ld - shift + static_cast<int64_t>(w.hi) * elems;
                    if (a < 0 || b > extent) {
                      printf("elems %d d %ld N %ld ld %ld shift0 %d blocks %d row %ld: elements "
                             "%ld to %ld of %ld\n", elems, (long)d, (long)N, (long)ld, shift0,
                             blocks, (long)row, (long)a, (long)b, (long)extent);
                      return 1;
                    }
                  }
                  for (int p = piece0; p < piece0 + mine; ++p) {
                    const bool whole = p >= w.lo && p < w.hi;
                    if (!whole && p != w.lo - 1 && p != w.hi) return 2;  // not loaded at all
                    for (int e = 0; e < elems; ++e) {
                      const int64_t c = static_cast<int64_t>(p) * elems - shift + e;
                      if (c >= 0 && c < d) ++seen[c];
                    }
                  }
                }
                for (int n : seen)
                  if (n != 1) return 3;
              }
            }
    }
  printf("ok %ld\n", cases);
  return 0;
}
"""


def test_copied_windows_stay_inside_the_arrays(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "rows.cc", tmp_path / "rows"
    src.write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", "-O2", "-I", CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout
