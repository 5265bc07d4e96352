"""How lengths are cut into partitions (csrc/pkd_split.h), compiled for the host: right for every 32-bit length."""
import os
import shutil
import subprocess

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_decode_21_gb300", "csrc")

PROGRAM = r"""
#include <climits>
#include <cstdio>
#include "pkd_split.h"
int main() {
  const int lens[] = {INT_MIN, -70000, -1, 0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1023, 8192, 8193, 1 << 30,
                      (1 << 30) + 1, INT_MAX - 8192, INT_MAX - 127, INT_MAX - 126, INT_MAX - 1, INT_MAX};
  const int parts[] = {1, 16, 32, 64, 128, 512, 8192, 1 << 30, INT_MAX};
  const int grids[] = {1, 2, 7, 4096, INT_MAX};
  for (int L : lens) {
    for (int P : parts)
      for (int np : grids) {
        const long long n = L > 0 ? ((long long)L + P - 1) / P : 0, want = n < np ? n : np;
        if (pkd::partitions_of(L, P, np) != want) { std::printf("%d %d %d\n", L, P, np); return 1; }
      }
    if (L < 0) continue;
    const long long half = ((long long)L + 1) / 2;
    if (pkd::half_up(L) != half || pkd::tail_half_partition(L) != (half + 63) / 64 * 64) {
      std::printf("half of %d\n", L);
      return 1;
    }
  }
  return 0;
}
"""


def test_partitions_of_any_length(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    src, exe = tmp_path / "split.cc", tmp_path / "split"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover",
                    "-I", SRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr

