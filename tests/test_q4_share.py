"""The closed form of what a request's row tiles are charged (attend_q4.cuh) against the tiles' charges one by one: host code
of the kernels' header, compiled with nvcc.  CPU only."""
import os
import subprocess

from block_sparse_attention_pbsa_b200 import build

CODE = r"""
#include <stdio.h>
#include "attend_q4.cuh"
using namespace pbsa;
int main() {
  const int rows[] = {8, 16, 256};
  for (int num : rows)
    for (int group = 1; group <= 200; ++group)
      for (int base = 3; base < 40; base += 17) {
        Q4Request x = {};
        x.base = base;
        x.num = num;
        x.den = BT * group;
        long long sum = 0;
        for (int n = 0; n <= 700; ++n) {
          if (x.charged_to(n) != sum) { printf("rows %d group %d: %lld, not %lld, up to tile %d\n", num, group, x.charged_to(n), sum, n); return 1; }
          const long long c = base + ((long long)num * (n + 1) + x.den - 1) / x.den;
          if (x.charge(n) != c) { printf("rows %d group %d: charge of tile %d\n", num, group, n); return 1; }
          sum += c;
        }
      }
  // the most rows that a call takes, 2^30: nothing passes its type
  for (int group = 1; group <= 4096; ++group) {
    Q4Request x = {};
    x.base = 1 << 25;
    x.num = 256;
    x.den = BT * group;
    const int n = (1 << 30) / 256;
    if (x.charged_to(n) - x.charged_to(n - 1) != x.charge(n - 1)) { printf("group %d at 2^30 rows\n", group); return 1; }
  }
  return 0;
}
"""


def test_charges_add_up(tmp_path):
    src, exe = tmp_path / "share.cu", tmp_path / "share"
    src.write_text(CODE)
    r = subprocess.run([build.nvcc(), *build.ARCH, "-O1", "-std=c++17", f"-I{os.path.join(build.ROOT, 'include')}", f"-I{build.CSRC}", "-o",
                        str(exe), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
