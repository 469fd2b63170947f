"""The index quotients of the 4-bit KV kernels (csrc/quotient.h), compiled for the
host: exact over all rows and warps that the calls accept, up to 2^31."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "drift_aware_kv_spherical_gb300", "csrc")

SOURCE = r"""
#include <cstdio>
#include "quotient.h"

int main() {
  // both ends of every range: a call's first rows, 2^24, 2^25 (the most rows),
  // 2^30, 2^31; one multiple of d and its neighbours near each
  const uint64_t near[] = {0, 1ull << 12, 1ull << 23, 1ull << 24, 1ull << 25, (1ull << 25) + 255,
                           1ull << 29, 1ull << 30, (1ull << 31) - 1};
  uint64_t x = 88172645463325252ull;
  for (uint32_t d = 1; d <= 4200; ++d) {
    const ps::Quotient q = ps::quotient(d);
    const ps::RowQuotient row = ps::row_quotient(d);
    auto check = [&](uint64_t n) {
      if (n >= (1ull << 31)) return true;
      if (q.of((uint32_t)n) != (uint32_t)n / d ||
          (n < (1u << 26) && d <= 4096 && row.of((uint32_t)n) != (uint32_t)n / d)) {
        std::printf("%llu / %u: %u\n", (unsigned long long)n, d, q.of((uint32_t)n));
        return false;
      }
      return true;
    };
    for (uint64_t n : near)
      for (int k = -2; k <= 2; ++k) {
        const uint64_t at = (n / d + k) * d;
        if (!check(at - 1) || !check(at) || !check(at + 1)) return 1;
      }
    for (int i = 0; i < 2000; ++i) {
      x ^= x << 13; x ^= x >> 7; x ^= x << 17;
      if (!check(x >> 33) || !check(x >> 38)) return 1;
    }
  }
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_quotients_are_exact(tmp_path):
    src, exe = tmp_path / "q.cpp", tmp_path / "q"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
