"""What is done once a GPU (csrc/device_once.h), compiled for the host: one GPU's turn is
not another's, and threads may come together."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "drift_aware_kv_spherical_gb300", "csrc")

SOURCE = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "device_once.h"

template <int K>
ps::DeviceOnce& of() {  // as an instantiation of a launch keeps it
  static ps::DeviceOnce once;
  return once;
}

int main() {
  for (int d = -1; d < 70; ++d)
    if (of<0>().done(d)) return 1;
  of<0>().set(0);
  for (int d = -1; d < 70; ++d)
    if (of<0>().done(d) != (d == 0) || of<1>().done(d)) return 2;
  of<0>().set(63);
  of<0>().set(64);   // beyond what is kept: done again every time
  of<0>().set(-1);
  for (int d = -1; d < 70; ++d)
    if (of<0>().done(d) != (d == 0 || d == 63)) return 3;
  std::vector<std::thread> all;
  for (int d = 0; d < 64; ++d)
    all.emplace_back([d] {
      for (int i = 0; i < 1000; ++i) of<2>().set(d);
    });
  for (auto& t : all) t.join();
  for (int d = 0; d < 64; ++d)
    if (!of<2>().done(d)) return 4;
  std::puts("ok");
}
"""


def test_a_gpu_is_not_another(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src = tmp_path / "once.cpp"
    src.write_text(SOURCE)
    exe = tmp_path / "once"
    subprocess.run([gxx, "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "ok\n", r.returncode


def test_no_launch_keeps_a_limit_of_its_own():
    """Every kernel's limit of shared memory that is kept is kept by GPU."""
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            src = open(os.path.join(CSRC, name)).read()
            assert "static bool" not in src, name
