"""Sizes at the end of their type, on the host: a workspace size, or a refusal, and
never a division by an overflowed product."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MOST = (1 << 31) - 1

SIZES = [dict(B=1, N=100, Hq=2, Hkv=1, dh=128, P=MOST),     # P Hq / Hkv = -2 as an int
         dict(B=1, N=100, Hq=4, Hkv=1, dh=128, P=1 << 30),  # 0
         dict(B=65535, N=100, Hq=MOST, Hkv=1, dh=64, P=MOST),
         dict(B=MOST, N=MOST, Hq=MOST, Hkv=MOST, dh=256, P=MOST),
         dict(B=1 << 16, N=1, Hq=1 << 24, Hkv=1 << 10, dh=64, P=1 << 24),   # B P Hq = 0 as a long
         dict(B=1, N=MOST, Hq=1, Hkv=1, dh=64, P=1)]


@pytest.mark.parametrize("sizes", SIZES)
def test_workspace_of_sizes_that_no_call_takes(sizes):
    code = ("from drift_aware_kv_spherical_gb300 import _build, polestar as ps\n"
            "import os\n"
            "os.path.exists(ps.LIB_PATH) or _build.build()\n"
            f"print([ps.ps_workspace_bytes(op, **{sizes!r})"
            " for op in (ps.OP_KV4_ATTN, ps.OP_KV4_WEIGHT)])\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])   # a division by 0 ends the process
    assert r.stdout.strip() == "[0, 0]"
