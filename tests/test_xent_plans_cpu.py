"""The plan of the cross entropy's gradient on the host (no GPU):
tests/plans/xent_plans.cpp."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
def test_plans(tmp_path):
    exe = str(tmp_path / "xent_plans")
    r = subprocess.run(
        [HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-x", "hip",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(ROOT, "include"),
         os.path.join(ROOT, "tests", "plans", "xent_plans.cpp"), "-o", exe],
        capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
