"""The compiled code of the 8-bit kernels (no GPU), every instantiation that
the library launches."""
import os
import re
import subprocess

import pytest

from test_asm_lint_cpu import HIPCC, ROOT
from test_asm_lint_i8_cpu import kernels


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = str(tmp_path_factory.mktemp("asm") / "i8.s")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-I", os.path.join(ROOT, "include"), "--cuda-device-only", "-S",
           os.path.join(ROOT, "tests", "asm", "i8_all_kernels.hip"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    with open(out) as f:
        return f.read()


def test_stores_past_the_caches(listing):
    """Only a grouped product's 16-bit D of 256x256 tiles is stored past the
    caches: 16 stores for each of the two types.  fp32 rows are written in
    parts of lines, and a dense D is read next."""
    found = {n: b for n, b in kernels(listing) if "i8_pingpong_kernel" in n}
    assert len(found) == 3, sorted(found)
    for name, body in found.items():
        stores = [t for t in map(str.strip, body) if re.match(r"(global|flat|buffer)_store", t)]
        past = [t for t in stores if re.search(r"\bnt\b", t)]
        assert stores
        if re.search(r"kernelILb1E", name):               # grouped
            assert len(past) == 32 and all("dwordx4" in t for t in past), (name, len(past))
        else:
            assert not past, (name, past[:3])
