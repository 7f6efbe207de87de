"""The direct-to-LDS lint of test_asm_lint_cpu.py over the 8-bit kernels (no
GPU): every such load follows an m0 write with an instruction between them,
and no m0 write comes from outside inline assembly.  None of the kernels
spills a vector register."""
import os
import re
import subprocess

import pytest

from test_asm_lint_cpu import HIPCC, ROOT, lint


def kernels(text):
    """(kernel symbol, [lines]) up to the function's end: a workgroup with no
    tile leaves early, so a body has more than one s_endpgm."""
    for m in re.finditer(r"^(_Z\S*):(.*?)^\.Lfunc_end\d+:", text, flags=re.S | re.M):
        yield m.group(1), m.group(2).splitlines()


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
def test_i8_kernels_keep_their_m0(tmp_path):
    out = str(tmp_path / "i8.s")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-I", os.path.join(ROOT, "include"), "--cuda-device-only", "-S",
           os.path.join(ROOT, "tests", "asm", "i8_dma_kernels.hip"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    with open(out) as f:
        text = f.read()
    found = dict(kernels(text))
    assert len(found) == 5, sorted(found)
    for name, body in found.items():
        bad, n = lint(body)
        assert n > 0, f"{name}: no direct-to-LDS loads found"
        assert not bad, f"{name}: {bad[:5]}"
    spills = re.findall(r"\.vgpr_spill_count:\s*(\d+)", text)
    assert len(spills) == 5 and set(spills) == {"0"}
