"""The compiled code of the cross entropy's kernels (no GPU): the direct-to-LDS
lint of test_asm_lint_cpu.py, no spilled vector register, no scratch, no packed
fp32 instruction, and no atomic (their results depend on no order)."""
import os
import re
import subprocess

import pytest

from test_asm_lint_cpu import HIPCC, ROOT, lint
from test_asm_lint_i8_cpu import kernels


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = str(tmp_path_factory.mktemp("asm") / "xent.s")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "dense_gemm_swizzled_amd", "csrc"), "--cuda-device-only",
           "-S", os.path.join(ROOT, "tests", "asm", "xent_kernels.hip"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    with open(out) as f:
        return f.read()


def test_kernels_keep_their_m0(listing):
    found = {n: b for n, b in kernels(listing) if "kernel" in n}
    products = {n: b for n, b in found.items()
                if re.search(r"pingpong|deep|dense|split", n)}
    # stats and gradient, two types: ping-pong (K exact, any K), deep 64 and 128,
    # dense; the splits on three tiles; four products of any K
    assert len(products) == 20 + 6 + 4, sorted(products)
    for name, body in products.items():
        bad, n = lint(body)
        # (the two-stage kernel loads through builtins, whose m0 is the compiler's)
        if "xent_dense_kernel" in name:
            assert n > 0
            continue
        assert n > 0, f"{name}: no direct-to-LDS loads found"
        assert not bad, f"{name}: {bad[:5]}"


def test_joined_kernels_keep_their_m0(listing):
    """Products whose launch does something else as well."""
    found = {n: b for n, b in kernels(listing) if re.search(r"xent_(head|twin|few)_kernel", n)}
    assert len(found) == 6, sorted(found)
    for name, body in found.items():
        bad, n = lint(body)
        assert n > 0 and not bad, f"{name}: {n} loads, {bad[:5]}"


def test_no_kernel_spills(listing):
    spills = re.findall(r"\.vgpr_spill_count:\s*(\d+)", listing)
    assert len(spills) >= 30 and set(spills) == {"0"}
    assert set(re.findall(r"\.private_segment_fixed_size:\s*(\d+)", listing)) == {"0"}


def test_no_packed_fp32_and_no_atomics(listing):
    assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", listing)
    assert not re.search(r"\b(global|flat|buffer)_atomic", listing)
