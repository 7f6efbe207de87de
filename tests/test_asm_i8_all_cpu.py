"""The compiled code of the 8-bit kernels (no GPU), every instantiation that
the library launches."""
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


def library_kernels():
    """The 8-bit kernels of the built library: the launch stubs of its objects."""
    from dense_gemm_swizzled_amd import _build
    obj = os.path.join(_build.BUILD, "launch_i8.o")
    if not os.path.exists(obj):
        pytest.skip("the library's objects are not here")
    names = subprocess.run(["nm", obj], capture_output=True, text=True, check=True).stdout
    return set(re.findall(r"__device_stub__(i8_\w+_kernelI\w+?E)EvNS_8I8ParamsE", names))


def test_every_kernel_of_the_library_is_here(listing):
    here = {re.search(r"(i8_\w+_kernelI\w+?E)EvNS_8I8ParamsE", n).group(1)
            for n, _ in kernels(listing)}
    assert len(here) == 25
    assert here == library_kernels()


def test_no_kernel_spills_or_loses_its_m0(listing):
    found = dict(kernels(listing))
    assert len(found) == 25, sorted(found)
    for name, body in found.items():
        bad, n = lint(body)
        assert n > 0, f"{name}: no direct-to-LDS loads found"
        assert not bad, f"{name}: {bad[:5]}"
    spills = re.findall(r"\.vgpr_spill_count:\s*(\d+)", listing)
    assert len(spills) == 25 and set(spills) == {"0"}
    scratch = re.findall(r"\.private_segment_fixed_size:\s*(\d+)", listing)
    assert len(scratch) == 25 and set(scratch) == {"0"}
