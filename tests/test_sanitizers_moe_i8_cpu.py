"""The host code of the expert-routing and 8-bit entry points under
AddressSanitizer and UndefinedBehaviorSanitizer (no GPU): their validation
paths, the plan's chunks, and the kernel that each size of the tests of every
kernel takes (tests/sanitize/abi_moe_i8_driver.cpp).  Two streaming kernels
share a label, so that only the choice itself tells them apart."""
import os

import pytest

from test_sanitizers_cpu import HIPCC, ROOT, SAN, _run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
def test_routing_and_8bit_host_code_under_asan_ubsan():
    from dense_gemm_swizzled_amd import _build
    objs = [os.path.join(_build.BUILD, s.replace(".hip", ".o"))
            for s in _build.SOURCES if s != "api.hip"]
    if not all(os.path.exists(o) for o in objs):
        _build.build()
    os.makedirs(SAN, exist_ok=True)
    host_san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined"]
    drv_o, exe = (os.path.join(SAN, n) for n in ("abi_moe_i8_driver.o", "abi_moe_i8_san"))
    _run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", *host_san,
          "-Xarch_host", "-fno-sanitize-recover=all", "-fPIC",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-x", "hip",
          "-I", os.path.join(ROOT, "include"), "-c",
          os.path.join(ROOT, "tests", "sanitize", "abi_moe_i8_driver.cpp"), "-o", drv_o])
    _run([HIPCC, "--offload-arch=gfx950", *host_san, drv_o, *objs, "-o", exe])
    r = _run([exe], env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert "clean" in r.stdout
