// Device-only translation unit for the assembly lint in
// tests/test_asm_lint_i8_cpu.py: the 8-bit kernels whose direct-to-LDS loads
// take m0 from a separate, earlier write.
#include "../../dense_gemm_swizzled_amd/csrc/i8_kernels.h"

namespace sg {
template __global__ void i8_pingpong_kernel<false, false>(const I8Params);
template __global__ void i8_pingpong_kernel<true, false>(const I8Params);
template __global__ void i8_pingpong_kernel<true, true>(const I8Params);
template __global__ void i8_mid_kernel<64, 128, true, true>(const I8Params);
template __global__ void i8_mid_kernel<128, 128, true, true>(const I8Params);
}  // namespace sg
