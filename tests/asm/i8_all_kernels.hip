// Device-only translation unit for tests/test_asm_i8_all_cpu.py: every
// instantiation of the 8-bit kernels that launch_i8.hip launches.
#include "../../dense_gemm_swizzled_amd/csrc/i8_kernels.h"

namespace sg {
#define SG_FORMS(DEF) DEF(false, false) DEF(true, false) DEF(true, true)
#define SG_PINGPONG(G, R) template __global__ void i8_pingpong_kernel<G, R>(const I8Params);
SG_FORMS(SG_PINGPONG)
}  // namespace sg
