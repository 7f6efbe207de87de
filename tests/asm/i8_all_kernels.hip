// Device-only translation unit for tests/test_asm_i8_all_cpu.py: every
// instantiation of the 8-bit kernels that launch_i8.hip launches.
#include "../../dense_gemm_swizzled_amd/csrc/i8_kernels.h"

namespace sg {
#define SG_FORMS(DEF, ...) \
  DEF(__VA_ARGS__, false, false) DEF(__VA_ARGS__, true, false) DEF(__VA_ARGS__, true, true)
#define SG_PINGPONG(T, G, R) template __global__ void i8_pingpong_kernel<G, R>(const T);
#define SG_MID(M, N, G, R) template __global__ void i8_mid_kernel<M, N, G, R>(const I8Params);
#define SG_STREAM(M, N, W, S, G, R) \
  template __global__ void i8_stream_kernel<M, N, W, S, G, R>(const I8Params);
SG_FORMS(SG_PINGPONG, I8Params)
SG_FORMS(SG_MID, 64, 64)
SG_FORMS(SG_MID, 64, 128)
SG_FORMS(SG_MID, 128, 128)
SG_FORMS(SG_STREAM, 1, 1, 1, 4)
SG_FORMS(SG_STREAM, 1, 2, 1, 3)
SG_FORMS(SG_STREAM, 1, 2, 2, 2)
SG_STREAM(2, 1, 1, 5, false, false)  // (grouped products stream with 16 rows only)
SG_STREAM(2, 2, 1, 5, false, false)
SG_STREAM(2, 2, 1, 2, false, false)
SG_STREAM(4, 2, 1, 3, false, false)
}  // namespace sg
