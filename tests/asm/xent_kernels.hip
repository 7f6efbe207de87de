// Device-only translation unit for tests/test_asm_lint_xent_cpu.py: every kernel
// of the cross entropy, and the products of any K that its gradients run.
#include "../../dense_gemm_swizzled_amd/csrc/xent.hip"

namespace sg {
template __global__ void pingpong16_gemm_kernel<true, kSwzDefault, true, true, true, true>(
    const DenseParams);
template __global__ void pingpong16_gemm_kernel<false, kSwzDefault, true, true, true, true>(
    const DenseParams);
template __global__ void pingpong16_gemm_kernel<true, kSwzDefault, false, true, true, true>(
    const DenseParams);
template __global__ void pingpong16_gemm_kernel<false, kSwzDefault, false, true, true, true>(
    const DenseParams);
}  // namespace sg
