// launch.h -- host-side launchers of the kernel variants (internal).
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "gemm_kernels.h"
#include "mx_kernels.h"

namespace sg {

// Tile shapes the planner chooses between.
enum TileShape { kTile256 = 0, kTile128 = 1, kTile64 = 2 };

constexpr int kCUs = 256;  // MI355X compute units

// Dense GEMM: 256x256 tiles when they fill the CUs, else 128x128 tiles when
// they fill half of them, else 64x64 tiles (small problems: 1024^3 has 64
// tiles of 128 but 256 of 64).  Between those, when the 256x256 tiles would
// run on the ping-pong (`pingpong`: K-major operands, or a K that its loaders
// of MN-major operands take) and the 128x128 tiles would need three or more
// rounds of the CUs, one partial round of the ping-pong is faster (bf16 on
// MI355X, TFLOP/s 256 vs 128 tiles: 3584^3 1337 vs 911), though not against one
// or two rounds of 128x128 tiles (2560^3 753 vs 847, 2048x4096x4096 934 vs 1041).
// `fits256`: 256-row panels stay within 32-bit buffer offsets.
inline TileShape pick_dense_tile(int64_t M, int64_t N, bool pingpong, bool fits256) {
  auto tiles = [&](int64_t side) { return ((M + side - 1) / side) * ((N + side - 1) / side); };
  if (tiles(256) >= kCUs) return kTile256;
  if (pingpong && fits256 && (tiles(128) + kCUs - 1) / kCUs >= 3) return kTile256;
  if (tiles(128) >= kCUs / 2) return kTile128;
  return kTile64;
}

// The kernels of the 8-bit products (i8_kernels.h), named by rows x columns of
// a tile.  kI8Stream32x32: one workgroup a CU with five stages;
// kI8Stream32x32x2: two with two.
enum I8Tile {
  kI8Stream16x16, kI8Stream16x32, kI8Stream16x64, kI8Stream32x16, kI8Stream32x32,
  kI8Stream32x32x2, kI8Stream64x32, kI8Mid64x64, kI8Mid64x128, kI8Mid128x128, kI8PingPong256
};
struct I8Params;
struct RouteParams;
struct PlanParams;
struct BalanceParams;

// A grid of `blocks` workgroups over x and y: a launch has fewer than 2^32
// threads along x.  The kernel's block index is block_index().
inline dim3 grid_of(int64_t blocks) {
  constexpr int64_t kX = int64_t{1} << 20;
  return blocks <= kX ? dim3((unsigned)blocks)
                      : dim3((unsigned)kX, (unsigned)((blocks + kX - 1) / kX));
}
__device__ __forceinline__ int64_t block_index() {
  return (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
}

// Name of the kernel instantiation this thread launched last (set by every
// launcher; read through gemm_last_kernel()).
const char*& last_kernel();

// "name<a,b,...>" built once per instantiation.
template <class... Parts>
const char* kernel_label(const char* name, Parts... parts) {
  std::string s = std::string(name) + "<";
  const char* ps[] = {parts...};
  for (size_t i = 0; i < sizeof...(Parts); ++i) s += (i ? std::string(",") : std::string()) + ps[i];
  s += ">";
  char* out = new char[s.size() + 1];  // one per instantiation, kept for the process
  std::copy(s.begin(), s.end(), out);
  out[s.size()] = 0;
  return out;
}

// Launches the dense kernel for (tile, dtype, majorness).  Returns the
// launch status.
hipError_t launch_dense(TileShape tile, bool bf16, bool a_mn, bool b_mn,
                        const DenseParams& p, hipStream_t s);
// The same where B is MN-major, with 256x256 tiles on the ping-pong for any K.
// A row of a K-major A that ends inside a 16-byte chunk holds zeros in the rest
// of it.
hipError_t launch_dense_any_k(TileShape tile, bool bf16, bool a_mn, bool b_mn,
                              const DenseParams& p, hipStream_t s);
// The layout ablation: bf16, K-major operands, 256x256 tiles on the 32x32x16
// ping-pong kernel with the LDS layout swz (0, 8 or 16 units per line).
hipError_t launch_layout(int swz, const DenseParams& p, hipStream_t s);
// The input/output ablation on the library's 256x256 kernel (16x16x32
// MFMAs, 16-bit D staged in LDS): operand layout swz (16 or 0) and the
// epilogue's C/D staging swizzled (out_swz) or in logical order.
hipError_t launch_layout_io(int swz, bool out_swz, const DenseParams& p, hipStream_t s);
// The same on 128x128 tiles of the 4-wave GemmTile kernel, where the padded
// layout (kSwzPad) also fits: layout 16, 8, 0 or kSwzPad.
hipError_t launch_layout128(int layout, const DenseParams& p, hipStream_t s);
hipError_t launch_grouped(TileShape tile, bool bf16, int swz,
                          const GroupedParams& p, int grid, hipStream_t s);
hipError_t launch_mx(TileShape tile, const MxParams& p, hipStream_t s);
hipError_t launch_mxfp4(const MxParams& p, hipStream_t s);  // 256x256 tiles
hipError_t launch_mxfp6(bool e3m2, const MxParams& p, hipStream_t s);  // 256x256 tiles
// e8m0 scales [rows][K/32] (K a multiple of 128) into the blocks layout of
// SfMap (mx_kernels.h).
hipError_t launch_sf_blocks(const void* sf, int64_t rows, int64_t K, void* out, hipStream_t s);
// The 8-bit product, dense (p.G = 0) or grouped; `grid` workgroups.
hipError_t launch_i8(I8Tile t, const I8Params& p, int grid, hipStream_t s);
// Rows of floats (SG_F32, SG_BF16, SG_F16) to 8-bit codes and row scales.
hipError_t launch_i8_quant(const void* X, int64_t R, int64_t K, int64_t ldx, int dtype, void* Q,
                           int64_t ldq, float* S, hipStream_t s);
// Expert routing (moe.hip); dtype is the logits'.
hipError_t launch_moe_route(int dtype, const RouteParams& p, hipStream_t s);
hipError_t launch_moe_route_backward(int dtype, const RouteParams& p, hipStream_t s);
hipError_t launch_moe_plan(const PlanParams& p, hipStream_t s);
// The routing's balance loss (balance.hip).
hipError_t launch_moe_balance(int dtype, const BalanceParams& p, hipStream_t s);
hipError_t launch_moe_balance_backward(int dtype, const BalanceParams& p, hipStream_t s);
// The MFMA clock probe (diag.hip): one wave per SIMD of 256 CUs.
int clock_probe_waves();
hipError_t launch_clock_probe(int64_t iters, void* out, hipStream_t s);
// LDS images of the 256x256 kernels' loaders and the scaled-MFMA probe
// (diag.hip); kind is one of the SG_IMG_* codes.
hipError_t launch_lds_image_pp(int kind, const char* X, uint32_t x_bytes, uint32_t pitch,
                               int valid, uint32_t kbyte0, uint32_t kbytes_total,
                               uint32_t unshifted, uint32_t t, void* out, hipStream_t s);
hipError_t launch_lds_image_cblock(const void* C, int64_t ldc, int64_t row0, int64_t n0,
                                   int m_valid, int n_valid, void* out, hipStream_t s);
hipError_t launch_mfma_scale_probe(int fmt, const void* a, const void* b, const void* sa,
                                   const void* sb, void* out, hipStream_t s);
hipError_t launch_lds_image(const void* X, int64_t rows_total, int64_t K,
                            int elem_bytes, int64_t row0, int64_t k0,
                            int tile_rows, void* out, hipStream_t s);

}  // namespace sg
