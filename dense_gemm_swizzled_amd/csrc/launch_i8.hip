// launch_i8.hip -- instantiations and launchers of the 8-bit products.
#include "i8_kernels.h"
#include "launch.h"

namespace sg {

namespace {

constexpr const char* shape_name(bool grouped, bool rows) {
  return grouped ? (rows ? "grouped,rows" : "grouped") : "dense";
}

template <bool Grouped, bool Rows>
hipError_t go_pingpong(const I8Params& p, int grid, hipStream_t s) {
  static const char* const name = kernel_label("i8_pingpong_kernel", shape_name(Grouped, Rows));
  last_kernel() = name;
  hipLaunchKernelGGL((i8_pingpong_kernel<Grouped, Rows>), dim3(grid), dim3(512), 0, s, p);
  return hipGetLastError();
}

template <int BM, bool Grouped, bool Rows>
hipError_t go_deep(const I8Params& p, int grid, hipStream_t s) {
  static const char* const name = kernel_label("i8_deep_kernel", BM == 128 ? "128" : "64",
                                               shape_name(Grouped, Rows));
  last_kernel() = name;
  hipLaunchKernelGGL((i8_deep_kernel<BM, Grouped, Rows>), dim3(grid), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <int MT, int NT, bool Grouped, bool Rows>
hipError_t go_skinny(const I8Params& p, int grid, hipStream_t s) {
  static const char* const name =
      kernel_label("i8_skinny_kernel", MT == 1 ? "16" : MT == 2 ? "32" : "64",
                   shape_name(Grouped, Rows));
  last_kernel() = name;
  hipLaunchKernelGGL((i8_skinny_kernel<MT, NT, Grouped, Rows>), dim3(grid), dim3(512), 0, s, p);
  return hipGetLastError();
}

template <bool Grouped, bool Rows>
hipError_t by_tile(I8Tile t, const I8Params& p, int grid, hipStream_t s) {
  switch (t) {
    case kI8Skinny16: return go_skinny<1, 1, Grouped, Rows>(p, grid, s);
    case kI8Skinny32: return go_skinny<2, 1, Grouped, Rows>(p, grid, s);
    case kI8Skinny64: return go_skinny<4, 2, Grouped, Rows>(p, grid, s);
    case kI8Tile64: return go_deep<64, Grouped, Rows>(p, grid, s);
    case kI8Tile128: return go_deep<128, Grouped, Rows>(p, grid, s);
    default: return go_pingpong<Grouped, Rows>(p, grid, s);
  }
}

}  // namespace

hipError_t launch_i8(I8Tile t, const I8Params& p, int grid, hipStream_t s) {
  if (p.G == 0) return by_tile<false, false>(t, p, grid, s);
  return p.rows ? by_tile<true, true>(t, p, grid, s) : by_tile<true, false>(t, p, grid, s);
}

}  // namespace sg
