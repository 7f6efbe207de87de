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

template <int BM, int BN, bool Grouped, bool Rows>
hipError_t go_mid(const I8Params& p, int grid, hipStream_t s) {
  static const char* const name = kernel_label("i8_mid_kernel", BM == 128 ? "128" : "64",
                                               BN == 128 ? "128" : "64", shape_name(Grouped, Rows));
  last_kernel() = name;
  hipLaunchKernelGGL((i8_mid_kernel<BM, BN, Grouped, Rows>), dim3(grid), dim3(512), 0, s, p);
  return hipGetLastError();
}

template <int MT, int NT, int WN, int Stages, bool Grouped, bool Rows>
hipError_t go_stream(const I8Params& p, int grid, hipStream_t s) {
  static const char* const name = kernel_label(
      "i8_stream_kernel", MT == 1 ? "16" : MT == 2 ? "32" : "64",
      NT * WN == 1 ? "16" : NT * WN == 2 ? "32" : "64", shape_name(Grouped, Rows));
  last_kernel() = name;
  hipLaunchKernelGGL((i8_stream_kernel<MT, NT, WN, Stages, Grouped, Rows>), dim3(grid), dim3(512),
                     0, s, p);
  return hipGetLastError();
}

template <bool Grouped, bool Rows>
hipError_t by_tile(I8Tile t, const I8Params& p, int grid, hipStream_t s) {
  if constexpr (!Grouped) {  // grouped products stream with 16 rows only
    if (t == kI8Stream32x16) return go_stream<2, 1, 1, 5, Grouped, Rows>(p, grid, s);
    if (t == kI8Stream32x32) return go_stream<2, 2, 1, 5, Grouped, Rows>(p, grid, s);
    if (t == kI8Stream32x32x2) return go_stream<2, 2, 1, 2, Grouped, Rows>(p, grid, s);
    if (t == kI8Stream64x32) return go_stream<4, 2, 1, 3, Grouped, Rows>(p, grid, s);
  }
  switch (t) {
    case kI8Stream16x16: return go_stream<1, 1, 1, 4, Grouped, Rows>(p, grid, s);
    case kI8Stream16x32: return go_stream<1, 2, 1, 3, Grouped, Rows>(p, grid, s);
    case kI8Stream16x64: return go_stream<1, 2, 2, 2, Grouped, Rows>(p, grid, s);
    case kI8Mid64x64: return go_mid<64, 64, Grouped, Rows>(p, grid, s);
    case kI8Mid64x128: return go_mid<64, 128, Grouped, Rows>(p, grid, s);
    case kI8Mid128x128: return go_mid<128, 128, Grouped, Rows>(p, grid, s);
    case kI8PingPong256: return go_pingpong<Grouped, Rows>(p, grid, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_i8(I8Tile t, const I8Params& p, int grid, hipStream_t s) {
  if (p.G == 0) return by_tile<false, false>(t, p, grid, s);
  return p.rows ? by_tile<true, true>(t, p, grid, s) : by_tile<true, false>(t, p, grid, s);
}

}  // namespace sg
