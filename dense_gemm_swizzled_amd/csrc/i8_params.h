// i8_params.h -- launch parameters of the 8-bit products (i8_kernels.h).
#pragma once

#include <stdint.h>

#include "gemm_device.h"

namespace sg {

struct I8Params {
  const void* A;
  const void* B;
  const float* SA;
  const float* SB;
  void* D;
  int64_t M, N, K;           // M: rows of D
  int64_t lda, ldb, ldd;     // bytes, bytes, elements
  int d_dtype;
  bool vec;                  // D and its row pitch are 16-byte aligned
  int tiles_m, tiles_n;      // dense only: tiles_m
  int group_m;
  ClockTrace clk;
  // Grouped: group g owns rows [offsets[g], offsets[g+1]) of D and the matrix
  // B + g * N * ldb; row r of D takes row rows[r] (or r) of A.
  int G;
  const int32_t* offsets;
  const int32_t* rows;
  int a_total;               // rows of A
};

}  // namespace sg
