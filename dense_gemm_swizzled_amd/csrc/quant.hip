// quant.hip -- rows of 16- or 32-bit floats to 8-bit integer codes with one
// fp32 scale per row (i8_quant_run).
//
//   a = max |x| over the row, s = max(a, 2^-100) / 127,
//   q = round-to-nearest-even(x * (127 / max(a, 2^-100))),
//
// each step rounded once in fp32, so the codes are the same whole numbers in
// any IEEE implementation.  |q| <= 127: x * (127 / a) exceeds 127 by at most
// two roundings, far from 127.5.  The floor keeps 127 / a finite; a row below
// it has codes zero or coarse codes with an absolute error of at most 2^-107.
// A row that holds an infinity or a NaN has the scale NaN and codes zero.
//
// Bound by memory: es + 1 bytes a value.  A row is read once and stays in
// registers between the maximum and the codes: 16 to 64 lanes of a wave, a
// block of 256 or of 1024 threads, by the row's length (16384 x 8192 bf16 74 us,
// 5.4 TB/s, where a copy reaches 5.0; 200000 x 100 with a wave for each row 41
// us).  Rows past 65536 values are read twice.
#include <hip/hip_runtime.h>

#include "gemm_device.h"
#include "lane_ops.h"
#include "launch.h"

namespace sg {

namespace {

constexpr float kQuantFloor = 0x1p-100f;
constexpr int kChunk = 8;  // values a thread takes at a time

template <int DT>
__device__ __forceinline__ float to_f32(const void* X, int64_t i) {
  if constexpr (DT == SG_F32) return static_cast<const float*>(X)[i];
  const uint32_t h = static_cast<const uint16_t*>(X)[i];
  return DT == SG_BF16 ? bf16_to_f32(h) : f16_to_f32(h);
}

// Eight values from value i.  Rows may start at any element: global loads of
// 16 bytes need no alignment (single 2-byte loads took 171 us for 16384 x 8191
// bf16, these take 93).
template <int DT>
__device__ __forceinline__ void load8(const void* X, int64_t i, float (&v)[kChunk]) {
  if constexpr (DT == SG_F32) {
    f32x4 a, b;
    __builtin_memcpy(&a, static_cast<const float*>(X) + i, 16);
    __builtin_memcpy(&b, static_cast<const float*>(X) + i + 4, 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
  } else {
    u32x4 d;
    __builtin_memcpy(&d, static_cast<const uint16_t*>(X) + i, 16);
#pragma unroll
    for (int e = 0; e < kChunk; ++e) {
      const uint32_t h = (e & 1) ? d[e / 2] >> 16 : d[e / 2] & 0xffffu;
      v[e] = DT == SG_BF16 ? bf16_to_f32(h) : f16_to_f32(h);
    }
  }
}

// |x| of every value as its bits, which order like the values, infinity and
// NaN above all finite ones.
__device__ __forceinline__ uint32_t abs_bits(float x) {
  return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
}

__device__ __forceinline__ int code_of(float x, float inv) {
  return (int)__builtin_rintf(x * inv);
}

template <int Threads>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* lds) {
  m = lane_reduce<(Threads < 64 ? Threads : 64)>(m, OpMax{});
  if constexpr (Threads > 64) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
    __syncthreads();
    m = lds[0];
#pragma unroll
    for (int w = 1; w < Threads / 64; ++w) m = OpMax{}(m, lds[w]);
  }
  return m;
}

// Threads threads a row, each holding NV chunks of 8 values in registers; NV =
// 0: longer rows, read twice.
template <int DT, int Threads, int NV>
__global__ void __launch_bounds__(Threads < 256 ? 256 : Threads)
    i8_quant_kernel(const void* X, int64_t R, int64_t K, int64_t ldx, int8_t* Q, int64_t ldq,
                    float* S) {
  __shared__ uint32_t lds[16];
  constexpr int kRows = Threads < 256 ? 256 / Threads : 1;
  const int t = threadIdx.x % Threads;
  const int64_t row = block_index() * kRows + threadIdx.x / Threads;
  if (row >= R) return;  // a row's threads together
  const int64_t x0 = row * ldx;
  int8_t* const q = Q + row * ldq;
  const int64_t Kp = (K + 15) & ~(int64_t)15;
  constexpr int kBlock = Threads * kChunk;  // values that one chunk of every thread covers

  auto load = [&](int64_t at, float (&v)[kChunk]) {
    if (at + kChunk <= K) {
      load8<DT>(X, x0 + at, v);
      return;
    }
#pragma unroll
    for (int e = 0; e < kChunk; ++e) v[e] = at + e < K ? to_f32<DT>(X, x0 + at + e) : 0.0f;
  };
  auto store = [&](int64_t at, const float (&v)[kChunk], float inv) {
    if (at >= Kp) return;
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c0 = code_of(v[4 * h], inv), c1 = code_of(v[4 * h + 1], inv);
      const int c2 = code_of(v[4 * h + 2], inv), c3 = code_of(v[4 * h + 3], inv);
      w[h] = (uint32_t)(c0 & 255) | (uint32_t)(c1 & 255) << 8 | (uint32_t)(c2 & 255) << 16 |
             (uint32_t)c3 << 24;
    }
    *reinterpret_cast<u32x2*>(q + at) = u32x2{w[0], w[1]};
  };

  uint32_t m = 0;
  float v[NV > 0 ? NV : 1][kChunk];
  const int64_t first = (int64_t)t * kChunk;
  if constexpr (NV > 0) {
#pragma unroll
    for (int b = 0; b < NV; ++b) load(first + b * kBlock, v[b]);
#pragma unroll
    for (int b = 0; b < NV; ++b)
#pragma unroll
      for (int e = 0; e < kChunk; ++e) m = OpMax{}(m, abs_bits(v[b][e]));
  } else {
    for (int64_t at = first; at < Kp; at += kBlock) {
      load(at, v[0]);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) m = OpMax{}(m, abs_bits(v[0][e]));
    }
  }
  m = row_max<Threads>(m, lds);
  const bool finite = m < 0x7f800000u;
  const float a = __builtin_fmaxf(__builtin_bit_cast(float, m), kQuantFloor);
  const float inv = finite ? 127.0f / a : 0.0f;
  if (t == 0) S[row] = finite ? a / 127.0f : __builtin_nanf("");
  auto finish = [&](int64_t at, float (&x)[kChunk]) {
    if (!finite)
#pragma unroll
      for (int e = 0; e < kChunk; ++e) x[e] = 0.0f;
    store(at, x, inv);
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int b = 0; b < NV; ++b) finish(first + b * kBlock, v[b]);
  } else {
    for (int64_t at = first; at < Kp; at += kBlock) {
      load(at, v[0]);
      finish(at, v[0]);
    }
  }
}

template <int DT, int Threads, int NV>
hipError_t go(const void* X, int64_t R, int64_t K, int64_t ldx, int8_t* Q, int64_t ldq, float* S,
              hipStream_t s) {
  constexpr int kRows = Threads < 256 ? 256 / Threads : 1;
  static const char* const name = kernel_label(
      "i8_quant_kernel", Threads <= 64 ? "wave" : Threads == 256 ? "256" : "1024",
      NV == 0 ? "twice" : "once");
  last_kernel() = name;
  hipLaunchKernelGGL((i8_quant_kernel<DT, Threads, NV>), grid_of((R + kRows - 1) / kRows),
                     dim3(Threads < 256 ? 256 : Threads), 0, s, X, R, K, ldx, Q, ldq, S);
  return hipGetLastError();
}

// The fewest threads that hold the row in at most 64 registers each, and no
// barrier while a wave can (1024 values).
template <int DT>
hipError_t by_length(const void* X, int64_t R, int64_t K, int64_t ldx, int8_t* Q, int64_t ldq,
                     float* S, hipStream_t s) {
  const int64_t Kp = (K + 15) & ~(int64_t)15;
  if (Kp <= 128) return go<DT, 16, 1>(X, R, K, ldx, Q, ldq, S, s);
  if (Kp <= 256) return go<DT, 32, 1>(X, R, K, ldx, Q, ldq, S, s);
  if (Kp <= 512) return go<DT, 64, 1>(X, R, K, ldx, Q, ldq, S, s);
  if (Kp <= 1024) return go<DT, 64, 2>(X, R, K, ldx, Q, ldq, S, s);
  if (Kp <= 2048) return go<DT, 256, 1>(X, R, K, ldx, Q, ldq, S, s);
  if (Kp <= 4096) return go<DT, 256, 2>(X, R, K, ldx, Q, ldq, S, s);
  if (Kp <= 8192) return go<DT, 256, 4>(X, R, K, ldx, Q, ldq, S, s);
  if (Kp <= 16384) return go<DT, 256, 8>(X, R, K, ldx, Q, ldq, S, s);
  if (Kp <= 32768) return go<DT, 1024, 4>(X, R, K, ldx, Q, ldq, S, s);
  if (Kp <= 65536) return go<DT, 1024, 8>(X, R, K, ldx, Q, ldq, S, s);
  return go<DT, 1024, 0>(X, R, K, ldx, Q, ldq, S, s);
}

}  // namespace

hipError_t launch_i8_quant(const void* X, int64_t R, int64_t K, int64_t ldx, int dtype, void* Q,
                           int64_t ldq, float* S, hipStream_t s) {
  int8_t* q = static_cast<int8_t*>(Q);
  if (dtype == SG_F32) return by_length<SG_F32>(X, R, K, ldx, q, ldq, S, s);
  if (dtype == SG_BF16) return by_length<SG_BF16>(X, R, K, ldx, q, ldq, S, s);
  return by_length<SG_F16>(X, R, K, ldx, q, ldq, S, s);
}

}  // namespace sg
