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
// Bound by memory: es + 1 bytes a value.  The row is read once and stays in
// registers between the maximum and the codes.
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

// Chunk c of a row: 8 consecutive values with vector loads (Vec: every row is
// 16-byte aligned and K a multiple of 8), else the values c, c + n, c + 2n ...
// of a block of 8n so that a wave's loads stay contiguous.
template <int DT>
__device__ __forceinline__ void load8(const void* X, int64_t i, float (&v)[kChunk]) {
  if constexpr (DT == SG_F32) {
    const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(X) + i);
    const f32x4 a = p[0], b = p[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
  } else {
    const u32x4 d = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(X) + i);
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
  m = lane_reduce<64>(m, OpMax{});
  if constexpr (Threads > 64) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
    __syncthreads();
    m = lds[0];
#pragma unroll
    for (int w = 1; w < Threads / 64; ++w) m = OpMax{}(m, lds[w]);
  }
  return m;
}

// Threads threads a row (one wave, or the whole block of 256), NV chunks each
// held in registers; NV = 0: rows longer than that, read twice.
template <int DT, int Threads, int NV, bool Vec>
__global__ void __launch_bounds__(256) i8_quant_kernel(const void* X, int64_t R, int64_t K,
                                                       int64_t ldx, int8_t* Q, int64_t ldq,
                                                       float* S) {
  __shared__ uint32_t lds[4];
  const int t = threadIdx.x % Threads;
  const int64_t row = (int64_t)blockIdx.x * (256 / Threads) + threadIdx.x / Threads;
  if (row >= R) return;  // whole waves only, and with Threads = 256 whole blocks
  const int64_t x0 = row * ldx;
  int8_t* const q = Q + row * ldq;
  const int64_t Kp = (K + 15) & ~(int64_t)15;
  constexpr int kBlock = Threads * kChunk;  // values a chunk index covers

  auto at = [&](int64_t b, int e) {  // the column of value e of this thread's chunk
    return Vec ? b * kBlock + t * kChunk + e : b * kBlock + e * Threads + t;
  };
  auto load = [&](int64_t b, float (&v)[kChunk]) {
    if constexpr (Vec) {
      if (at(b, 0) < K) {
        load8<DT>(X, x0 + at(b, 0), v);
        return;
      }
    }
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
      v[e] = !Vec && at(b, e) < K ? to_f32<DT>(X, x0 + at(b, e)) : 0.0f;
  };
  auto store = [&](int64_t b, const float (&v)[kChunk], float inv) {
    if constexpr (Vec) {
      if (at(b, 0) >= Kp) return;
      uint32_t w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c0 = code_of(v[4 * h], inv), c1 = code_of(v[4 * h + 1], inv);
        const int c2 = code_of(v[4 * h + 2], inv), c3 = code_of(v[4 * h + 3], inv);
        w[h] = (uint32_t)(c0 & 255) | (uint32_t)(c1 & 255) << 8 | (uint32_t)(c2 & 255) << 16 |
               (uint32_t)c3 << 24;
      }
      *reinterpret_cast<u32x2*>(q + at(b, 0)) = u32x2{w[0], w[1]};
    } else {
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        if (at(b, e) < Kp) q[at(b, e)] = (int8_t)code_of(v[e], inv);
    }
  };

  uint32_t m = 0;
  constexpr int kHeld = NV > 0 ? NV : 1;
  float v[kHeld][kChunk];
  const int64_t blocks = NV > 0 ? NV : (Kp + kBlock - 1) / kBlock;
  if constexpr (NV > 0) {
#pragma unroll
    for (int b = 0; b < NV; ++b) load(b, v[b]);
#pragma unroll
    for (int b = 0; b < NV; ++b)
#pragma unroll
      for (int e = 0; e < kChunk; ++e) m = OpMax{}(m, abs_bits(v[b][e]));
  } else {
    for (int64_t b = 0; b < blocks; ++b) {
      load(b, v[0]);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) m = OpMax{}(m, abs_bits(v[0][e]));
    }
  }
  m = row_max<Threads>(m, lds);
  const bool finite = m < 0x7f800000u;
  const float a = __builtin_fmaxf(__builtin_bit_cast(float, m), kQuantFloor);
  const float inv = finite ? 127.0f / a : 0.0f;
  if (t == 0) S[row] = finite ? a / 127.0f : __builtin_nanf("");
  if constexpr (NV > 0) {
#pragma unroll
    for (int b = 0; b < NV; ++b) {
      if (!finite)
#pragma unroll
        for (int e = 0; e < kChunk; ++e) v[b][e] = 0.0f;
      store(b, v[b], inv);
    }
  } else {
    for (int64_t b = 0; b < blocks; ++b) {
      load(b, v[0]);
      if (!finite)
#pragma unroll
        for (int e = 0; e < kChunk; ++e) v[0][e] = 0.0f;
      store(b, v[0], inv);
    }
  }
}

template <int DT, int Threads, int NV, bool Vec>
hipError_t go(const void* X, int64_t R, int64_t K, int64_t ldx, int8_t* Q, int64_t ldq, float* S,
              hipStream_t s) {
  constexpr int kRows = 256 / Threads;
  static const char* const name =
      kernel_label("i8_quant_kernel", Threads == 64 ? "wave" : "block", Vec ? "vec" : "any");
  last_kernel() = name;
  hipLaunchKernelGGL((i8_quant_kernel<DT, Threads, NV, Vec>), dim3((R + kRows - 1) / kRows),
                     dim3(256), 0, s, X, R, K, ldx, Q, ldq, S);
  return hipGetLastError();
}

// One wave a row while the row fits its registers (no barrier), then a block.
template <int DT, bool Vec>
hipError_t by_length(const void* X, int64_t R, int64_t K, int64_t ldx, int8_t* Q, int64_t ldq,
                     float* S, hipStream_t s) {
  const int64_t Kp = (K + 15) & ~(int64_t)15;
  if (Kp <= 512) return go<DT, 64, 1, Vec>(X, R, K, ldx, Q, ldq, S, s);
  if (Kp <= 1024) return go<DT, 64, 2, Vec>(X, R, K, ldx, Q, ldq, S, s);
  if (Kp <= 2048) return go<DT, 256, 1, Vec>(X, R, K, ldx, Q, ldq, S, s);
  if (Kp <= 4096) return go<DT, 256, 2, Vec>(X, R, K, ldx, Q, ldq, S, s);
  if (Kp <= 8192) return go<DT, 256, 4, Vec>(X, R, K, ldx, Q, ldq, S, s);
  if (Kp <= 16384) return go<DT, 256, 8, Vec>(X, R, K, ldx, Q, ldq, S, s);
  return go<DT, 256, 0, Vec>(X, R, K, ldx, Q, ldq, S, s);
}

}  // namespace

hipError_t launch_i8_quant(const void* X, int64_t R, int64_t K, int64_t ldx, int dtype, void* Q,
                           int64_t ldq, float* S, hipStream_t s) {
  const int es = dtype == SG_F32 ? 4 : 2;
  const bool vec = K % 8 == 0 && (ldx * es) % 16 == 0 &&
                   (reinterpret_cast<uintptr_t>(X) & 15u) == 0;
  int8_t* q = static_cast<int8_t*>(Q);
#define SG_Q(DT) \
  return vec ? by_length<DT, true>(X, R, K, ldx, q, ldq, S, s) \
             : by_length<DT, false>(X, R, K, ldx, q, ldq, S, s)
  if (dtype == SG_F32) SG_Q(SG_F32);
  if (dtype == SG_BF16) SG_Q(SG_BF16);
  SG_Q(SG_F16);
#undef SG_Q
}

}  // namespace sg
