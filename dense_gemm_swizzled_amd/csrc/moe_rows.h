// moe_rows.h -- a token's row of router logits over a group of lanes: loads,
// masks, scores and stores (moe.hip, balance.hip).  A Params has T, E, logits
// [T][ldl] and vec (four logits at a multiple of four are one aligned load);
// for the stores dlogits [T][lddl] and vec_d.
#pragma once

#include <cfloat>

#include "gemm_kernels.h"
#include "lane_ops.h"

namespace sg {

constexpr int kHeld = 4;             // experts of a quad: a lane holds one, or more in the gradient
constexpr float kTiny = 0x1p-126f;   // smallest sum that weights are divided by

template <int DT>
__device__ __forceinline__ float load_logit(const void* X, int64_t i) {
  if constexpr (DT == SG_F32) return static_cast<const float*>(X)[i];
  const uint32_t h = static_cast<const uint16_t*>(X)[i];
  return DT == SG_BF16 ? bf16_to_f32(h) : f16_to_f32(h);
}

// A masked logit (-inf or NaN) is -inf; +inf counts as the largest float, so
// that differences of logits stay numbers.
__device__ __forceinline__ float clean(float x) {
  return x > -__builtin_inff() ? __builtin_fminf(x, FLT_MAX) : -__builtin_inff();
}

// The same in two instructions: a maximum with a NaN is the other number.
__device__ __forceinline__ float clean_fast(float x) {
  return __builtin_fminf(__builtin_fmaxf(x, -__builtin_inff()), FLT_MAX);
}

// The logits of experts e0 .. e0+3 of row t, masked past E.  vec: four logits
// from any multiple of four are one aligned load.
template <int DT, bool Fast = false, class Params>
__device__ __forceinline__ void load_row4(const Params& p, int64_t t, int e0, bool live,
                                          float (&x)[kHeld]) {
  auto cleaned = [](float v) { return Fast ? clean_fast(v) : clean(v); };
  if (live && p.vec && e0 + kHeld <= p.E) {
    const int64_t at = t * p.ldl + e0;
    if constexpr (DT == SG_F32) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p.logits) + at);
#pragma unroll
      for (int i = 0; i < kHeld; ++i) x[i] = cleaned(v[i]);
    } else {
      const u32x2 v = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p.logits) + at);
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const uint32_t h = (i & 1) ? v[i / 2] >> 16 : v[i / 2] & 0xffffu;
        x[i] = cleaned(DT == SG_BF16 ? bf16_to_f32(h) : f16_to_f32(h));
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    x[i] = live && e0 + i < p.E ? cleaned(load_logit<DT>(p.logits, t * p.ldl + e0 + i))
                                : -__builtin_inff();
}

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

// 1 / (1 + e^-x) without overflow; small results keep their denormals.
template <class F>
__device__ __forceinline__ F sigmoid_of(F x) {
  const F z = exp_of(x < 0 ? x : -x);
  return (x < 0 ? z : F(1)) / (F(1) + z);
}

__device__ __forceinline__ float lane_top(const float (&x)[kHeld]) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < kHeld; ++i) m = OpMax{}(m, x[i]);
  return m;
}
template <int DT, class Params>
__device__ __forceinline__ void store_row4(const Params& p, int64_t t, int e0, f32x4 v) {
  const int64_t at = t * p.lddl + e0;
  if (p.vec_d && e0 + kHeld <= p.E) {
    if constexpr (DT == SG_F32)
      *reinterpret_cast<f32x4*>(static_cast<float*>(p.dlogits) + at) = v;
    else
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.dlogits) + at) = pack_d16<DT>(v);
    return;
  }
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    if (e0 + i >= p.E) break;
    if constexpr (DT == SG_F32)
      static_cast<float*>(p.dlogits)[at + i] = v[i];
    else if constexpr (DT == SG_BF16)
      static_cast<__bf16*>(p.dlogits)[at + i] = (__bf16)(float)v[i];
    else
      static_cast<_Float16*>(p.dlogits)[at + i] = (_Float16)(float)v[i];
  }
}

}  // namespace sg
