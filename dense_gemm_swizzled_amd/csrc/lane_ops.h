// lane_ops.h -- reductions over aligned groups of 8, 16, 32 or 64 lanes of a
// wave, result in every lane.  Steps 1 to 8 are DPP moves inside a row of 16
// lanes (swap neighbours, swap pairs, mirror 8, mirror 16: after the earlier
// steps the mirrored partner holds the other half's result), 16 and 32 the
// gfx950 row swaps; none touches LDS.  The order of a sum is fixed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sg {

// The value of the lane that step S pairs this one with (S = 1, 2, 4, 8).
template <int S>
__device__ __forceinline__ uint32_t dpp_partner(uint32_t v) {
  constexpr int kCtrl = S == 1 ? 0xB1 : S == 2 ? 0x4E : S == 4 ? 0x141 : 0x140;
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xf, 0xf, true);
}

// Both sides of step S (16, 32): the lower and the upper partner's value.
template <int S>
__device__ __forceinline__ void swap_pair(uint32_t v, uint32_t& lo, uint32_t& hi) {
  if constexpr (S == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    lo = r[0];
    hi = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    lo = r[0];
    hi = r[1];
  }
}

template <int S, class T, class Op>
__device__ __forceinline__ T reduce_step(T v, Op op) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    if constexpr (S < 16) return op(v, __builtin_bit_cast(T, dpp_partner<S>(u)));
    uint32_t lo, hi;
    swap_pair<S < 16 ? 16 : S>(u, lo, hi);
    return op(__builtin_bit_cast(T, lo), __builtin_bit_cast(T, hi));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t u0 = (uint32_t)u, u1 = (uint32_t)(u >> 32);
    if constexpr (S < 16)
      return op(v, __builtin_bit_cast(T, (uint64_t)dpp_partner<S>(u1) << 32 | dpp_partner<S>(u0)));
    uint32_t lo0, hi0, lo1, hi1;
    swap_pair<S < 16 ? 16 : S>(u0, lo0, hi0);
    swap_pair<S < 16 ? 16 : S>(u1, lo1, hi1);
    return op(__builtin_bit_cast(T, (uint64_t)lo1 << 32 | lo0),
              __builtin_bit_cast(T, (uint64_t)hi1 << 32 | hi0));
  }
}

template <int Lanes, class T, class Op>
__device__ __forceinline__ T lane_reduce(T v, Op op) {
  static_assert(Lanes == 8 || Lanes == 16 || Lanes == 32 || Lanes == 64, "lane groups");
  v = reduce_step<1>(v, op);
  v = reduce_step<2>(v, op);
  v = reduce_step<4>(v, op);
  if constexpr (Lanes >= 16) v = reduce_step<8>(v, op);
  if constexpr (Lanes >= 32) v = reduce_step<16>(v, op);
  if constexpr (Lanes >= 64) v = reduce_step<32>(v, op);
  return v;
}

struct OpMax {
  template <class T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a > b ? a : b; }
  __device__ __forceinline__ float operator()(float a, float b) const {
    return __builtin_fmaxf(a, b);
  }
  __device__ __forceinline__ double operator()(double a, double b) const {
    return __builtin_fmax(a, b);
  }
};
struct OpSum {
  template <class T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};

}  // namespace sg
