// balance.hip -- the balance loss of expert routing (moe_balance_run) and the
// gradient of the router's logits (moe_balance_backward_run):
//
//   share[t][e] = s[t][e] / sum_e s[t][e]     (s: softmax or sigmoid scores),
//   load[e]     = E counts[e] / sum_e counts[e],
//   loss        = sum_e load[e] * (1/n) sum_t share[t][e],
//
// over the n tokens that have an expert left; 1 where either side is even.
#include <hip/hip_runtime.h>

#include "launch.h"
#include "moe.h"
#include "moe_rows.h"

namespace sg {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kSumThreads = 1024;
constexpr int kGradThreads = 256;

// A token's scores over Lanes lanes with Quads quads of experts each (quad q of
// the lane: experts from 4 * (q * Lanes + lane)), their sum, and for a sigmoid
// 1 - s.  A masked logit scores zero; a token with all masked has the sum zero.
// With many tokens the pass waits for chains of these instructions as much as for
// memory (its waves stand two thirds of their time, 27 to 29% of the vector issue
// of 65521 x 128 is used), so they are few: expf, a division and the masks of
// moe_rows.h made 16384 x 256 fp32 take 1 us more.  The exponentials are off by
// |x - top|, or |x| for a sigmoid, units of 2^-24 of themselves, the rounding of
// their arguments; the reciprocals, here and of the sums, by one unit.
template <int Lanes, int Quads, bool Rest>
__device__ __forceinline__ float scores(float (&x)[Quads][kHeld], float (&rest)[Quads][kHeld],
                                        bool soft) {
  float part = 0.0f;
  if (soft) {
    float top = -__builtin_inff();
#pragma unroll
    for (int q = 0; q < Quads; ++q) top = OpMax{}(top, lane_top(x[q]));
    top = lane_reduce<Lanes>(top, OpMax{});
    if (top == -__builtin_inff()) top = 0.0f;
#pragma unroll
    for (int q = 0; q < Quads; ++q)
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {  // (2^-inf is zero)
        x[q][i] = __builtin_amdgcn_exp2f((x[q][i] - top) * kLog2e);
        part += x[q][i];
      }
  } else {
#pragma unroll
    for (int q = 0; q < Quads; ++q)
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const float z = __builtin_amdgcn_exp2f(x[q][i] * -kLog2e);  // (of -inf: +inf)
        x[q][i] = __builtin_amdgcn_rcpf(1.0f + z);
        if constexpr (Rest) rest[q][i] = __builtin_fminf(z, FLT_MAX) * x[q][i];
        part += x[q][i];
      }
  }
  return lane_reduce<Lanes>(part, OpSum{});
}

// The instructions above flush a sigmoid score below 2^-126 to zero.  Beside a sum
// of kFar or more that is a share of less than 2^-96; a token below it, a far
// one, is left to a second pass, which makes its shares from ratios.  (Made where
// it is met, in a branch of the first pass: 16384 x 256 fp32 0.4 us more, the
// gradient too.)
constexpr float kFar = 0x1p-30f;

// The scores of a far token (logits below -20: sigmoid x is e^x and 1 - s is 1 to
// 2^-30) over the largest, their sum, and 2^-126 over the largest, which is the
// least that they are divided by.
struct FarSum {
  float sum, least;
};
template <int Lanes, int Quads>
__device__ __forceinline__ FarSum far_scores(float (&x)[Quads][kHeld]) {
  float top = -__builtin_inff(), part = 0.0f;
#pragma unroll
  for (int q = 0; q < Quads; ++q) top = OpMax{}(top, lane_top(x[q]));
  top = lane_reduce<Lanes>(top, OpMax{});
  if (top == -__builtin_inff()) top = 0.0f;
#pragma unroll
  for (int q = 0; q < Quads; ++q)
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      x[q][i] = __builtin_amdgcn_exp2f((x[q][i] - top) * kLog2e);
      part += x[q][i];
    }
  return {lane_reduce<Lanes>(part, OpSum{}),
          __builtin_amdgcn_exp2f(__builtin_fmaf(top, -kLog2e, -126.0f))};
}

// The workspace: for each workgroup E pairs of a sum and a count, a pair (0,
// tokens), and one more where that makes the rows multiples of 16 bytes.
__host__ __device__ constexpr int part_pitch(int E) { return (E + 2) & ~1; }

// The loss from the sums S and counts of the experts, one thread each (none
// from E on); n: the tokens.  In 64 bits, added in a fixed order.
__device__ __forceinline__ void finish(const BalanceParams& p, float S, int count, int n,
                                       double (&area)[2][4]) {
  double dot = (double)S * count, all = count;
  dot = lane_reduce<64>(dot, OpSum{});
  all = lane_reduce<64>(all, OpSum{});
  if ((threadIdx.x & 63) == 0 && threadIdx.x < SG_MAX_GROUPS) {
    area[0][threadIdx.x >> 6] = dot;
    area[1][threadIdx.x >> 6] = all;
  }
  if ((int)threadIdx.x < p.E) p.counts[threadIdx.x] = count;
  __syncthreads();
  if (threadIdx.x == 0) {
    dot = (area[0][0] + area[0][1]) + (area[0][2] + area[0][3]);
    all = (area[1][0] + area[1][1]) + (area[1][2] + area[1][3]);
    p.loss[0] = n > 0 && all > 0 ? (float)(p.E * dot / (all * n)) : 0.0f;
    p.tokens[0] = n;
  }
}

// The value of the lane 8 places on in its row of 16, round the end.
__device__ __forceinline__ float eight_away(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x128, 0xf, 0xf, true));
}

// One workgroup adds up the shares of a run of tokens and counts their ids.  A
// lane keeps the sums of its experts in registers over its tokens (the next
// token's logits loading meanwhile), the lanes that hold the same experts are
// added through LDS in a fixed order, the counts are integers in LDS.  Alone:
// the only workgroup, which finishes the loss itself.
template <int DT, int Lanes, int Quads, bool Alone>
__global__ void __launch_bounds__(kSumThreads) moe_balance_kernel(const BalanceParams p) {
  constexpr int kTokens = kSumThreads / Lanes, kWaves = kSumThreads / 64;
  constexpr int kExperts = Lanes * Quads * kHeld;
  __shared__ __attribute__((aligned(16))) float sums[kWaves][kExperts];
  __shared__ int counts[SG_MAX_GROUPS + 1];  // the last: tokens
  __shared__ double area[2][4];
  const int tid = threadIdx.x, lane = tid % Lanes, slot = tid / Lanes;
  const bool soft = p.score == SG_SCORE_SOFTMAX;
  const int64_t first = (int64_t)blockIdx.x * p.chunk, end = min(first + p.chunk, p.T);
  float sum[Quads][kHeld] = {}, next[Quads][kHeld];
  int live = 0;
  bool far = false;
  auto load = [&](int64_t t) {
#pragma unroll
    for (int q = 0; q < Quads; ++q)
      load_row4<DT, true>(p, t, kHeld * (q * Lanes + lane), t < end, next[q]);
  };
  load(first + slot);
  if (tid <= SG_MAX_GROUPS) counts[tid] = 0;
  __syncthreads();
  for (int64_t i = first * p.top_k + tid; i < end * p.top_k; i += kSumThreads) {
    const int id = p.ids[i];
    if ((uint32_t)id < (uint32_t)p.E) atomicAdd(&counts[id], 1);
  }
  for (int64_t t = first + slot; t - slot < end; t += kTokens) {  // (whole waves go round)
    float x[Quads][kHeld], none[Quads][kHeld];
#pragma unroll
    for (int q = 0; q < Quads; ++q)
#pragma unroll
      for (int i = 0; i < kHeld; ++i) x[q][i] = next[q][i];
    if (t - slot + kTokens < end) load(t + kTokens);
    bool any = false;
#pragma unroll
    for (int q = 0; q < Quads; ++q) any |= lane_top(x[q]) > -__builtin_inff();
    const float total = scores<Lanes, Quads, false>(x, none, soft);
    const uint64_t who = __ballot(any) >> (tid & 63 & ~(Lanes - 1));
    live += lane == 0 && (Lanes == 64 ? who : who & ((1ull << (Lanes & 63)) - 1)) ? 1 : 0;
    far |= any && total < kFar;
    const float over = total < kFar ? 0.0f : __builtin_amdgcn_rcpf(total);
#pragma unroll
    for (int q = 0; q < Quads; ++q)
#pragma unroll
      for (int i = 0; i < kHeld; ++i) sum[q][i] += x[q][i] * over;
  }
  if (__any(far)) {  // (of the wave's tokens)
    for (int64_t t = first + slot; t - slot < end; t += kTokens) {
      float x[Quads][kHeld], none[Quads][kHeld];
      load(t);
#pragma unroll
      for (int q = 0; q < Quads; ++q)
#pragma unroll
        for (int i = 0; i < kHeld; ++i) x[q][i] = next[q][i];
      if (scores<Lanes, Quads, false>(x, none, soft) >= kFar) continue;
      const FarSum f = far_scores<Lanes, Quads>(next);
      const float over = __builtin_amdgcn_rcpf(__builtin_fmaxf(f.sum, f.least));
#pragma unroll
      for (int q = 0; q < Quads; ++q)
#pragma unroll
        for (int i = 0; i < kHeld; ++i) sum[q][i] += next[q][i] * over;
    }
  }
  if (live) atomicAdd(&counts[SG_MAX_GROUPS], live);
#pragma unroll
  for (int q = 0; q < Quads; ++q) {
    f32x4 v;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      float s = sum[q][i];
      if constexpr (Lanes <= 8) s += eight_away(s);
      if constexpr (Lanes <= 16) s = reduce_step<16>(s, OpSum{});
      if constexpr (Lanes <= 32) s = reduce_step<32>(s, OpSum{});
      v[i] = s;
    }
    if ((tid & 63) < Lanes)
      *reinterpret_cast<f32x4*>(&sums[tid >> 6][kHeld * (q * Lanes + lane)]) = v;
  }
  __syncthreads();
  float S = 0.0f;
  if (tid < kExperts) {
#pragma unroll
    for (int w = 0; w < kWaves; ++w) S += sums[w][tid];
  }
  if constexpr (Alone) {
    finish(p, tid < p.E ? S : 0.0f, tid < p.E ? counts[tid] : 0, counts[SG_MAX_GROUPS], area);
  } else {
    u32x2* const out = static_cast<u32x2*>(p.part) + (int64_t)blockIdx.x * part_pitch(p.E);
    if (tid < p.E) out[tid] = u32x2{__builtin_bit_cast(uint32_t, S), (uint32_t)counts[tid]};
    if (tid == p.E) out[tid] = u32x2{0u, (uint32_t)counts[SG_MAX_GROUPS]};
  }
}

// Adds up the workgroups' pairs and finishes the loss: one workgroup, a thread for
// two experts and a fixed share of the rows, 16 loads of 16 bytes in flight.  What
// a CU can read bounds it (256 experts of 256 workgroups, 0.5 MB).  (Sixteen
// workgroups and a last one that waits for them took 7 us for any number of
// experts: their fences and the count of those that are done.)
template <int Wide>
__global__ void __launch_bounds__(kSumThreads) moe_balance_join_kernel(const BalanceParams p) {
  constexpr int kCols = Wide / 2, kSegs = kSumThreads / kCols, kBatch = 16;
  __shared__ float sums[kSegs][Wide];
  __shared__ int counts[kSegs][Wide], tokens[kSumThreads / 64];
  __shared__ double area[2][4];
  const int tid = threadIdx.x, c = tid % kCols, seg = tid / kCols;
  const int pitch = part_pitch(p.E);
  const u32x2* const part = static_cast<const u32x2*>(p.part);
  float S[2] = {};
  int count[2] = {}, n = 0;
  if (tid < p.parts) n = (int)part[tid * pitch + p.E][1];
  for (int b0 = seg; b0 < p.parts; b0 += kBatch * kSegs) {
    u32x4 v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      v[i] = *reinterpret_cast<const u32x4*>(part + min(b0 + i * kSegs, p.parts - 1) * pitch +
                                             min(2 * c, pitch - 2));
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const bool on = b0 + i * kSegs < p.parts;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t bits = v[i][2 * h], number = v[i][2 * h + 1];
        S[h] += on ? __builtin_bit_cast(float, bits) : 0.0f;
        count[h] += on ? (int)number : 0;
      }
    }
  }
  n = lane_reduce<64>(n, OpSum{});
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    sums[seg][2 * c + h] = S[h];
    counts[seg][2 * c + h] = count[h];
  }
  if ((tid & 63) == 0) tokens[tid >> 6] = n;
  __syncthreads();
  float all = 0.0f;
  int number = 0;
  n = 0;
  if (tid < p.E) {
#pragma unroll
    for (int i = 0; i < kSegs; ++i) {
      all += sums[i][tid];
      number += counts[i][tid];
    }
  }
#pragma unroll
  for (int w = 0; w < kSumThreads / 64; ++w) n += tokens[w];
  finish(p, all, number, n, area);
}

// With d_e = dloss E counts[e] / (sum counts * n), the gradient of share e:
//   softmax  dx_e = share_e (d_e - sum_j share_j d_j),
//   sigmoid  dx_e = share_e (1 - s_e) (d_e - sum_j share_j d_j),
// without the sum over j where the scores are divided by 2^-126.
// Bound by memory: reads the logits, writes their gradient.
template <int DT, int Lanes, int Quads>
__global__ void __launch_bounds__(kGradThreads) moe_balance_backward_kernel(
    const BalanceParams p) {
  constexpr int kTokens = kGradThreads / Lanes;
  const int lane = threadIdx.x % Lanes, slot = threadIdx.x / Lanes;
  const bool soft = p.score == SG_SCORE_SOFTMAX;
  const int64_t step = (int64_t)gridDim.x * kTokens;
  const int64_t first = (int64_t)blockIdx.x * kTokens;
  float next[Quads][kHeld];
  auto load = [&](int64_t t) {
#pragma unroll
    for (int q = 0; q < Quads; ++q)
      load_row4<DT, true>(p, t, kHeld * (q * Lanes + lane), t < p.T, next[q]);
  };
  load(first + slot);
  // (sums of counts in fp32: off by a unit of 2^-24 a step)
  float d[Quads][kHeld], all = 0.0f;
#pragma unroll
  for (int q = 0; q < Quads; ++q)
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int e = kHeld * (q * Lanes + lane) + i;
      d[q][i] = e < p.E ? (float)p.counts[e] : 0.0f;
      all += d[q][i];
    }
  all = lane_reduce<Lanes>(all, OpSum{});
  const float n = (float)p.tokens[0];
  const float f = all > 0 && n > 0 ? p.dloss[0] * ((float)p.E / all / n) : 0.0f;
#pragma unroll
  for (int q = 0; q < Quads; ++q)
#pragma unroll
    for (int i = 0; i < kHeld; ++i) d[q][i] *= f;

  // One token's gradient from its scores and what they are multiplied by; fixed: by
  // a constant, so that no other share changes with one.
  auto gradient = [&](int64_t t, float (&x)[Quads][kHeld], const float (&rest)[Quads][kHeld],
                      bool ones, float over, bool fixed) {
    float dot = 0.0f;
#pragma unroll
    for (int q = 0; q < Quads; ++q)
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        x[q][i] *= over;
        dot += x[q][i] * d[q][i];
      }
    dot = lane_reduce<Lanes>(dot, OpSum{});
    if (fixed) dot = 0.0f;
    if (t >= p.T) return;
#pragma unroll
    for (int q = 0; q < Quads; ++q) {
      const int e0 = kHeld * (q * Lanes + lane);
      if (e0 >= p.E) break;
      f32x4 v;
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        v[i] = x[q][i] * (ones ? 1.0f : rest[q][i]) * (d[q][i] - dot);
      store_row4<DT>(p, t, e0, v);
    }
  };
  auto pass = [&](auto kind) {
    constexpr bool kSoft = decltype(kind)::value;
    bool far = false;
    for (int64_t t = first + slot; t - slot < p.T; t += step) {
      float x[Quads][kHeld], rest[Quads][kHeld];
#pragma unroll
      for (int q = 0; q < Quads; ++q)
#pragma unroll
        for (int i = 0; i < kHeld; ++i) x[q][i] = next[q][i];
      if (t - slot + step < p.T) load(t + step);
      bool any = false;
      if constexpr (!kSoft) {
#pragma unroll
        for (int q = 0; q < Quads; ++q) any |= lane_top(x[q]) > -__builtin_inff();
      }
      const float total = scores<Lanes, Quads, true>(x, rest, kSoft);
      far |= any && total < kFar;
      gradient(t, x, rest, kSoft, total < kFar ? 0.0f : __builtin_amdgcn_rcpf(total), false);
    }
    if (kSoft || !__any(far)) return;
    // (the wave's far tokens, whose rows are written again)
    for (int64_t t = first + slot; t - slot < p.T; t += step) {
      float x[Quads][kHeld], rest[Quads][kHeld];
      load(t);
#pragma unroll
      for (int q = 0; q < Quads; ++q)
#pragma unroll
        for (int i = 0; i < kHeld; ++i) x[q][i] = next[q][i];
      if (scores<Lanes, Quads, false>(x, rest, false) >= kFar) continue;
      const FarSum f = far_scores<Lanes, Quads>(next);
      gradient(t, next, rest, true, __builtin_amdgcn_rcpf(__builtin_fmaxf(f.sum, f.least)),
               f.least > f.sum);
    }
  };
  if (soft) pass(std::true_type{});
  else pass(std::false_type{});
}

constexpr const char* type_label(int dt) {
  return dt == SG_F32 ? "f32" : dt == SG_BF16 ? "bf16" : "f16";
}
constexpr const char* digits(int n) {
  return n == 1 ? "1" : n == 2 ? "2" : n == 4 ? "4" : n == 8 ? "8" : n == 16 ? "16"
         : n == 32 ? "32" : "64";
}

template <int DT, int Lanes, int Quads>
hipError_t go_sum(const BalanceParams& p, hipStream_t s) {
  static const char* const name =
      kernel_label("moe_balance_kernel", type_label(DT), digits(Lanes), digits(Quads));
  last_kernel() = name;
  if (p.parts == 1) {
    hipLaunchKernelGGL((moe_balance_kernel<DT, Lanes, Quads, true>), dim3(1), dim3(kSumThreads),
                       0, s, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((moe_balance_kernel<DT, Lanes, Quads, false>), dim3(p.parts),
                     dim3(kSumThreads), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int kWide = Lanes * Quads * kHeld <= 64 ? 64 : Lanes * Quads * kHeld;
  hipLaunchKernelGGL((moe_balance_join_kernel<kWide>), dim3(1), dim3(kSumThreads), 0, s, p);
  return hipGetLastError();
}

template <int DT, int Lanes, int Quads>
hipError_t go_grad(const BalanceParams& p, hipStream_t s) {
  static const char* const name =
      kernel_label("moe_balance_backward_kernel", type_label(DT), digits(Lanes), digits(Quads));
  last_kernel() = name;
  constexpr int kTokens = kGradThreads / Lanes;
  // Three or four workgroups a CU that go on to their next tokens, whose logits
  // load meanwhile (us in a graph, 16384 x 256 fp32 with 512 | 768 | 1024 | one
  // for each 8 tokens: 11.5 | 10.6 | 11.8 | 13.5; 65521 x 128 bf16 14.8 | 12.8 |
  // 12.4 | 15.9).
  constexpr int64_t kMost = Lanes > 16 ? 768 : 1024;
  const int64_t blocks = std::min<int64_t>((p.T + kTokens - 1) / kTokens, kMost);
  hipLaunchKernelGGL((moe_balance_backward_kernel<DT, Lanes, Quads>), dim3((unsigned)blocks),
                     dim3(kGradThreads), 0, s, p);
  return hipGetLastError();
}

// Lanes and quads by measured times (us in a graph, 16 x 4 | 32 x 2 | 64 x 1:
// 16384 x 256 fp32 sigmoid 18.2 | 17.5 | 16.9, its gradient 13.2 | 10.6 | 10.8;
// 8 x 4 | 16 x 2 | 32 x 1: 65521 x 128 bf16 15.9 | 15.3 | 16.4, its gradient
// 12.7 | 12.4 | 13.7).
template <int DT>
hipError_t forward(const BalanceParams& p, hipStream_t s) {
  if (p.E <= 32) return go_sum<DT, 8, 1>(p, s);
  if (p.E <= 64) return go_sum<DT, 8, 2>(p, s);
  if (p.E <= 128) return go_sum<DT, 16, 2>(p, s);
  return go_sum<DT, 64, 1>(p, s);
}

template <int DT>
hipError_t backward(const BalanceParams& p, hipStream_t s) {
  if (p.E <= 32) return go_grad<DT, 8, 1>(p, s);
  if (p.E <= 64) return go_grad<DT, 8, 2>(p, s);
  if (p.E <= 128) return go_grad<DT, 16, 2>(p, s);
  return go_grad<DT, 32, 2>(p, s);
}

}  // namespace

hipError_t launch_moe_balance(int dtype, const BalanceParams& p, hipStream_t s) {
  if (dtype == SG_F32) return forward<SG_F32>(p, s);
  if (dtype == SG_BF16) return forward<SG_BF16>(p, s);
  return forward<SG_F16>(p, s);
}

hipError_t launch_moe_balance_backward(int dtype, const BalanceParams& p, hipStream_t s) {
  if (dtype == SG_F32) return backward<SG_F32>(p, s);
  if (dtype == SG_BF16) return backward<SG_BF16>(p, s);
  return backward<SG_F16>(p, s);
}

}  // namespace sg
