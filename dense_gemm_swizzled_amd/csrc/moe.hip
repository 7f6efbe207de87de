// moe.hip -- routing of tokens to experts: the choice and its weights
// (moe_route_run), the weights' gradient (moe_route_backward_run), and the
// sort of the (token, expert) pairs by expert (moe_plan_run).
#include <hip/hip_runtime.h>

#include <cfloat>

#include "gemm_device.h"
#include "lane_ops.h"
#include "launch.h"
#include "moe.h"

namespace sg {

namespace {

constexpr int kHeld = 4;             // experts a lane holds: e = i * Lanes + lane
constexpr float kTiny = 0x1p-126f;   // smallest sum that weights are divided by
constexpr int kBlockThreads = 256;

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

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

// 1 / (1 + e^-x) without overflow; small results keep their denormals.
template <class F>
__device__ __forceinline__ F sigmoid_of(F x) {
  const F z = exp_of(x < 0 ? x : -x);
  return (x < 0 ? z : F(1)) / (F(1) + z);
}

// The scores of a token's experts in type F; x masked (-inf) scores zero.
template <int Lanes, class F>
__device__ __forceinline__ void scores_of(const float (&x)[kHeld], int score, F (&s)[kHeld]) {
  if (score == SG_SCORE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      s[i] = x[i] > -__builtin_inff() ? sigmoid_of((F)x[i]) : F(0);
    return;
  }
  float m = x[0];
#pragma unroll
  for (int i = 1; i < kHeld; ++i) m = OpMax{}(m, x[i]);
  m = lane_reduce<Lanes>(m, OpMax{});
  F sum = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    s[i] = x[i] > -__builtin_inff() ? exp_of((F)x[i] - (F)m) : F(0);
    sum += s[i];
  }
  sum = lane_reduce<Lanes>(sum, OpSum{});
  sum = sum > F(kTiny) ? sum : F(kTiny);
#pragma unroll
  for (int i = 0; i < kHeld; ++i) s[i] /= sum;
}

// One group of Lanes lanes a token.  Key: what the experts are ordered by --
// the logits themselves (float: score is increasing in the logit, so without
// a bias they give the exact order of the scores), or score + bias in 64 bits.
template <int DT, int Lanes, class Key>
__global__ void __launch_bounds__(kBlockThreads) moe_route_kernel(const RouteParams p) {
  constexpr int kTokens = kBlockThreads / Lanes;
  constexpr bool kScores = sizeof(Key) == 8;
  const Key kNone = -(Key)__builtin_inff();
  const int lane = threadIdx.x % Lanes, slot = threadIdx.x / Lanes;
  const int64_t t = (int64_t)blockIdx.x * kTokens + slot;
  const bool live = t < p.T;  // a token past the end goes along for the barriers

  float x[kHeld], s[kHeld];
  Key key[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int e = i * Lanes + lane;
    x[i] = live && e < p.E ? clean(load_logit<DT>(p.logits, t * p.ldl + e)) : -__builtin_inff();
  }
  if constexpr (kScores) {
    double wide[kHeld];
    scores_of<Lanes>(x, p.score, wide);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int e = i * Lanes + lane;
      s[i] = (float)wide[i];
      const double b = p.bias && e < p.E ? (double)p.bias[e] : 0.0;
      const double k = wide[i] + b;
      key[i] = x[i] > -__builtin_inff() && k > kNone ? k : kNone;
    }
  } else {
    scores_of<Lanes>(x, p.score, s);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) key[i] = x[i];
  }

  if (p.n_groups > 1) {  // keep the top_groups best groups
    __shared__ Key keys[kBlockThreads * kHeld];
    __shared__ Key best[kTokens * SG_MAX_ROUTE_GROUPS];
    Key* const kt = keys + slot * Lanes * kHeld;
    Key* const bt = best + slot * SG_MAX_ROUTE_GROUPS;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) kt[i * Lanes + lane] = key[i];
    __syncthreads();
    const int size = p.E / p.n_groups;
    for (int g = lane; g < p.n_groups; g += Lanes) {
      Key b0 = kNone, b1 = kNone;
      for (int m = 0; m < size; ++m) {
        const Key k = kt[g * size + m];
        if (k > b0) {
          b1 = b0;
          b0 = k;
        } else if (k > b1) {
          b1 = k;
        }
      }
      bt[g] = p.group_score == SG_GROUP_TOP2 && b1 > kNone ? b0 + b1 : b0;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int e = i * Lanes + lane;
      if (e >= p.E) continue;
      const int g = e / size;
      const Key mine = bt[g];
      int above = 0;  // groups before this expert's; ties go to the lowest
      for (int h = 0; h < p.n_groups; ++h) above += bt[h] > mine || (bt[h] == mine && h < g);
      if (above >= p.top_groups) key[i] = kNone;
    }
  }

  // top_k times the largest key, the lowest expert among equal ones.
  int rank[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) rank[i] = -1;
  const int base = (threadIdx.x & 63) / Lanes * Lanes;
  const uint64_t mask = Lanes == 64 ? ~0ull : ((1ull << (Lanes & 63)) - 1) << base;
  int found = 0;
  for (int k = 0; k < p.top_k; ++k) {
    Key m = key[0];
#pragma unroll
    for (int i = 1; i < kHeld; ++i) m = OpMax{}(m, key[i]);
    m = lane_reduce<Lanes>(m, OpMax{});
    if (!(m > kNone)) break;  // (this lane group; the others may go on)
    bool open = true;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const uint64_t eq = __ballot(key[i] == m) & mask;
      if (open && eq) {
        open = false;
        if ((int)__builtin_ctzll(eq) == (int)(threadIdx.x & 63)) {
          rank[i] = k;
          key[i] = kNone;
        }
      }
    }
    ++found;
  }

  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) sum += rank[i] >= 0 ? s[i] : 0.0f;
  sum = lane_reduce<Lanes>(sum, OpSum{});
  const float div = p.renorm ? __builtin_fmaxf(sum, kTiny) : 1.0f;
  if (!live) return;
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (rank[i] >= 0) {
      p.ids[t * p.top_k + rank[i]] = i * Lanes + lane;
      p.weights[t * p.top_k + rank[i]] = s[i] / div * p.scale;
    }
  for (int k = found + lane; k < p.top_k; k += Lanes) {
    p.ids[t * p.top_k + k] = -1;
    p.weights[t * p.top_k + k] = 0.0f;
  }
}

template <int DT>
__device__ __forceinline__ void store_logit(void* D, int64_t i, float v) {
  if constexpr (DT == SG_F32)
    static_cast<float*>(D)[i] = v;
  else if constexpr (DT == SG_BF16)
    static_cast<__bf16*>(D)[i] = (__bf16)v;
  else
    static_cast<_Float16*>(D)[i] = (_Float16)v;
}

// With r_j = s_j / S (S = max(sum s, 2^-126) with renorm, else 1) and g_j the
// gradient of weight j times the scale, the gradient of expert id_j's score
// times that score is
//   u_j = r_j (g_j - [renorm, S above the floor] sum_i g_i r_i),
// and of the logits, summing u_j over the j that name the expert,
//   sigmoid  dx_e = u_e (1 - s_e),
//   softmax  dx_e = u_e - s_e sum_j u_j   (the sum is zero with renorm).
// Only ratios of scores appear, so small scores lose nothing.
template <int DT, int Lanes>
__global__ void __launch_bounds__(kBlockThreads) moe_route_backward_kernel(
    const RouteParams p) {
  constexpr int kTokens = kBlockThreads / Lanes;
  __shared__ float us[kTokens * SG_MAX_TOP_K];
  __shared__ int is[kTokens * SG_MAX_TOP_K];
  const int lane = threadIdx.x % Lanes, slot = threadIdx.x / Lanes;
  const int64_t t = (int64_t)blockIdx.x * kTokens + slot;
  const bool live = t < p.T;
  float x[kHeld], s[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int e = i * Lanes + lane;
    x[i] = live && e < p.E ? clean(load_logit<DT>(p.logits, t * p.ldl + e)) : -__builtin_inff();
  }
  scores_of<Lanes>(x, p.score, s);

  // The chosen experts' scores travel through LDS to the lanes of their j.
  __shared__ float sc[kBlockThreads * kHeld];
  float* const st = sc + slot * Lanes * kHeld;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) st[i * Lanes + lane] = s[i];
  __syncthreads();
  float sum = 0.0f;
  for (int k = lane; k < p.top_k; k += Lanes) {
    const int id = live ? p.ids[t * p.top_k + k] : -1;
    is[slot * SG_MAX_TOP_K + k] = id;
    sum += (uint32_t)id < (uint32_t)p.E ? st[id] : 0.0f;
  }
  sum = lane_reduce<Lanes>(sum, OpSum{});
  const bool floor = !(sum >= kTiny);
  const float div = !p.renorm ? 1.0f : floor ? kTiny : sum;
  float dot = 0.0f;
  for (int k = lane; k < p.top_k; k += Lanes) {
    const int id = is[slot * SG_MAX_TOP_K + k];
    const bool in = (uint32_t)id < (uint32_t)p.E;
    const float g = in ? p.dweights[t * p.top_k + k] * p.scale : 0.0f;
    const float r = in ? st[id] / div : 0.0f;
    dot += g * r;
  }
  dot = lane_reduce<Lanes>(dot, OpSum{});
  const float mean = p.renorm && !floor ? dot : 0.0f;
  for (int k = lane; k < p.top_k; k += Lanes) {
    const int id = is[slot * SG_MAX_TOP_K + k];
    const bool in = (uint32_t)id < (uint32_t)p.E;
    const float g = in ? p.dweights[t * p.top_k + k] * p.scale : 0.0f;
    us[slot * SG_MAX_TOP_K + k] = in ? st[id] / div * (g - mean) : 0.0f;
  }
  const float total = p.renorm && !floor ? 0.0f : dot;
  __syncthreads();
  float u[kHeld] = {};
  for (int k = 0; k < p.top_k; ++k) {
    const int id = is[slot * SG_MAX_TOP_K + k];
    const float v = us[slot * SG_MAX_TOP_K + k];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) u[i] += id == i * Lanes + lane ? v : 0.0f;
  }
  if (!live) return;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int e = i * Lanes + lane;
    if (e >= p.E) continue;
    const float d = p.score == SG_SCORE_SIGMOID ? u[i] * (1.0f - s[i]) : u[i] - s[i] * total;
    store_logit<DT>(p.dlogits, t * p.lddl + e, x[i] > -__builtin_inff() ? d : 0.0f);
  }
}

// ------------------------------------------------------------------ the plan
//
// A stable counting sort of P = T * top_k ids: bucket of an id outside [0, E)
// is E, behind all experts.  Each block owns a contiguous chunk of pairs, each
// of its waves a contiguous part of the chunk.  Lanes of a wave that hold the
// same id find each other by one ballot per bit of the id, which gives their
// order; no atomic decides a place, so the result is the same every time.

constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;
constexpr int kPlanBins = SG_MAX_GROUPS + 1;

// The lanes of the wave that hold the same key (0 .. 2^bits - 1).
__device__ __forceinline__ uint64_t same_key(int key, int bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool on = (key >> b) & 1;
    const uint64_t v = __ballot(on);
    m &= on ? v : ~v;
  }
  return m;
}

__global__ void __launch_bounds__(kPlanThreads) moe_plan_count_kernel(const PlanParams p) {
  __shared__ int bins[kPlanBins];
  const int n = p.E + 1;
  for (int e = threadIdx.x; e < n; e += kPlanThreads) bins[e] = 0;
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * p.chunk;
  const int64_t c1 = c0 + p.chunk < p.P ? c0 + p.chunk : p.P;
  for (int64_t i = c0 + threadIdx.x; i < c1; i += kPlanThreads) {
    const int id = p.ids[i];
    atomicAdd(&bins[(uint32_t)id < (uint32_t)p.E ? id : p.E], 1);  // counts: any order
  }
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += kPlanThreads)
    p.counts[(int64_t)blockIdx.x * n + e] = bins[e];
}

// Multi: the chunks' counts are in p.counts; else this block owns all pairs.
template <bool Multi>
__global__ void __launch_bounds__(kPlanThreads) moe_plan_place_kernel(const PlanParams p) {
  __shared__ int bins[kPlanWaves][kPlanBins];  // first counts, then next places
  __shared__ int start[kPlanBins];
  __shared__ int wave_sum[kPlanWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = p.E + 1, bits = 32 - __builtin_clz(p.E);
  for (int e = tid; e < kPlanWaves * kPlanBins; e += kPlanThreads) (&bins[0][0])[e] = 0;
  __syncthreads();

  const int64_t c0 = (int64_t)blockIdx.x * p.chunk;
  const int64_t c1 = c0 + p.chunk < p.P ? c0 + p.chunk : p.P;
  const int64_t per = ((p.chunk + kPlanWaves - 1) / kPlanWaves + 63) / 64 * 64;
  const int64_t w0 = c0 + wave * per, w1 = w0 + per < c1 ? w0 + per : c1;
  auto bucket = [&](int64_t i) {
    if (i >= w1) return -1;
    const int id = p.ids[i];
    return (uint32_t)id < (uint32_t)p.E ? id : p.E;
  };
  for (int64_t b = w0; b < w1; b += 64) {
    const int key = bucket(b + lane);
    if (key >= 0) atomicAdd(&bins[wave][key], 1);
  }
  __syncthreads();

  // Totals of the buckets, and how many of each come before this block.
  int total = 0, before = 0, own = 0;
  if (tid < n) {
    for (int w = 0; w < kPlanWaves; ++w) own += bins[w][tid];
    if constexpr (Multi) {
      for (int b = 0; b < (int)gridDim.x; ++b) {
        const int v = p.counts[(int64_t)b * n + tid];
        total += v;
        before += b < (int)blockIdx.x ? v : 0;
      }
    } else {
      total = own;
    }
  }
  // Exclusive scan of the totals (the first n <= 257 threads: waves 0 .. 4).
  int upto = total;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 63) wave_sum[wave] = upto;
  __syncthreads();
  if (tid < n) {
    int first = upto - total;
    for (int w = 0; w < wave; ++w) first += wave_sum[w];
    if (blockIdx.x == 0) p.offsets[tid] = first;  // n = E + 1 entries
    start[tid] = first + before;
  }
  __syncthreads();
  if (tid < n) {  // counts of the waves become their first places
    int at = start[tid];
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = bins[w][tid];
      bins[w][tid] = at;
      at += c;
    }
  }
  __syncthreads();

  for (int64_t b = w0; b < w1; b += 64) {
    const int64_t i = b + lane;
    const int key = bucket(i);
    const bool in = key >= 0;
    const uint64_t same = same_key(in ? key : 0, bits) & __ballot(in);
    if (in) {
      const int before_me = __builtin_popcountll(same & ((1ull << lane) - 1));
      const int place = bins[wave][key] + before_me;
      p.slots[i] = key < p.E ? place : -1;
      if (place < p.P) p.rows[place] = key < p.E ? (int)(i / p.top_k) : -1;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (in && (same >> lane) == 1)  // the last lane of its id moves the place on
      bins[wave][key] += __builtin_popcountll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

constexpr const char* dt_label(int dt) {
  return dt == SG_F32 ? "f32" : dt == SG_BF16 ? "bf16" : "f16";
}

template <int DT, int Lanes, bool Back>
hipError_t go_route(const RouteParams& p, hipStream_t s) {
  constexpr int kTokens = kBlockThreads / Lanes;
  const dim3 grid((unsigned)((p.T + kTokens - 1) / kTokens));
  constexpr const char* kL = Lanes == 8 ? "8" : Lanes == 16 ? "16" : Lanes == 32 ? "32" : "64";
  if constexpr (Back) {
    static const char* const name = kernel_label("moe_route_backward_kernel", dt_label(DT), kL);
    last_kernel() = name;
    hipLaunchKernelGGL((moe_route_backward_kernel<DT, Lanes>), grid, dim3(kBlockThreads), 0, s, p);
  } else {
    static const char* const names[2] = {
        kernel_label("moe_route_kernel", dt_label(DT), kL, "logits"),
        kernel_label("moe_route_kernel", dt_label(DT), kL, "scores")};
    last_kernel() = names[p.by_score ? 1 : 0];
    if (p.by_score)
      hipLaunchKernelGGL((moe_route_kernel<DT, Lanes, double>), grid, dim3(kBlockThreads), 0, s,
                         p);
    else
      hipLaunchKernelGGL((moe_route_kernel<DT, Lanes, float>), grid, dim3(kBlockThreads), 0, s,
                         p);
  }
  return hipGetLastError();
}

// The fewest lanes that hold a token's experts, four to a lane.
template <int DT, bool Back>
hipError_t by_experts(const RouteParams& p, hipStream_t s) {
  if (p.E <= 32) return go_route<DT, 8, Back>(p, s);
  if (p.E <= 64) return go_route<DT, 16, Back>(p, s);
  if (p.E <= 128) return go_route<DT, 32, Back>(p, s);
  return go_route<DT, 64, Back>(p, s);
}

template <bool Back>
hipError_t by_type(int dtype, const RouteParams& p, hipStream_t s) {
  if (dtype == SG_F32) return by_experts<SG_F32, Back>(p, s);
  if (dtype == SG_BF16) return by_experts<SG_BF16, Back>(p, s);
  return by_experts<SG_F16, Back>(p, s);
}

}  // namespace

hipError_t launch_moe_route(int dtype, const RouteParams& p, hipStream_t s) {
  return by_type<false>(dtype, p, s);
}

hipError_t launch_moe_route_backward(int dtype, const RouteParams& p, hipStream_t s) {
  return by_type<true>(dtype, p, s);
}

hipError_t launch_moe_plan(const PlanParams& p, hipStream_t s) {
  static const char* const names[2] = {kernel_label("moe_plan_place_kernel", "single"),
                                       kernel_label("moe_plan_place_kernel", "multi")};
  const int blocks = (int)((p.P + p.chunk - 1) / p.chunk);
  last_kernel() = names[blocks > 1 ? 1 : 0];
  if (blocks <= 1) {
    hipLaunchKernelGGL((moe_plan_place_kernel<false>), dim3(1), dim3(kPlanThreads), 0, s, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(moe_plan_count_kernel, dim3(blocks), dim3(kPlanThreads), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_plan_place_kernel<true>), dim3(blocks), dim3(kPlanThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace sg
