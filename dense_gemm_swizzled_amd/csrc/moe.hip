// moe.hip -- routing of tokens to experts: the choice and its weights
// (moe_route_run), the weights' gradient (moe_route_backward_run), and the
// sort of the (token, expert) pairs by expert (moe_plan_run).
#include <hip/hip_runtime.h>

#include <cfloat>
#include <type_traits>

#include "gemm_kernels.h"
#include "lane_ops.h"
#include "launch.h"
#include "moe.h"
#include "moe_rows.h"

namespace sg {

namespace {

constexpr float kDenormalOff = 0x1p-146f;  // error of a score below 2^-126, eight steps
constexpr int kBlockThreads = 256;

template <int Lanes>
__device__ __forceinline__ float row_top(const float (&x)[kHeld]) {
  return lane_reduce<Lanes>(lane_top(x), OpMax{});
}

// The scores of a token's experts in type F, up to a common divisor, which is
// returned: the chosen ones alone are divided by it.  x masked (-inf) scores
// zero.
template <int Lanes, class F>
__device__ __forceinline__ F scores_of(const float (&x)[kHeld], int score, F (&s)[kHeld]) {
  if (score == SG_SCORE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      s[i] = x[i] > -__builtin_inff() ? sigmoid_of((F)x[i]) : F(0);
    return F(1);
  }
  const float m = row_top<Lanes>(x);
  F sum = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    s[i] = x[i] > -__builtin_inff() ? exp_of((F)x[i] - (F)m) : F(0);
    sum += s[i];
  }
  sum = lane_reduce<Lanes>(sum, OpSum{});
  return sum > F(kTiny) ? sum : F(kTiny);
}

// A token's lanes are in one wave, whose LDS accesses complete in order: what
// one lane wrote another may read after this.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// LDS of one token.
template <int Lanes, class Key>
struct RouteScratch {
  Key keys[Lanes * kHeld];
  Key best[SG_MAX_ROUTE_GROUPS];
  int keep[SG_MAX_ROUTE_GROUPS];  // first the bits of a group's slack
};

// Masks (kNone) the experts outside the top_groups best groups.  2^j lanes
// share a group's members and merge their two largest; half of their sum is
// the group's score, which no finite keys make infinite.  With Certify, keys
// are fp32 sums of a bias and a score that is off by up to `noise`; returns
// whether every kept group stays above every dropped one whatever the errors.
// In units of 2^-24 of a group's larger key, half the sum is off by noise, one
// unit for the keys' own rounding and one for the sum's; a bound rounds by one.
template <int Lanes, bool Certify, class Key>
__device__ __forceinline__ bool keep_groups(const RouteParams& p, RouteScratch<Lanes, Key>& sc,
                                            int lane, Key (&key)[kHeld], float noise = 0.0f) {
  const Key kNone = -(Key)__builtin_inff();
#pragma unroll
  for (int i = 0; i < kHeld; ++i) sc.keys[kHeld * lane + i] = key[i];
  wave_sync();
  const int G = p.n_groups, size = p.E / G;
  int share = 1;
  while (2 * share * G <= Lanes) share *= 2;
  const int part = lane & (share - 1);
  for (int g0 = 0; g0 < G; g0 += Lanes / share) {
    const int g = g0 + lane / share;
    Key b0 = kNone, b1 = kNone;
    if (g < G)
      for (int m = part; m < size; m += share) {
        const Key k = sc.keys[g * size + m];
        b1 = OpMax{}(b1, k < b0 ? k : b0);
        b0 = OpMax{}(b0, k);
      }
    for (int d = 1; d < share; d *= 2) {
      const Key o0 = __shfl_xor(b0, d), o1 = __shfl_xor(b1, d);
      b1 = OpMax{}(OpMax{}(b1, o1), b0 < o0 ? b0 : o0);
      b0 = OpMax{}(b0, o0);
    }
    if (g < G && part == 0) {
      const bool two = p.group_score == SG_GROUP_TOP2;
      sc.best[g] = !two ? b0 : b1 > kNone ? b0 / 2 + b1 / 2 : b0 / 2;
      if constexpr (Certify) {
        const float a0 = __builtin_fabsf(b0), a1 = __builtin_fabsf(b1), inf = __builtin_inff();
        const float m0 = a0 < inf ? a0 : 0.0f, m1 = two && a1 < inf ? a1 : 0.0f;
        sc.keep[g] = __builtin_bit_cast(int, noise + 0x1p-22f * OpMax{}(m0, m1));
      }
    }
  }
  wave_sync();
  Key low = (Key)__builtin_inff(), high = kNone;  // of the kept and the dropped groups
  for (int g = lane; g < G; g += Lanes) {
    const Key mine = sc.best[g];
    int above = 0;  // groups before this one; ties go to the lowest
    for (int h = 0; h < G; ++h) {
      const Key o = sc.best[h];
      above += o > mine || (o == mine && h < g);
    }
    const bool keep = above < p.top_groups;
    if constexpr (Certify) {
      const float slack = __builtin_bit_cast(float, sc.keep[g]);
      low = keep && mine - slack < low ? mine - slack : low;
      high = keep ? high : OpMax{}(high, mine + slack);
    }
    sc.keep[g] = keep;
  }
  wave_sync();
  const int inv = (65536 + size - 1) / size;  // e / size for e < 256
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int e = kHeld * lane + i;
    if (e < p.E && !sc.keep[(e * inv) >> 16]) key[i] = kNone;
  }
  if constexpr (!Certify) return true;
  low = -lane_reduce<Lanes>(-low, OpMax{});
  high = lane_reduce<Lanes>(high, OpMax{});
  return !(high > kNone) || low > high;  // (a dropped group without a key leaves no doubt)
}

// What keys are compared as: doubles as they are, floats as integers of the
// same order (one instruction a step of a maximum, where a float's maximum
// first quiets its operands).  -0 and 0 are one key.
__device__ __forceinline__ double order_of(double k) { return k; }
__device__ __forceinline__ int order_of(float k) {
  const int u = __builtin_bit_cast(int, k + 0.0f);
  return u ^ (int)((uint32_t)(u >> 31) >> 1);
}
__device__ __forceinline__ double key_at(double o) { return o; }
__device__ __forceinline__ float key_at(int o) {
  return __builtin_bit_cast(float, o ^ (int)((uint32_t)(o >> 31) >> 1));
}

// top_k times the largest key, the lowest expert among equal ones: chosen[k]
// receives (expert, s).  Each lane keeps its four keys sorted, so a round
// compares the lanes' heads, finds the lowest lane that holds the largest and
// pops it.  Returns how many experts were found; with Gaps, `gap` is the
// smallest distance between one choice and the next, the first expert not
// chosen included, less what the keys' own rounding can make up: two units of
// 2^-24 of the larger.
struct Chosen {
  int id;
  float s;
};
template <int Lanes, bool Gaps, class Key>
__device__ __forceinline__ int choose(const RouteParams& p, int lane, const Key (&key)[kHeld],
                                      const float (&s)[kHeld], Chosen* chosen, Key& gap) {
  typedef decltype(order_of(key[0])) Ord;
  const Ord kNone = order_of(-(Key)__builtin_inff());
  Ord h[kHeld];
  int at[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    h[i] = order_of(key[i]);
    at[i] = i;
  }
  // Neighbours change places only when out of order, so equal keys keep theirs.
  auto order = [&](int i) {
    const bool swap = h[i] < h[i + 1];
    const Ord a = h[i], b = h[i + 1];
    const int m = at[i], n = at[i + 1];
    h[i] = swap ? b : a;
    h[i + 1] = swap ? a : b;
    at[i] = swap ? n : m;
    at[i + 1] = swap ? m : n;
  };
  order(0), order(2), order(1), order(0), order(2), order(1);
  static_assert(kHeld == 4, "the sorting network");
  const int self = threadIdx.x & 63, base = self / Lanes * Lanes;
  const uint64_t mask = Lanes == 64 ? ~0ull : ((1ull << (Lanes & 63)) - 1) << base;
  int found = 0;
  Key last = (Key)__builtin_inff();
  gap = (Key)__builtin_inff();
  // (Infinite keys are exact, as is the end of the keys: their NaN is no gap.)
  auto note = [&](Key v) {
    const Key m = OpMax{}(__builtin_fabsf(last), __builtin_fabsf(v));
    gap = __builtin_fminf(gap, __builtin_fmaf(-0x1p-23f, m, last - v));
    last = v;
  };
  for (int k = 0; k < p.top_k; ++k) {
    const Ord m = lane_reduce<Lanes>(h[0], OpMax{});
    const bool any = m > kNone;
    if constexpr (Gaps) note(key_at(m));
    const uint64_t eq = __ballot(h[0] == m) & mask;
    found += any;
    if (any && (int)__builtin_ctzll(eq) == self) {
      const int i = at[0];
      chosen[k] = {kHeld * lane + i, i == 0 ? s[0] : i == 1 ? s[1] : i == 2 ? s[2] : s[3]};
#pragma unroll
      for (int q = 0; q + 1 < kHeld; ++q) {
        h[q] = h[q + 1];
        at[q] = at[q + 1];
      }
      h[kHeld - 1] = kNone;
    }
  }
  if constexpr (Gaps) {
    const Ord m = lane_reduce<Lanes>(h[0], OpMax{});
    note(key_at(m));
  }
  return found;
}

// One group of Lanes lanes a token.  Scores: experts are ordered by score +
// bias, else by the logits themselves (the score increases with the logit, so
// this is the exact order of the scores).
//
// Score keys are defined in 64 bits.  They are first made in 32.  In units of
// 2^-24 of the row's largest score, a sigmoid is off by at most 8 (expf 4, the
// sum and the quotient 1 each, twice), a softmax score by 40 (the rounded
// difference in the exponent and expf 24, the sum over the experts 10, the
// divisor's reciprocal and product 3), and the sum with the bias by a unit of
// the key.  Scores below 2^-126 are 2^-149 apart and off by up to three such
// steps (expf 2, the quotient and a half sum of two the third), whatever their
// size.  If two keys whose order matters lie closer than twice all that, or
// two groups than their bounds allow, the wave decides again in 64 bits: with
// 256 experts, top 8, some four tokens in ten thousand are (softmax one).  The
// unit is that of the two keys: rounding is monotonic, so no expert behind them
// passes them by an error of its own size, and a large bias that switches an
// expert off (or forces it) sends no token to the 64 bits.
//
// Bound by the instructions of the rounds (about 30 of a wave each), not by
// the logits' bytes: 16384 tokens, top 8, softmax, us in a graph: 256 experts
// fp32 13.6 to 14.5 (3.4 for the bytes), 128 bf16 8.3 to 8.7, 64 fp32 5.6, 16
// bf16 4.6; with sigmoid scores, a bias and groups 26.5 to 28, 17 to 18, 12.4,
// 6.7 to 10.7, of which the bounds that decide between 32 and 64 bits are half
// a microsecond.  (Keys compared as floats and every score divided: 16.6 and
// 30 for 256.)  Four tokens of 256 experts with groups take 6.3, of which 3
// are a launch.
template <int DT, int Lanes, bool Scores>
__global__ void __launch_bounds__(kBlockThreads) moe_route_kernel(const RouteParams p) {
  constexpr int kTokens = kBlockThreads / Lanes;
  typedef typename std::conditional<Scores, double, float>::type Wide;
  __shared__ RouteScratch<Lanes, Wide> scratch[kTokens];
  __shared__ Chosen chosen_all[kTokens * SG_MAX_TOP_K];
  const int lane = threadIdx.x % Lanes, slot = threadIdx.x / Lanes;
  const int64_t t = block_index() * kTokens + slot;
  const bool live = t < p.T;  // lanes past the last token go along for the wave
  Chosen* const chosen = chosen_all + slot * SG_MAX_TOP_K;
  const float kNone = -__builtin_inff();

  float x[kHeld], s[kHeld], key[kHeld], b[kHeld];
  load_row4<DT>(p, t, kHeld * lane, live, x);
  if constexpr (Scores) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int e = kHeld * lane + i;
      b[i] = p.bias && e < p.E ? p.bias[e] : 0.0f;
    }
  }
  const float over = scores_of<Lanes>(x, p.score, s);
  float noise = 0.0f;  // the largest error of a score
#pragma unroll
  for (int i = 0; i < kHeld; ++i) key[i] = x[i];
  if constexpr (Scores) {
    const float inv = 1.0f / over;
    float top = 0.0f;  // the largest score
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const float v = s[i] * inv, k = v + b[i];
      key[i] = x[i] > kNone && k > kNone ? k : kNone;
      top = OpMax{}(top, v);
    }
    const float units = p.score == SG_SCORE_SIGMOID ? 8.0f : 40.0f;
    noise = 0x1p-24f * units * lane_reduce<Lanes>(top, OpMax{}) + kDenormalOff;
  }
  bool sure = true;
  if (p.n_groups > 1)
    sure = keep_groups<Lanes, Scores>(
        p, reinterpret_cast<RouteScratch<Lanes, float>&>(scratch[slot]), lane, key, noise);
  float gap;
  int found = choose<Lanes, Scores>(p, lane, key, s, chosen, gap);
  if constexpr (Scores) {
    if (__any(!sure || !(gap > 2 * noise))) {
      double wide[kHeld];
      const double div = scores_of<Lanes>(x, p.score, wide);
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const double k = wide[i] / div + (double)b[i];
        wide[i] = x[i] > kNone && k > (double)kNone ? k : (double)kNone;
      }
      wave_sync();
      if (p.n_groups > 1) keep_groups<Lanes, false>(p, scratch[slot], lane, wide);
      double ignored;
      found = choose<Lanes, false>(p, lane, wide, s, chosen, ignored);
    }
  }
  wave_sync();

  float sum = 0.0f;
  for (int k = lane; k < found; k += Lanes) {
    const float v = chosen[k].s / over;
    chosen[k].s = v;
    sum += v;
  }
  sum = lane_reduce<Lanes>(sum, OpSum{});
  const float div = p.renorm ? __builtin_fmaxf(sum, kTiny) : 1.0f;
  if (!live) return;
  for (int k = lane; k < p.top_k; k += Lanes) {
    const Chosen c = chosen[k];
    p.ids[t * p.top_k + k] = k < found ? c.id : -1;
    p.weights[t * p.top_k + k] = k < found ? c.s / div * p.scale : 0.0f;
  }
}

// With r_j = s_j / S (S = max(sum s, 2^-126) with renorm, else 1) and g_j the
// gradient of weight j times the scale, the gradient of expert id_j's score
// times that score is
//   u_j = r_j (g_j - [renorm, S above the floor] sum_i g_i r_i),
// and of the logits, summing u_j over the j that name the expert,
//   sigmoid  dx_e = u_e (1 - s_e),
//   softmax  dx_e = u_e - s_e sum_j u_j   (the sum is zero with renorm).
// Only ratios of scores appear, so small scores lose nothing; 1 - s_e is made
// from the logit, so that scores near one do not either.  Bound by
// memory: the gradient's rows are written whole; softmax reads the logits'
// rows, sigmoid only the chosen logits.  Lane j of a token's lanes handles its
// j-th expert and puts the result into the token's row in LDS; quad q of the
// lane holds experts from 4 * (q * Lanes + lane), so that a quad's loads and
// stores of neighbouring lanes adjoin.  16384 x 256 fp32, us in a graph:
// sigmoid 6.5, softmax 9.7, and 7.8 and 10.7 with three sets of rows in turn
// (both rows' bytes 6.7, one's written 3.4); every lane comparing every chosen
// id with its experts instead took 15.4 (with one quad).
struct Graded {
  int id;
  float s;     // the score, then its gradient u
  float rest;  // 1 - s of a sigmoid
};
template <int DT, int Lanes, int Quads>
__global__ void __launch_bounds__(kBlockThreads) moe_route_backward_kernel(
    const RouteParams p) {
  constexpr int kTokens = kBlockThreads / Lanes;
  __shared__ __attribute__((aligned(16))) float rows[kTokens][Quads * Lanes * kHeld];
  __shared__ Graded us_all[kTokens * SG_MAX_TOP_K];
  const int lane = threadIdx.x % Lanes, slot = threadIdx.x / Lanes;
  const int64_t t = block_index() * kTokens + slot;
  const bool live = t < p.T;
  auto first = [&](int q) { return kHeld * (q * Lanes + lane); };
  float* const row = rows[slot];
  Graded* const us = us_all + slot * SG_MAX_TOP_K;
  const bool soft = p.score == SG_SCORE_SOFTMAX;

  // Softmax: the row's largest logit and sum of exponentials.
  float s[Quads][kHeld] = {}, top = 0.0f, total = 1.0f;
  if (soft) {
    top = -__builtin_inff();
#pragma unroll
    for (int q = 0; q < Quads; ++q) {
      load_row4<DT>(p, t, first(q), live, s[q]);
      top = OpMax{}(top, lane_top(s[q]));
    }
    top = lane_reduce<Lanes>(top, OpMax{});
    total = 0.0f;
#pragma unroll
    for (int q = 0; q < Quads; ++q) {
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        s[q][i] = s[q][i] > -__builtin_inff() ? expf(s[q][i] - top) : 0.0f;
        part += s[q][i];
      }
      total += part;
    }
    total = __builtin_fmaxf(lane_reduce<Lanes>(total, OpSum{}), kTiny);
  }
#pragma unroll
  for (int q = 0; q < Quads; ++q) *reinterpret_cast<f32x4*>(row + first(q)) = f32x4{};

  // The chosen experts' scores, then their sum and mean gradient.
  float sum = 0.0f;
  for (int k = lane; k < p.top_k; k += Lanes) {
    const int id = live ? p.ids[t * p.top_k + k] : -1;
    float sk = 0.0f, rest = 0.0f;
    if ((uint32_t)id < (uint32_t)p.E) {
      const float xk = clean(load_logit<DT>(p.logits, t * p.ldl + id));
      if (xk > -__builtin_inff()) {
        const float z = expf(soft ? xk - top : -__builtin_fabsf(xk));
        const float under = soft ? total : 1.0f + z;
        sk = (soft || xk < 0 ? z : 1.0f) / under;
        rest = (xk < 0 ? 1.0f : z) / under;
      }
    }
    us[k] = {id, sk, rest};
    sum += sk;
  }
  sum = lane_reduce<Lanes>(sum, OpSum{});
  const bool floor = !(sum >= kTiny);
  const float div = !p.renorm ? 1.0f : floor ? kTiny : sum;
  float dot = 0.0f;
  for (int k = lane; k < p.top_k; k += Lanes)
    dot += us[k].s > 0.0f ? p.dweights[t * p.top_k + k] * p.scale * (us[k].s / div) : 0.0f;
  dot = lane_reduce<Lanes>(dot, OpSum{});
  const float mean = p.renorm && !floor ? dot : 0.0f;
  for (int k = lane; k < p.top_k; k += Lanes) {
    const float sk = us[k].s;
    float u = 0.0f;
    if (sk > 0.0f) {
      u = sk / div * (p.dweights[t * p.top_k + k] * p.scale - mean);
      if (!soft) u *= us[k].rest;
    }
    us[k].s = u;
  }
  wave_sync();
  // An expert named more than once takes the sum, in the order of its names.
  for (int k = lane; k < p.top_k; k += Lanes) {
    const int id = us[k].id;
    float u = 0.0f;
    for (int q = 0; q < p.top_k; ++q) u += us[q].id == id ? us[q].s : 0.0f;
    if ((uint32_t)id < (uint32_t)p.E) row[id] = u;
  }
  wave_sync();
  if (!live) return;
  const float all = p.renorm && !floor ? 0.0f : dot / total;
#pragma unroll
  for (int q = 0; q < Quads; ++q) {
    const int e0 = first(q);
    if (e0 >= p.E) return;
    f32x4 d = *reinterpret_cast<const f32x4*>(row + e0);
    if (soft)
#pragma unroll
      for (int i = 0; i < kHeld; ++i) d[i] -= s[q][i] * all;
    store_row4<DT>(p, t, e0, d);
  }
}

// ------------------------------------------------------------------ the plan
//
// A stable counting sort of the P = T * top_k ids in [0, E); the others have
// no place.  Each block owns a contiguous chunk of pairs, each of its waves a
// contiguous part of the chunk.  A pair's place is the count of smaller ids,
// of its id in earlier blocks, in earlier waves and in earlier lanes.  Lanes
// of a wave that hold the same id find each other by one ballot per bit of the
// id, which gives their order; no atomic decides a place, so the result is the
// same every time.
//
// The ballots make a step of 64 pairs about 100 instructions of a wave, so
// that many workgroups share them; counting takes a tenth.  Up to 16384 pairs
// each workgroup counts all ids by itself, beyond that a launch before counts
// them by chunks.  us in a graph, 8 | 256 experts, of which 3 are a launch:
// 256 pairs 3.1 | 3.3, 4096 4.3 | 4.8, 16384 6.6 | 7.2, 131072 6.8 | 9.2 (the
// pairs' bytes 0.3).  One workgroup for all 4096 took 6.0 | 7.3.

constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;
static_assert(SG_MAX_GROUPS == 256, "four experts a lane");

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
  __shared__ int bins[SG_MAX_GROUPS];
  if (threadIdx.x < SG_MAX_GROUPS) bins[threadIdx.x] = 0;
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * p.chunk;
  const int64_t c1 = c0 + p.chunk < p.P ? c0 + p.chunk : p.P;
  for (int64_t i = c0 + threadIdx.x; i < c1; i += kPlanThreads) {
    const int id = p.ids[i];
    if ((uint32_t)id < (uint32_t)p.E) atomicAdd(&bins[id], 1);  // counts: any order
  }
  __syncthreads();
  if ((int)threadIdx.x < p.E) p.counts[(int64_t)blockIdx.x * p.E + threadIdx.x] = bins[threadIdx.x];
}

// Counted: the chunks' counts are in p.counts; else a chunk is kPlanThreads
// pairs and the block counts the others' ids itself.
template <bool Counted>
__global__ void __launch_bounds__(kPlanThreads) moe_plan_place_kernel(const PlanParams p) {
  // One counter of an expert for each eighth lane, so that ids that are all
  // the same do not take 64 turns (8192 pairs of one expert 10.3 us with one).
  constexpr int kCopies = Counted ? 1 : 8;
  __shared__ int bins[kPlanWaves][SG_MAX_GROUPS];  // first counts, then next places
  __shared__ int earlier[SG_MAX_GROUPS][kCopies], others[SG_MAX_GROUPS][kCopies];
  __shared__ int wave_sum[kPlanWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int bits = 32 - __builtin_clz(2 * p.E - 1) - 1;  // of E - 1, none for one expert

  // Pairs, and sums of a chunk and its start, are below 2^32.
  const uint32_t P = (uint32_t)p.P, chunk = (uint32_t)p.chunk;
  const uint32_t block = blockIdx.x, blocks = gridDim.x;
  const uint32_t c0 = block * chunk, c1 = c0 + chunk < P ? c0 + chunk : P;
  const uint32_t per = chunk / kPlanWaves;  // a multiple of 64
  const uint32_t w0 = c0 + wave * per, w1 = w0 + per < c1 ? w0 + per : c1;
  auto id_at = [&](uint32_t i, uint32_t end) {
    const int id = i < end ? p.ids[i] : -1;
    return (uint32_t)id < (uint32_t)p.E ? id : -1;
  };
  int next = id_at(w0 + lane, w1);
  for (int e = tid; e < kPlanWaves * SG_MAX_GROUPS; e += kPlanThreads) (&bins[0][0])[e] = 0;
  if (blocks > 1)
    for (int e = tid; e < SG_MAX_GROUPS * kCopies; e += kPlanThreads)
      (&earlier[0][0])[e] = (&others[0][0])[e] = 0;
  __syncthreads();
  // The wave's own counts: the last lane of an id knows the first step's.
  uint64_t same = 0;
  if (w0 < w1) same = same_key(next, bits) & __ballot(next >= 0);
  if (next >= 0 && (same >> lane) == 1) bins[wave][next] = __builtin_popcountll(same);
  wave_sync();
  for (uint32_t b = w0 + 64; b < w1; b += 64) {
    const int id = id_at(b + lane, w1);
    if (id >= 0) atomicAdd(&bins[wave][id], 1);
  }
  // The other blocks' counts of each expert, and the earlier ones' among them.
  if constexpr (Counted) {
    // 2^bits threads a chunk's row, eight chunks' loads in flight.
    const int e = tid & ((1 << bits) - 1);
    const uint32_t step = kPlanThreads >> bits;
    int sum = 0, first = 0;
    for (uint32_t b0 = tid >> bits; b0 < blocks; b0 += 8 * step) {
      int v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t b = b0 + q * step;
        v[q] = p.counts[(b < blocks ? b : block) * (uint32_t)p.E + (e < p.E ? e : 0)];
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t b = b0 + q * step;
        sum += b < blocks && b != block ? v[q] : 0;
        first += b < block ? v[q] : 0;
      }
    }
    if (e < p.E) {
      atomicAdd(&others[e][0], sum);
      atomicAdd(&earlier[e][0], first);
    }
  } else {
    // Here `others` has the later blocks' alone until the sums below.
#pragma unroll 4
    for (uint32_t b = 0; b < blocks; ++b) {
      const int id = b == block ? -1 : id_at(b * kPlanThreads + tid, P);
      if (id >= 0) atomicAdd(&(b < block ? earlier : others)[id][tid % kCopies], 1);
    }
  }
  __syncthreads();

  // Expert tid's pairs: in all, and before this block; then the exclusive scan
  // over the experts (the first four waves).
  int total = 0, before = 0;
  if (tid < SG_MAX_GROUPS) {
    if (blocks > 1) {
#pragma unroll
      for (int c = 0; c < kCopies; ++c) {
        total += others[tid][c];
        before += earlier[tid][c];
      }
      if (!Counted) total += before;
    }
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) total += bins[w][tid];
  }
  int upto = total;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 63) wave_sum[wave] = upto;
  __syncthreads();
  const int last = wave_sum[0] + wave_sum[1] + wave_sum[2] + wave_sum[3];  // offsets[E]
  if (tid < SG_MAX_GROUPS) {
    int at = upto - total;
    for (int w = 0; w < wave; ++w) at += wave_sum[w];
    if (block == 0) {
      if (tid < p.E) p.offsets[tid] = at;
      if (tid == 0) p.offsets[p.E] = last;
    }
    at += before;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {  // counts of the waves become their first places
      const int c = bins[w][tid];
      bins[w][tid] = at;
      at += c;
    }
  }
  __syncthreads();

  for (uint32_t b = w0; b < w1; b += 64) {
    const uint32_t i = b + lane;
    const int id = next;
    const bool in = id >= 0;
    if (b > w0) same = same_key(id, bits) & __ballot(in);
    next = id_at(i + 64, w1);
    if (in) {
      const int place = bins[wave][id] + __builtin_popcountll(same & ((1ull << lane) - 1));
      // t = i / top_k, i below 2^31 (the multiplier is 2^32 (2^shift - top_k) / top_k + 1)
      const uint32_t t = (__umulhi(p.div_mul, i) + i) >> p.div_shift;
      p.slots[i] = place;
      if ((uint32_t)place < P) p.rows[place] = (int)t;
    } else if (i < w1) {
      p.slots[i] = -1;
    }
    if (i < w1 && i >= (uint32_t)last) p.rows[i] = -1;
    wave_sync();
    if (in && (same >> lane) == 1)  // the last lane of its id moves the place on
      bins[wave][id] += __builtin_popcountll(same);
    wave_sync();
  }
}

constexpr const char* dt_label(int dt) {
  return dt == SG_F32 ? "f32" : dt == SG_BF16 ? "bf16" : "f16";
}

dim3 route_grid(int64_t T, int lanes) {
  const int tokens = kBlockThreads / lanes;
  return grid_of((T + tokens - 1) / tokens);
}
constexpr const char* digits(int n) {
  return n == 1    ? "1"
         : n == 2  ? "2"
         : n == 4  ? "4"
         : n == 8  ? "8"
         : n == 16 ? "16"
         : n == 32 ? "32"
                   : "64";
}

template <int DT, int Lanes>
hipError_t go_route(const RouteParams& p, hipStream_t s) {
  static const char* const names[2] = {
      kernel_label("moe_route_kernel", dt_label(DT), digits(Lanes), "logits"),
      kernel_label("moe_route_kernel", dt_label(DT), digits(Lanes), "scores")};
  last_kernel() = names[p.by_score ? 1 : 0];
  const dim3 grid = route_grid(p.T, Lanes);
  if (p.by_score)
    hipLaunchKernelGGL((moe_route_kernel<DT, Lanes, true>), grid, dim3(kBlockThreads), 0, s, p);
  else
    hipLaunchKernelGGL((moe_route_kernel<DT, Lanes, false>), grid, dim3(kBlockThreads), 0, s, p);
  return hipGetLastError();
}

template <int DT, int Lanes, int Quads>
hipError_t go_back(const RouteParams& p, hipStream_t s) {
  static const char* const name =
      kernel_label("moe_route_backward_kernel", dt_label(DT), digits(Lanes), digits(Quads));
  last_kernel() = name;
  hipLaunchKernelGGL((moe_route_backward_kernel<DT, Lanes, Quads>), route_grid(p.T, Lanes),
                     dim3(kBlockThreads), 0, s, p);
  return hipGetLastError();
}

// The fewest lanes that hold a token's experts, four to a lane.  Eight a lane
// made the choice slower at every size: 4 tokens of 256 experts 4.0 -> 5.4 us,
// 16384 of 128 8.2 -> 9.5 us, a round having more to look at in one chain.
template <int DT>
hipError_t forward(const RouteParams& p, hipStream_t s) {
  if (p.E <= 32) return go_route<DT, 8>(p, s);
  if (p.E <= 64) return go_route<DT, 16>(p, s);
  if (p.E <= 128) return go_route<DT, 32>(p, s);
  return go_route<DT, 64>(p, s);
}

// The gradient takes one quad of experts a lane while its waves fit the card
// about at once, then fewer lanes with two or four, so that the short steps
// over the choice serve more tokens of a wave.  Microseconds with 1 | 2 | 4
// quads: 512 tokens of 256 fp32 softmax 4.0 | 4.3 | 5.0, 4096 5.3 | 5.0 | 5.5,
// 16384 12.3 | 10.1 | 9.7, sigmoid 9.1 | 7.2 | 6.5; 16384 of 128 bf16 softmax
// 6.8 | 5.7 | 5.9, 65536 19.4 | 14.2 | 12.9.
template <int DT>
hipError_t backward(const RouteParams& p, hipStream_t s) {
  if (p.E <= 32) return go_back<DT, 8, 1>(p, s);
  const int lanes = p.E <= 64 ? 16 : p.E <= 128 ? 32 : 64;
  const int64_t threads = p.T * lanes;
  if (threads < 1 << 18) {
    if (p.E <= 64) return go_back<DT, 16, 1>(p, s);
    if (p.E <= 128) return go_back<DT, 32, 1>(p, s);
    return go_back<DT, 64, 1>(p, s);
  }
  if (p.E <= 64) return go_back<DT, 8, 2>(p, s);
  if (threads < 1 << 20)
    return p.E <= 128 ? go_back<DT, 16, 2>(p, s) : go_back<DT, 32, 2>(p, s);
  return p.E <= 128 ? go_back<DT, 8, 4>(p, s) : go_back<DT, 16, 4>(p, s);
}

template <bool Back, int DT>
hipError_t either(const RouteParams& p, hipStream_t s) {
  if constexpr (Back)
    return backward<DT>(p, s);
  else
    return forward<DT>(p, s);
}

template <bool Back>
hipError_t by_type(int dtype, const RouteParams& p, hipStream_t s) {
  if (dtype == SG_F32) return either<Back, SG_F32>(p, s);
  if (dtype == SG_BF16) return either<Back, SG_BF16>(p, s);
  return either<Back, SG_F16>(p, s);
}

}  // namespace

hipError_t launch_moe_route(int dtype, const RouteParams& p, hipStream_t s) {
  return by_type<false>(dtype, p, s);
}

hipError_t launch_moe_route_backward(int dtype, const RouteParams& p, hipStream_t s) {
  return by_type<true>(dtype, p, s);
}

hipError_t launch_moe_plan(const PlanParams& p, hipStream_t s) {
  static const char* const names[2] = {kernel_label("moe_plan_place_kernel", "alone"),
                                       kernel_label("moe_plan_place_kernel", "counted")};
  const int blocks = (int)(p.P > 0 ? (p.P + p.chunk - 1) / p.chunk : 1);
  last_kernel() = names[p.counts ? 1 : 0];
  if (!p.counts) {
    hipLaunchKernelGGL((moe_plan_place_kernel<false>), dim3(blocks), dim3(kPlanThreads), 0, s, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(moe_plan_count_kernel, dim3(blocks), dim3(kPlanThreads), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_plan_place_kernel<true>), dim3(blocks), dim3(kPlanThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace sg
