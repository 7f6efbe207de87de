// xent.h -- softmax cross entropy over a vocabulary as epilogues of the 16-bit
// product z = alpha * A.B^T (A: tokens, B: one row per word):
//
//   lse[m] = log sum_n exp z[m][n],   loss[m] = lse[m] - z[m][t[m]],
//   g[m][n] = alpha * ((dloss[m] + dlse[m]) exp(z[m][n] - lse[m])
//                      - dloss[m] [n = t[m]]),   dA = g B,   dB = g^T A.
//
// The logits never leave the registers they were summed in.  Forward, a tile
// reduces each of its rows to the maximum and the sum of exponentials of its
// columns (XentStats), and a second kernel joins the tiles of a row in a fixed
// order.  Backward, the product runs again, its epilogue turns the logits into
// g in 16 bits (XentGrad) a run of words at a time, and two products of the
// library's own kernels take g to dA and dB.
#pragma once

#include <cfloat>

#include "deep64.h"
#include "lane_ops.h"
#include "pingpong16.h"

namespace sg {

constexpr float kLog2e = 1.44269504088896340736f;

struct XentParams {
  DenseParams d;   // the product (D: the gradient's workspace)
  XentJob x;       // pointers to row 0, column 0
  int64_t col0;    // the word of column 0
};

// What the join of a row's tiles and the gradient's preparation read.
struct XentRows {
  int64_t M, N;
  float alpha;
  const void* targets;
  bool wide;
  const float* part;   // [tiles][M][2]
  const float* zt;     // [M]
  int tiles;
  float* loss;
  float* lse;          // written by the join, read by the preparation
  const float* dloss;
  const float* dlse;   // or NULL
  float* rows;         // [M][4]
  float* scale;        // [1]: the factor that undoes the gradient's scale
  float2* most;        // [parts]: the largest factors
  int parts;
};

// A below itself, [2 M][K]: the tokens of a gradient in two parts.
struct XentTwice {
  const char* A;
  int64_t M, chunks, pitch;  // chunks of 16 bytes a row
  char* D;                   // or NULL: not wanted
};

// What the sum of dA's parts reads and writes.
struct XentSum {
  int64_t M, K, rows;
  int splits;
  const float* parts;
  const float* before;  // [M][K] or NULL
  const float* scale;
  void* D;
  int64_t ldd;
};

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// Token m's target as it lies in memory.  Two loads whatever its type: a branch
// would wait for each token's load before the next.
struct TargetWords {
  uint32_t low, high;  // (high: low again for 32-bit targets)
};
__device__ __forceinline__ TargetWords load_target(const void* t, bool wide, int64_t m) {
  const uint32_t* const p = static_cast<const uint32_t*>(t) + (wide ? 2 * m : m);
  return {p[0], p[wide ? 1 : 0]};
}

// The target, -1 where it is no word of [0, N).
__device__ __forceinline__ int target_of(const TargetWords& w, bool wide, int64_t N) {
  const int64_t v = wide ? (int64_t)((uint64_t)w.high << 32 | w.low) : (int64_t)(int32_t)w.low;
  return v >= 0 && v < N ? (int)v : -1;
}
__device__ __forceinline__ int target_of(const void* t, bool wide, int64_t m, int64_t N) {
  return target_of(load_target(t, wide, m), wide, N);
}

// (maximum, sum of exp(z - maximum)) of two sets of logits from those of each.
// A set without a finite logit has the maximum -inf and the sum 0, or NaN.
__device__ __forceinline__ void join_stats(float& m, float& s, float m2, float s2) {
  const float top = __builtin_fmaxf(m, m2);
  const float base = top == -__builtin_inff() ? 0.0f : top;
  s = s * exp2_of((m - base) * kLog2e) + s2 * exp2_of((m2 - base) * kLog2e);
  m = top;
}

// The scale of a gradient's terms: a power of two over the largest |dloss|
// (`most`; `top`: the largest |dloss| + |dloss + dlse|).  The largest weight, so
// all of a mean's, becomes that power of two and the gradient of its target, where
// the probability is small, rounds to it exactly; other weights take a rounding of
// fp32 here.  fp16's narrow range (2^-24 to 2^16) is used from 2^14 down.  The
// terms, with alpha, become dloss * up and so on; the products undo it by `down`
// in fp32.
struct XentScale {
  float up, down;
};
__device__ __forceinline__ XentScale scale_of(float alpha, float most, float top) {
  if (!(most > 0x1p-20f * top)) most = top;  // (dlse alone)
  const float a = __builtin_fabsf(alpha) * most;
  if (!(a >= FLT_MIN && a < 0x1p100f)) return {alpha, 1.0f};
  int e, em;
  frexpf(top / most, &e);  // top / most in [2^(e-1), 2^e)
  frexpf(most, &em);       // (`up` stays below 2^120, however small `most` is)
  const float size = ldexpf(1.0f, min(14 - e, em + 119));
  return {(alpha < 0 ? -size : size) / most, a / size};
}

// What a token's weights count for the scale: |dloss| and |dloss| + |dloss + dlse|,
// or nothing where one is no number, which only its own terms become then.
__device__ __forceinline__ float2 weight_of(float dl, float whole) {
  const float a = __builtin_fabsf(dl), b = __builtin_fabsf(whole);
  const bool on = a < __builtin_inff() && b < __builtin_inff();
  return make_float2(on ? a : 0.0f, on ? a + b : 0.0f);
}

// log2(e) lse, or +inf where that is no number: exp(z - lse) is then 0 for every
// logit, so that a factor of 0 stays 0 (lse is -inf where all logits are).
__device__ __forceinline__ float base_of(float lse) {
  return __builtin_fabsf(lse) < __builtin_inff() ? lse * kLog2e : __builtin_inff();
}

// The softmax's factor of a token's gradient: 0 where neither loss nor lse has a
// weight, whatever the token's logits are (padding may hold anything), else NaN
// where lse is no number.
__device__ __forceinline__ float softmax_factor(float dl, float whole, float up, float lse) {
  if (dl == 0.0f && whole == 0.0f) return 0.0f;
  return __builtin_fabsf(lse) < __builtin_inff() ? whole * up : __builtin_nanf("");
}

// Forward.
struct XentStats {
  // The maximum and sum of NV logits that lanes S apart (Steps) share a row of.
  template <int NV, bool Four>
  __device__ __forceinline__ static void reduce(const float (&v)[NV], float& m, float& s) {
    m = v[0];
#pragma unroll
    for (int e = 1; e < NV; ++e) m = __builtin_fmaxf(m, v[e]);
    if constexpr (Four) m = reduce_step<16>(m, OpMax{});
    m = reduce_step<32>(m, OpMax{});
    const float base = m == -__builtin_inff() ? 0.0f : m;
    s = 0.0f;
#pragma unroll
    for (int e = 0; e < NV; ++e) s += exp2_of((v[e] - base) * kLog2e);
    if constexpr (Four) s = reduce_step<16>(s, OpSum{});
    s = reduce_step<32>(s, OpSum{});
  }

  // Joins the waves' columns of each row (area: [waves][rows][2] floats) and
  // writes the tile's pair.
  template <int Waves, int Rows>
  __device__ __forceinline__ static void write(const TileJob& j, const float* area) {
    __syncthreads();
    const int r = threadIdx.x;
    if (r >= Rows || r >= j.m_valid) return;
    float m = area[2 * r], s = area[2 * r + 1];
#pragma unroll
    for (int w = 1; w < Waves; ++w)
      join_stats(m, s, area[2 * (w * Rows + r)], area[2 * (w * Rows + r) + 1]);
    *reinterpret_cast<float2*>(j.x.part + 2 * (int64_t)r) = make_float2(m, s);
  }

  // The column, inside the tile, of a target (or below 0, or past the tile).
  __device__ __forceinline__ static int column(const TileJob& j, const TargetWords& w) {
    const int64_t t = (int64_t)target_of(w, j.x.wide, j.x.words) - j.x.col0;
    return t >= 0 && t < 256 ? (int)t : -1;
  }
  // The target of tile row ml.
  __device__ __forceinline__ static TargetWords fetch(const TileJob& j, int ml) {
    return load_target(j.x.targets, j.x.wide, min(ml, j.m_valid - 1));
  }

  // The targets of a lane's rows, loaded before the mainloop so that their latency
  // is not the tile's last, and first looked at behind it.
  struct Rows16 {
    TargetWords t[8];
  };
  __device__ __forceinline__ static Rows16 fetch16(const TileJob& j, int lane, int g) {
    Rows16 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.t[i] = fetch(j, 128 * g + 16 * i + (lane & 15));
    return r;
  }
  template <int FM>
  struct Rows32 {
    TargetWords t[FM];
  };
  template <int FM, int WM>
  __device__ __forceinline__ static Rows32<FM> fetch32(const TileJob& j, int lane, int wm) {
    Rows32<FM> r;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) r.t[fm] = fetch(j, WM * wm + 32 * fm + (lane & 31));
    return r;
  }

  // Lane l of block (i, jn) holds row 128g + 16i + l%16, columns 64 w4 + 16 jn
  // + 4(l/16) .. +3.
  template <class Tile>
  __device__ __forceinline__ static void finish16(f32x4 (&acc)[Tile::kI][Tile::kJ],
                                                  const TileJob& j, const Rows16& rows, char* smem,
                                                  int, void*, int64_t, int lane, int g, int w4) {
    float* area = reinterpret_cast<float*>(smem);
    const int c0 = 64 * w4 + 4 * (lane >> 4);
    if (j.m_valid > 128 * g) {
#pragma unroll
      for (int i = 0; i < Tile::kI; ++i) {
        const int ml = 128 * g + 16 * i + (lane & 15);
        float v[4 * Tile::kJ];
#pragma unroll
        for (int jn = 0; jn < Tile::kJ; ++jn)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * jn + e] = acc[i][jn][e] * j.alpha;
        if (j.n_valid < 256) {
#pragma unroll
          for (int e = 0; e < 4 * Tile::kJ; ++e)
            if (c0 + 16 * (e >> 2) + (e & 3) >= j.n_valid) v[e] = -__builtin_inff();
        }
        const int at = column(j, rows.t[i]) - c0;  // 16 jn + e of the target
        if (at >= 0 && at < 64 && (at & 12) == 0 && ml < j.m_valid) {
          float z = 0.0f;
#pragma unroll
          for (int e = 0; e < 4 * Tile::kJ; ++e)
            if (at == 16 * (e >> 2) + (e & 3)) z = v[e];
          j.x.zt[ml] = z;
        }
        float m, s;
        reduce<4 * Tile::kJ, true>(v, m, s);
        if (lane < 16) *reinterpret_cast<float2*>(area + 2 * (256 * w4 + ml)) = make_float2(m, s);
      }
    }
    write<4, 256>(j, area);
  }

  // Lane l of block (fm, fn) holds row WM wm + 32 fm + l%32, columns WN wn +
  // 32 fn + 8q + 4(l/32) .. +3 in registers 4q .. 4q+3.
  template <int FM, int FN, int WM, int WN, int WavesN>
  __device__ __forceinline__ static void finish32(f32x16 (&acc)[FM][FN], const TileJob& j,
                                                  const Rows32<FM>& rows, char* smem, void*,
                                                  int64_t, int lane, int wm, int wn) {
    constexpr int kRows = 2 * WM;
    float* area = reinterpret_cast<float*>(smem);
    const int c0 = WN * wn + 4 * (lane >> 5);
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
      const int ml = WM * wm + 32 * fm + (lane & 31);
      float v[16 * FN];
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          v[16 * fn + r] = acc[fm][fn][r] * j.alpha;
          if (c0 + 32 * fn + 8 * (r >> 2) + (r & 3) >= j.n_valid)
            v[16 * fn + r] = -__builtin_inff();
        }
      const int at = column(j, rows.t[fm]) - c0;
      if (at >= 0 && at < WN && (at & 4) == 0 && ml < j.m_valid) {
        float z = 0.0f;
#pragma unroll
        for (int e = 0; e < 16 * FN; ++e)
          if (at == 32 * (e >> 4) + 8 * ((e >> 2) & 3) + (e & 3)) z = v[e];
        j.x.zt[ml] = z;
      }
      float m, s;
      reduce<16 * FN, false>(v, m, s);
      if (lane < 32)
        *reinterpret_cast<float2*>(area + 2 * (kRows * wn + ml)) = make_float2(m, s);
    }
    write<WavesN, kRows>(j, area);
  }
};

// Backward: the logits of a tile become the gradient in 16 bits, each value
// rounded once, by at most half a step of its own size, so that dA and dB are one
// 16-bit product each; a second part of every value (XentGradFew) would double
// both, 10 M N K operations for 6.  What the rounding costs depends on the
// weights, not on the number of tokens.  Equal ones make the targets' terms
// exact (XentScale); others round them too.  Errors over the norms of dA and dB
// against 64 bits, the results' own rounding being 0.00166 in bf16 and 0.00021
// in fp16 (65, 512 and 2048 tokens x 4000 x 512): equal weights 0.0017 to 0.0019
// and 0.00023 to 0.00025, weights uniform in [0, 1) 0.0022 and 0.00028, normal
// ones 0.0023 and 0.00029.  (8192 x 65536 x 4096 bf16, equal: 0.0018.)
template <int DD>
struct XentGrad {
  // Row terms: log2(e) lse, the factor of the softmax, what the target's column
  // loses, the target (the factors are zero for a token without a loss).
  struct Row {
    float l2, p, t;
    int at;
  };
  __device__ __forceinline__ static f32x4 fetch(const TileJob& j, int ml) {
    return *reinterpret_cast<const f32x4*>(j.x.rows + 4 * (int64_t)min(ml, j.m_valid - 1));
  }
  __device__ __forceinline__ static Row row_of(const TileJob& j, const f32x4& r) {
    const int t = __builtin_bit_cast(int, (float)r[3]);
    const int64_t at = (int64_t)t - j.x.col0;
    return {r[0], r[1], r[2], t >= 0 && at >= 0 && at < 256 ? (int)at : -1};
  }
  // (A logit of NaN counts as probability 0 here, and so do those of a row whose
  // lse is no number: the row has no weight, or the factor NaN.)
  __device__ __forceinline__ static float value(float acc, float k, const Row& r) {
    return r.p * exp2_of(__builtin_fmaxf(__builtin_fmaf(acc, k, -r.l2), -FLT_MAX));
  }

  // A lane's rows, loaded before the mainloop.
  struct Rows16 {
    f32x4 row[8];
  };
  __device__ __forceinline__ static Rows16 fetch16(const TileJob& j, int lane, int g) {
    Rows16 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.row[i] = fetch(j, 128 * g + 16 * i + (lane & 15));
    return r;
  }
  template <int FM>
  struct Rows32 {
    f32x4 row[FM];
  };
  template <int FM, int WM>
  __device__ __forceinline__ static Rows32<FM> fetch32(const TileJob& j, int lane, int wm) {
    Rows32<FM> r;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) r.row[fm] = fetch(j, WM * wm + 32 * fm + (lane & 31));
    return r;
  }

  template <class Tile>
  __device__ __forceinline__ static void finish16(f32x4 (&acc)[Tile::kI][Tile::kJ],
                                                  const TileJob& j, const Rows16& rows, char* smem,
                                                  int T, void* D, int64_t ldd, int lane, int g,
                                                  int w4) {
    if (j.m_valid <= 128 * g) return;
    const int c0 = 64 * w4 + 4 * (lane >> 4);
    const float k = j.alpha * kLog2e;
#pragma unroll
    for (int i = 0; i < Tile::kI; ++i) {
      const Row r = row_of(j, rows.row[i]);
#pragma unroll
      for (int jn = 0; jn < Tile::kJ; ++jn)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][jn][e] = value(acc[i][jn][e], k, r);
      const int at = r.at - c0;
      if (at >= 0 && at < 64 && (at & 12) == 0) {
#pragma unroll
        for (int jn = 0; jn < Tile::kJ; ++jn)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (at == 16 * jn + e) acc[i][jn][e] -= r.t;
      }
      if (j.n_valid < 256) {
#pragma unroll
        for (int jn = 0; jn < Tile::kJ; ++jn)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c0 + 16 * jn + e >= j.n_valid) acc[i][jn][e] = 0.0f;
      }
    }
    TileJob out = j;
    out.alpha = 1.0f;
    out.n_valid = j.x.n_store;
    char* cq[4];
    cblock_quarters(cq, smem, T, g, Tile::kTileBytes, Tile::kHalfBytes);
    Tile::template epilogue_lds_t<SG_NONE, DD>(acc, out, cq, D, ldd, lane, g, w4);
  }

  // Four columns, from c on, of tile row ml: the gradient in place of the sums
  // (zero past the words).
  __device__ __forceinline__ static f32x4 values(const f32x16& acc, int q, float k, const Row& r,
                                                 const TileJob& j, int c) {
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = value(acc[4 * q + e], k, r);
      if (r.at == c + e) v[e] -= r.t;
      if (c + e >= j.n_valid) v[e] = 0.0f;
    }
    return v;
  }

  template <int FM, int FN, int WM, int WN, int WavesN>
  __device__ __forceinline__ static void finish32(f32x16 (&acc)[FM][FN], const TileJob& j,
                                                  const Rows32<FM>& rows, char*, void* D,
                                                  int64_t ldd, int lane, int wm, int wn) {
    const int c0 = WN * wn + 4 * (lane >> 5);
    const float k = j.alpha * kLog2e;
    const u32x2 none{};
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
      const int ml = WM * wm + 32 * fm + (lane & 31);
      if (ml >= j.m_valid) continue;
      const Row r = row_of(j, rows.row[fm]);
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = c0 + 32 * fn + 8 * q;
          if (c >= j.x.n_store) continue;
          store_d_chunk<SG_NONE, DD>(values(acc[fm][fn], q, k, r, j, c), none, D,
                                     (j.d_row0 + ml) * ldd + j.n0 + c, 1.0f, 0.0f);
        }
    }
  }
};

// The same for up to 64 tokens, all in one tile: what the rounding took away is
// kept as a second 16-bit number, `low` further on, and the products add both, so
// that dA and dB are as exact as their own rounding (0.00166 of the norm in bf16,
// where one part gives 0.0020 to 0.0023 with random weights).  Here that is
// cheap, as the time goes into reading B and writing dB (us with | without it:
// 8 x 32000 x 4096 175 | 176, 32 of them 193 | 181, 64 210 | 195, 64 x 8192 x
// 1024 28.3 | 27.0, 64 x 50257 x 768 80 | 66).  Every wave
// makes the tokens' terms for itself, lane l those of token l.
template <int DD>
struct XentGradFew {
  using Grad = XentGrad<DD>;
  template <int FM>
  struct Rows32 {
    TargetWords t;
    float dloss, dlse, lse;
  };
  template <int FM, int WM>
  __device__ __forceinline__ static Rows32<FM> fetch32(const TileJob& j, int lane, int) {
    const int m = min(lane, j.m_valid - 1);
    return {load_target(j.x.targets, j.x.wide, m), j.x.dloss[m],
            (j.x.dlse ? j.x.dlse : j.x.dloss)[m], j.x.lse[m]};
  }
  __device__ __forceinline__ static typename Grad::Row row_of(const TileJob& j,
                                                              const Rows32<1>& own, int ml) {
    const int t = target_of(own.t, j.x.wide, j.x.words);
    const float dl = t >= 0 ? own.dloss : 0.0f;
    const float whole = j.x.dlse ? dl + own.dlse : dl;
    const float2 size = weight_of(dl, whole);
    const XentScale f = scale_of(j.alpha, lane_reduce<64>(size.x, OpMax{}),
                                 lane_reduce<64>(size.y, OpMax{}));
    if (j.x.col0 == 0 && threadIdx.x == 0) j.x.scale[0] = f.down;
    const int64_t at = (int64_t)t - j.x.col0;
    const int in = t >= 0 && at >= 0 && at < 256 ? (int)at : -1;
    return {__shfl(base_of(own.lse), ml), __shfl(softmax_factor(dl, whole, f.up, own.lse), ml),
            __shfl(dl * f.up, ml), __shfl(in, ml)};
  }

  template <int FM, int FN, int WM, int WN, int WavesN>
  __device__ __forceinline__ static void finish32(f32x16 (&acc)[FM][FN], const TileJob& j,
                                                  const Rows32<FM>& own, char*, void* D,
                                                  int64_t ldd, int lane, int wm, int wn) {
    static_assert(FM == 1 && FN == 1 && 2 * WM == kWaveSize, "a row for each lane");
    const int ml = WM * wm + (lane & 31), c0 = WN * wn + 4 * (lane >> 5);
    const float k = j.alpha * kLog2e;
    const typename Grad::Row r = row_of(j, own, ml);
    if (ml >= j.m_valid) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = c0 + 8 * q;
      if (c >= j.x.n_store) continue;
      f32x4 v = Grad::values(acc[0][0], q, k, r, j, c);
      uint16_t* const d = static_cast<uint16_t*>(D) + (j.d_row0 + ml) * ldd + j.n0 + c;
      const u32x2 high = pack_d16<DD>(v);
      *reinterpret_cast<u32x2*>(d) = high;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t h = (e & 1) ? high[e / 2] >> 16 : high[e / 2] & 0xffffu;
        v[e] -= DD == SG_BF16 ? bf16_to_f32(h) : f16_to_f32(h);
      }
      *reinterpret_cast<u32x2*>(d + j.x.low) = pack_d16<DD>(v);
    }
  }
};

template <int BM>
__device__ __forceinline__ TileJob xent_job(const XentParams& p, int wg) {
  TileJob j = dense_tile_job<BM, BM, false, false>(p.d, wg);
  const int64_t m0 = j.d_row0;
  j.x = p.x;
  j.x.col0 = p.col0 + j.n0;
  j.x.targets = static_cast<const char*>(p.x.targets) + m0 * (p.x.wide ? 8 : 4);
  j.x.part = p.x.part + 2 * ((j.n0 / BM) * p.d.M + m0);
  j.x.zt = p.x.zt + m0;
  j.x.rows = p.x.rows + 4 * m0;
  j.x.n_store = (int)min<int64_t>(BM, p.x.n_store - j.n0);
  return j;
}

// Tail: K is no multiple of 64.
template <bool BF, class Epi, bool Tail>
__global__ void __launch_bounds__(512, 1) xent_pingpong_kernel(const XentParams p) {
  using Tile = PingPong16Tile<BF, kSwzDefault, false, false, true, false, Epi, Tail>;
  __shared__ __attribute__((aligned(4096))) char smem[Tile::kLdsBytes];
  const ClockStamp cs = clock_begin(p.d.clk);
  const TileJob j = xent_job<256>(p, blockIdx.x);
  Tile::run(smem, j, p.d.K, nullptr, SG_NONE, p.d.D, p.d.d_dtype, p.d.ldd);
  clock_end(p.d.clk, cs);
}

// 64x64 and 128x128 tiles with a ring of five stages: 80 KiB of LDS, two
// workgroups a CU, or 160.  (The eight stages that plain products of 64x64 tiles
// run, one workgroup a CU: 4 x 32768 x 2048 with B in memory 37.9 us against
// 34.9, 4 x 65536 x 2048 69 against 60; four stages 36.4 and 68.)
template <int BM, bool BF, class Epi>
__global__ void __launch_bounds__(256, 1) xent_deep_kernel(const XentParams p) {
  using Tile = DeepTile<BM, BF, false, false, Epi, 5>;
  __shared__ __attribute__((aligned(4096))) char smem[Tile::kLdsBytes];
  const ClockStamp cs = clock_begin(p.d.clk);
  const TileJob j = xent_job<BM>(p, blockIdx.x);
  Tile::run(smem, j, p.d.K, nullptr, SG_NONE, p.d.D, p.d.d_dtype, p.d.ldd);
  clock_end(p.d.clk, cs);
}

// 128x128 tiles beyond one round of the CUs: two workgroups a CU.
template <bool BF, class Epi>
__global__ void __launch_bounds__(256, 1) xent_dense_kernel(const XentParams p) {
  using Tile = GemmTile<128, 128, BF, false, false, kSwzDefault, 4, Epi>;
  __shared__ __attribute__((aligned(4096))) char s0[Tile::kStageBytes];
  __shared__ __attribute__((aligned(4096))) char s1[Tile::kStageBytes];
  const ClockStamp cs = clock_begin(p.d.clk);
  const TileJob j = xent_job<128>(p, blockIdx.x);
  Tile::run(s0, s1, j, p.d.K, nullptr, SG_NONE, p.d.D, p.d.d_dtype, p.d.ldd);
  clock_end(p.d.clk, cs);
}

}  // namespace sg
