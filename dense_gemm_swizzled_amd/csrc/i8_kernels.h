// i8_kernels.h -- the product of 8-bit integer matrices with a scale per row
// of A (token) and per row of B (output channel),
//
//   D[m][n] = (sum_k A[m][k] * B[n][k]) * SA[m] * SB[n],
//
// dense, and grouped over experts whose row ranges lie in device memory.
//
// The sum is exact: products are at most 2^14 and K at most 131056, so every
// partial sum stays below 2^31 and neither the order of the additions nor the
// split of K changes the result.  A K tile of the 16-bit kernels is 128 bytes
// of a row whatever the element, and v_mfma_i32_16x16x64_i8 and
// v_mfma_i32_32x32x32_i8 take the same 16 bytes a lane as their 16-bit
// counterparts in the same cycles, so large products run the mainloops of
// pingpong16.h and deep64.h (Elem = kElemI8) at twice the operations per
// byte.  Products of few rows are bound by reading B once and run
// i8_skinny_kernel below.
#pragma once

#include "deep64.h"
#include "i8_params.h"
#include "pingpong16.h"

namespace sg {

// The panels of the tile at D row row0 (m_valid rows) and column n0 (bn wide).
template <bool Rows>
__device__ __forceinline__ TileJob i8_job(const I8Params& p, int64_t row0, int m_valid,
                                          int64_t n0, int bn, int g) {
  TileJob j;
  j.m_valid = m_valid;
  j.n_valid = (int)min<int64_t>(bn, p.N - n0);
  if constexpr (Rows) {
    j.a = static_cast<const char*>(p.A);
    j.a_bytes = p.K > 0 && p.a_total > 0 ? (uint32_t)((p.a_total - 1) * p.lda + p.K) : 0u;
    j.rows = p.rows + row0;
    j.a_total = p.a_total;
    j.sa = p.SA;
  } else {
    j.a = static_cast<const char*>(p.A) + row0 * p.lda;
    j.a_bytes = p.K > 0 ? (uint32_t)((m_valid - 1) * p.lda + p.K) : 0u;
    j.rows = nullptr;
    j.a_total = 0;
    j.sa = p.SA + row0;
  }
  j.a_pitch = (uint32_t)p.lda;
  j.b = static_cast<const char*>(p.B) + ((int64_t)g * p.N + n0) * p.ldb;
  j.b_bytes = p.K > 0 ? (uint32_t)((j.n_valid - 1) * p.ldb + p.K) : 0u;
  j.b_pitch = (uint32_t)p.ldb;
  j.sb = p.SB + (int64_t)g * p.N + n0;
  j.d_row0 = row0;
  j.n0 = n0;
  j.ldc = 0;
  j.alpha = 1.0f;
  j.beta = 0.0f;
  j.vec = p.vec;
  return j;
}

template <int BM>
__device__ __forceinline__ TileJob i8_dense_job(const I8Params& p, int wg, int bn) {
  const int t = xcd_remap(wg, p.tiles_m * p.tiles_n);
  int tm, tn;
  raster(t, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
  const int64_t m0 = (int64_t)tm * BM;
  return i8_job<false>(p, m0, (int)min<int64_t>(BM, p.M - m0), (int64_t)tn * bn, bn, 0);
}

// The tile of workgroup `wg` among the groups' tiles, found from the offsets
// in device memory: lane l adds up the row tiles of groups 4l .. 4l+3, a scan
// over the wave places them, and the lane whose range holds the tile names
// the group.  About a microsecond of latency against a host round trip for
// the offsets.  Offsets outside [0, M] are clamped and a decreasing pair is
// an empty group, so no offsets make the kernel leave its buffers; tiles that
// such offsets add beyond the grid are not computed.  False: no tile.
template <int BM, bool Rows>
__device__ __forceinline__ bool i8_grouped_job(const I8Params& p, int wg, TileJob& j, int bn) {
  const int lane = threadIdx.x & 63;
  const int R = (int)p.M;
  int lo[5], tiles[4], mine = 0;
#pragma unroll
  for (int i = 0; i < 5; ++i) lo[i] = min(max(p.offsets[min(4 * lane + i, p.G)], 0), R);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    tiles[i] = (max(lo[i + 1] - lo[i], 0) + BM - 1) / BM;
    mine += tiles[i];
  }
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  const int64_t total64 =
      (int64_t)__builtin_amdgcn_readlane(upto, 63) * p.tiles_n;
  const int total = (int)min<int64_t>(total64, gridDim.x);
  if (wg >= total) return false;
  const int t = xcd_remap(wg, total);
  const int tr = t / p.tiles_n;  // row tile, counted over all groups
  const uint64_t holds = __ballot(tr >= upto - mine && tr < upto);
  const int who = (int)__builtin_ctzll(holds);
  int first = __builtin_amdgcn_readlane(upto - mine, who);
  int g = 4 * who, row0 = 0, rows_g = 0, tiles_g = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = __builtin_amdgcn_readlane(tiles[i], who);
    const int a = __builtin_amdgcn_readlane(lo[i], who);
    const int b = __builtin_amdgcn_readlane(lo[i + 1], who);
    if (tiles_g == 0) {
      if (tr < first + n) {
        g = 4 * who + i;
        row0 = a;
        rows_g = b - a;
        tiles_g = n;
      } else {
        first += n;
      }
    }
  }
  int tm, tn;
  raster(t - first * p.tiles_n, tiles_g, p.tiles_n, p.group_m, tm, tn);
  const int m0 = tm * BM;
  j = i8_job<Rows>(p, (int64_t)row0 + m0, min(BM, rows_g - m0), (int64_t)tn * bn, bn, g);
  return true;
}

// ---- large and middle sizes: the mainloops of the 16-bit kernels, K in pairs

template <bool Grouped, bool Rows>
__global__ void __launch_bounds__(512, 1) i8_pingpong_kernel(const I8Params p) {
  using Tile = PingPong16Tile<kElemI8, kSwzDefault, false, false, true, Rows>;
  __shared__ __attribute__((aligned(4096))) char smem[Tile::kLdsBytes];
  const ClockStamp cs = clock_begin(p.clk);
  TileJob j;
  if constexpr (Grouped) {
    if (!i8_grouped_job<256, Rows>(p, blockIdx.x, j, 256)) return;
  } else {
    j = i8_dense_job<256>(p, blockIdx.x, 256);
  }
  Tile::run(smem, j, p.K / 2, nullptr, SG_NONE, p.D, p.d_dtype, p.ldd);
  clock_end(p.clk, cs);
}

template <int BM, bool Grouped, bool Rows>
__global__ void __launch_bounds__(256, 1) i8_deep_kernel(const I8Params p) {
  using Tile = DeepTile<BM, kElemI8, false, false, Rows>;
  __shared__ __attribute__((aligned(4096))) char smem[Tile::kLdsBytes];
  const ClockStamp cs = clock_begin(p.clk);
  TileJob j;
  if constexpr (Grouped) {
    if (!i8_grouped_job<BM, Rows>(p, blockIdx.x, j, BM)) return;
  } else {
    j = i8_dense_job<BM>(p, blockIdx.x, BM);
  }
  Tile::run(smem, j, p.K / 2, nullptr, SG_NONE, p.D, p.d_dtype, p.ldd);
  clock_end(p.clk, cs);
}

// ---- few rows

// 16*MT rows by 16*NT*(8/wk) columns.  Bound by the bytes of B, which every
// row tile reads once and no two waves share, so B goes from memory to the
// MFMA operands through registers (lane l: row l%16, 16 bytes at 16(l/16) of
// a 64-byte K step) with two stages of U steps in flight per wave.  wk of the
// eight waves split K among them and add their integer sums through LDS.
template <int MT, int NT>
struct SkinnyTile {
  static constexpr int kU = MT * NT == 1 ? 4 : MT * NT <= 4 ? 2 : 1;
  struct Stage {
    u32x4 a[kU][MT], b[kU][NT];
  };
  static constexpr int kBlocks = MT * NT;
  static constexpr int kLdsBytes = 8 * kBlocks * 1024;

  template <bool Rows>
  __device__ __forceinline__ static void run(char* smem, const TileJob& j, const I8Params& p) {
    const int tid = threadIdx.x;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4;
    const int wk = p.wk, part = wave & (wk - 1), nb = wave / wk * (16 * NT);
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(j.a, j.a_bytes), rb = make_rsrc(j.b, j.b_bytes);
    uint32_t ao[MT], bo[NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int m = 16 * mt + r;
      ao[mt] = kOutOfRange;
      if (m < j.m_valid) {
        const int src = Rows ? j.rows[m] : m;
        if (!Rows || (uint32_t)src < (uint32_t)j.a_total)
          ao[mt] = (uint32_t)src * j.a_pitch + 16u * (uint32_t)c;
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = nb + 16 * nt + r;
      bo[nt] = n < j.n_valid ? (uint32_t)n * j.b_pitch + 16u * (uint32_t)c : kOutOfRange;
    }
    f32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = f32x4{};

    const int steps = (int)((p.K + 63) >> 6);
    const int s0 = steps * part / wk, s1 = steps * (part + 1) / wk;
    const uint32_t kend = (uint32_t)p.K - 16u * (uint32_t)c;  // K is a multiple of 16
    auto load = [&](Stage& f, int s) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t k = 64u * (uint32_t)(s + u);
        const bool ok = s + u < s1 && (int)k < (int)kend;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          f.b[u][nt] = buffer_load16(rb, ok ? bo[nt] + k : kOutOfRange);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          f.a[u][mt] = buffer_load16(ra, ok ? ao[mt] + k : kOutOfRange);
      }
    };
    auto mma = [&](const Stage& f) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            acc[mt][nt] = mfma16x16x32<kElemI8>(f.b[u][nt], f.a[u][mt], acc[mt][nt]);
    };
    Stage f0, f1;
    load(f0, s0);
    for (int s = s0; s < s1; s += 2 * kU) {
      load(f1, s + kU);
      mma(f0);
      load(f0, s + 2 * kU);
      mma(f1);
    }

    // Lane l of a block holds columns 4c .. 4c+3 of row l%16.  Block b's sums
    // over the wk waves are finished by wave b mod wk of them.
    if (wk > 1) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
        lds_write16(smem, (uint32_t)((wave * kBlocks + b) * 1024 + 16 * lane),
                    __builtin_bit_cast(u32x4, acc[b / NT][b % NT]));
      __syncthreads();
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      if (b % wk != part) continue;
      i32x4 v = __builtin_bit_cast(i32x4, acc[b / NT][b % NT]);
      if (wk > 1) {
        v = i32x4{};
        for (int w = 0; w < wk; ++w) {
          const u32x4 o = lds_read16(
              smem, (uint32_t)(((wave - part + w) * kBlocks + b) * 1024 + 16 * lane));
          v += __builtin_bit_cast(i32x4, o);
        }
      }
      const int ml = 16 * (b / NT) + r, nl = nb + 16 * (b % NT) + 4 * c;
      if (ml >= j.m_valid || nl >= j.n_valid) continue;
      float sb[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) sb[e] = j.sb[min(nl + e, j.n_valid - 1)];
      const f32x4 d = i8_scale4(__builtin_bit_cast(f32x4, v), i8_row_scale<Rows>(j, ml), sb);
      store_i8_chunk(d, p.D, p.d_dtype, (j.d_row0 + ml) * p.ldd + j.n0 + nl, j.n_valid - nl,
                     j.vec);
    }
  }
};

template <int MT, int NT, bool Grouped, bool Rows>
__global__ void __launch_bounds__(512, 1) i8_skinny_kernel(const I8Params p) {
  using Tile = SkinnyTile<MT, NT>;
  __shared__ __attribute__((aligned(16))) char smem[Tile::kLdsBytes];
  const ClockStamp cs = clock_begin(p.clk);
  const int bn = 16 * NT * 8 / p.wk;
  TileJob j;
  if constexpr (Grouped) {
    if (!i8_grouped_job<16 * MT, Rows>(p, blockIdx.x, j, bn)) return;
  } else {
    j = i8_dense_job<16 * MT>(p, blockIdx.x, bn);
  }
  Tile::template run<Rows>(smem, j, p);
  clock_end(p.clk, cs);
}

}  // namespace sg
