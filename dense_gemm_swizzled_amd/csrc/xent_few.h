// xent_few.h -- the cross entropy's product for up to 64 tokens, bound by
// reading the vocabulary's matrix B once.
//
// A workgroup's eight waves take 16 CT words each and all of K, so a word's
// logits are whole in one wave's registers and no wave waits for another's
// words.  B goes from memory straight into the registers that the matrix
// instruction reads, 16 loads of 1 KiB ahead a wave (128 KiB a CU), A (up to
// 64 tokens) lies in LDS in runs of K.  Lane l takes row l%16 of a block and, of
// each 128 bytes of a row, bytes [32 (l/16), +32) for two instructions: A and B
// agree on that order, so the sum does not depend on it, and the two loads of a
// lane use up the line together.
#pragma once

#include "xent.h"

namespace sg {

template <bool BF, int MT, int CT>
struct XentFewTile {
  static constexpr int kRows = 16 * MT, kCols = 128 * CT;  // of a workgroup
  static constexpr int kAhead = 8 / CT;                    // units of 64 k in flight
  static constexpr int kRunK = 4096 / MT;                  // k of A in LDS
  // (rows 16 bytes longer than a multiple of the banks' 256: the 16 rows of a
  // read start in different banks)
  static constexpr int kPitch = 2 * kRunK + 16;
  static constexpr int kLdsBytes = kRows * kPitch;
  static_assert(kLdsBytes <= 163840 && kLdsBytes >= 8 * kRows * 8, "A's run, then the pairs");

  f32x4 acc[CT][MT];

  __device__ __forceinline__ void run(char* smem, const XentParams& p, int64_t n0) {
    const int tid = threadIdx.x;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4;
    const int64_t K = p.d.K;
    const int64_t first = n0 + 16 * CT * wave;
    const int words = (int)max<int64_t>(0, min<int64_t>(16 * CT, p.d.N - first));
    const uint32_t pitch = (uint32_t)(2 * p.d.ldb), kbytes = (uint32_t)(2 * K);
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(
        static_cast<const char*>(p.d.B) + (words ? first : 0) * p.d.ldb * 2,
        words ? (uint32_t)(words - 1) * pitch + kbytes : 0u);
    uint32_t voff[CT];
#pragma unroll
    for (int i = 0; i < CT; ++i)
      voff[i] = 16 * i + r < words ? (uint32_t)(16 * i + r) * pitch + 32u * (uint32_t)c
                                   : kOutOfRange;
    u32x4 b[kAhead][CT][2];
    auto load = [&](int s, int u) {
      const uint32_t k = 128u * (uint32_t)u;
#pragma unroll
      for (int i = 0; i < CT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t at = k + 16u * (uint32_t)h;
          b[s][i][h] = buffer_load16(
              rb, at + 32u * (uint32_t)c < kbytes && voff[i] != kOutOfRange ? voff[i] + at
                                                                          : kOutOfRange);
        }
    };
    // A's next run of K, 16 chunks of 16 bytes a thread, loaded while the run
    // before is multiplied; zeros past K and M.
    constexpr int kRunUnits = kRunK / 64, kChunks = kRunK / 8, kEach = kRows * kChunks / 512;
    static_assert(kEach == 16, "a run's chunks");
    u32x4 stage[kEach];
    auto fetch = [&](int u0) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int row = (tid + 512 * i) / kChunks, q = (tid + 512 * i) % kChunks;
        const int64_t k = 64 * (int64_t)u0 + 8 * q;
        stage[i] = row < p.d.M && k < K
                       ? *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.d.A) +
                                                         row * p.d.lda + k)
                       : u32x4{};
      }
    };
    auto commit = [&]() {
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        lds_write16(smem, (uint32_t)((tid + 512 * i) / kChunks * kPitch +
                                     (tid + 512 * i) % kChunks * 16), stage[i]);
    };
#pragma unroll
    for (int i = 0; i < CT; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[i][m] = f32x4{};
    const int units = (int)((K + 63) / 64);
    fetch(0);
#pragma unroll
    for (int s = 0; s < kAhead; ++s) load(s, s);

    for (int u0 = 0; u0 < units; u0 += kRunUnits) {
      if (u0) __syncthreads();  // every wave has read the run before
      commit();
      __syncthreads();
      if (u0 + kRunUnits < units) fetch(u0 + kRunUnits);
      const int run = min(kRunUnits, units - u0);
      for (int u = 0; u < run; u += kAhead) {
#pragma unroll
        for (int s = 0; s < kAhead; ++s) {
          if (u + s >= run) break;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            u32x4 a[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m)
              a[m] = lds_read16(smem, (uint32_t)((16 * m + r) * kPitch + 128 * (u + s) + 32 * c +
                                                 16 * h));
#pragma unroll
            for (int i = 0; i < CT; ++i)
#pragma unroll
              for (int m = 0; m < MT; ++m)
                acc[i][m] = mfma16x16x32<BF>(b[s][i][h], a[m], acc[i][m]);
          }
          load(s, u0 + u + s + kAhead);
        }
      }
    }
  }
};

// Lane l of block (i, m) holds words 16 i + 4(l/16) .. +3 of the wave's for token
// 16 m + l%16.
template <bool BF, int MT, int CT>
__global__ void __launch_bounds__(512, 1) xent_few_stats_kernel(const XentParams p) {
  using Tile = XentFewTile<BF, MT, CT>;
  __shared__ __attribute__((aligned(16))) char smem[Tile::kLdsBytes];
  const int64_t n0 = (int64_t)blockIdx.x * Tile::kCols;
  Tile tile;
  tile.run(smem, p, n0);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  TileJob j{};
  j.m_valid = (int)p.d.M;
  j.alpha = p.d.alpha;
  j.x = p.x;
  j.x.col0 = n0 + 16 * CT * wave + 4 * (lane >> 4);
  j.x.part = p.x.part + 2 * (int64_t)blockIdx.x * p.d.M;
  __syncthreads();  // every read of A is done
  float* area = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int ml = 16 * m + (lane & 15);
    const int at = XentStats::column(j, ml);
    float v[4 * CT];
#pragma unroll
    for (int e = 0; e < 4 * CT; ++e) {
      const int n = 16 * (e >> 2) + (e & 3);
      v[e] = tile.acc[e >> 2][m][e & 3] * j.alpha;
      if (j.x.col0 + n >= p.d.N) v[e] = -__builtin_inff();
      if (at == n && ml < j.m_valid) j.x.zt[ml] = v[e];
    }
    float top, sum;
    XentStats::reduce<4 * CT, true>(v, top, sum);
    if (lane < 16)
      *reinterpret_cast<float2*>(area + 2 * (Tile::kRows * wave + ml)) = make_float2(top, sum);
  }
  XentStats::write<8, Tile::kRows>(j, area);
}

// The gradient of the logits as the sum of two 16-bit numbers (rows m and M +
// m), which holds 16 bits of it (fp16: 22): with few tokens the rounding of one
// number would not average out, and the products are not what takes the time.
template <bool BF, int MT, int CT>
__global__ void __launch_bounds__(512, 1) xent_few_grad_kernel(const XentParams p) {
  constexpr int DD = BF ? SG_BF16 : SG_F16;
  using Tile = XentFewTile<BF, MT, CT>;
  using Grad = XentGrad<DD>;
  __shared__ __attribute__((aligned(16))) char smem[Tile::kLdsBytes];
  const int64_t n0 = (int64_t)blockIdx.x * Tile::kCols;
  Tile tile;
  tile.run(smem, p, n0);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  TileJob j{};
  j.m_valid = (int)p.d.M;
  j.x = p.x;
  const int64_t first = n0 + 16 * CT * wave + 4 * (lane >> 4);
  j.x.col0 = p.col0 + first;
  const float k = p.d.alpha * kLog2e;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int ml = 16 * m + (lane & 15);
    if (ml >= j.m_valid) continue;
    const typename Grad::Row r = Grad::row_of(j, ml);
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      if (first + 16 * i >= p.x.n_store) continue;
      f32x4 g, rest;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = Grad::value(tile.acc[i][m][e], k, r);
        if (r.at == 16 * i + e) v -= r.t;
        if (first + 16 * i + e >= p.d.N) v = 0.0f;
        g[e] = v;
      }
      const u32x2 high = pack_d16<DD>(g);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t h = (e & 1) ? high[e / 2] >> 16 : high[e / 2] & 0xffffu;
        rest[e] = g[e] - (BF ? bf16_to_f32(h) : f16_to_f32(h));
      }
      uint16_t* const D = static_cast<uint16_t*>(p.d.D) + ml * p.d.ldd + first + 16 * i;
      *reinterpret_cast<u32x2*>(D) = high;
      *reinterpret_cast<u32x2*>(D + p.d.M * p.d.ldd) = pack_d16<DD>(rest);
    }
  }
}

}  // namespace sg
