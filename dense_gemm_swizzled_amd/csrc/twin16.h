// twin16.h -- 256x128 tiles of a product of two MN-major operands over few terms
// (dB of up to a few hundred tokens), two workgroups a CU.
//
// Why.  With K of a few hundred, a 256x256 tile of the ping-pong, which has its
// CU to itself, spends half its time on its first loads and its last stores
// (32000 x 4096: 9 us of each tile whatever K is, and 9 for each 512 of K).  Here
// two workgroups share a CU: the stores and first loads of one run beside the
// MFMAs of the other, with no synchronisation between them.  Measured, us this |
// the ping-pong, 32000 x 4096 over 64 terms 55 | 71 (its 262 MB of D take 50),
// 128 74 | 84, 256 108 | 115, 512 160 | 162, 1024 275 | 255: the narrower tile
// reads more of LDS for each MFMA, by transposing reads, and loses where K is
// long.  (Delaying one of the two workgroups at the start changed nothing.)
//
// Layout.  72 KiB of LDS a workgroup: a ring of three stages of 32 k rows, A's
// two halves of 128 columns and B's 128 columns, each [32][128] as the ping-pong
// keeps an MN-major half (mn256_lds_offset; fragments by transposing reads).  Four
// waves, 2x2, of 128x64 outputs each: 8x4 blocks of 16x16x32 MFMAs, a stage being
// one step of K.  Every wave loads a quarter of a stage, two stages ahead.  D, 16
// bits, is staged in LDS and stored in whole 128-byte row segments
// (epilogue_lds_t).
#pragma once

#include "pingpong16.h"

namespace sg {

template <bool BF>
struct TwinTile {
  using Wide = PingPong16Tile<BF, kSwzDefault, true, true, true, false, void, true>;
  static constexpr int kBlock = 32 * 256;       // 32 k rows of 128 columns
  static constexpr int kStage = 3 * kBlock;     // A's halves, then B
  static constexpr int kStages = 3;
  static constexpr int kLdsBytes = kStages * kStage;
  static constexpr int kBK = 32;
  static constexpr int kI = Wide::kI, kJ = Wide::kJ;
  static_assert(kLdsBytes >= 4 * 16384, "D's staging area");

  // The barrier of the mainloop: the wave's LDS reads have returned and all but
  // its newest six loads, those of the next stage, have landed.
  __device__ __forceinline__ static void sync() {
    asm volatile("s_waitcnt vmcnt(6) lgkmcnt(0)" ::: "memory");
    Wide::PP::barrier();
  }

  __device__ __forceinline__ static void run(char* smem, const TileJob& j, int64_t K, void* D,
                                             int64_t ldd) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const u32x4 ra = rsrc_words(j.a, j.a_bytes), rb = rsrc_words(j.b, j.b_bytes);
    const uint32_t s0 = lds_addr(smem);

    // Loads: region 2 wave + i (four k rows) of each block; lane l fills byte 16
    // (l%16) of row l/16, whose place's columns the (self-inverse) unit XOR gives.
    // Columns past the tile's take its last ones (not stored).
    uint32_t va[2][2], vb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t k = (uint32_t)(4 * (2 * wave + i) + (lane >> 4));
      const int col = (int)(mn256_lds_offset(k, 16u * (uint32_t)(lane & 15)) - k * 256u) >> 1;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        va[h][i] = k * j.a_pitch + 2u * (uint32_t)min(128 * h + col, (j.m_valid - 1) & ~7);
      vb[i] = k * j.b_pitch + 2u * (uint32_t)min(col, (j.n_valid - 1) & ~7);
    }
    // Stage t, k rows 32 t .. 32 t + 31.  Rows past K start past the descriptors'
    // records and read as zero (offsets stay below 2^32: at most 2^31 bytes and 96
    // rows of 2^23).
    auto issue = [&](int t, uint32_t stage) {
      const uint32_t ka = (uint32_t)t * (32u * j.a_pitch), kb = (uint32_t)t * (32u * j.b_pitch);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t at = s0 + stage + (uint32_t)(2 * wave + i) * 1024u;
        dma16(ra, va[0][i] + ka, at);
        dma16(ra, va[1][i] + ka, at + kBlock);
        dma16(rb, vb[i] + kb, at + 2 * kBlock);
      }
    };
    const int T = (int)((K + kBK - 1) / kBK);
    issue(0, 0u);
    issue(1, kStage);

    // Block i's and j's offsets in a stage (PingPong16Tile::offsets).
    uint32_t oa[kI], ob[kJ];
    const int r = lane & 15, c = lane >> 4;
    const uint32_t krow = (uint32_t)(8 * c + (r >> 2));
#pragma unroll
    for (int i = 0; i < kI; ++i)
      oa[i] = wm * kBlock + mn256_lds_offset(krow, 2u * (uint32_t)(16 * i + 4 * (r & 3)));
#pragma unroll
    for (int k = 0; k < kJ; ++k)
      ob[k] = 2 * kBlock +
              mn256_lds_offset(krow, 2u * (uint32_t)(64 * wn + 16 * k + 4 * (r & 3)));
    f32x4 acc[kI][kJ];
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int k = 0; k < kJ; ++k) acc[i][k] = f32x4{};

    uint32_t now = 0, ahead = 2 * kStage;  // stages t and t + 2
    for (int t = 0; t < T; ++t) {
      sync();  // stage t is there for all waves, and all are done with stage t - 1
      issue(t + 2, ahead);
      typename Wide::Frags f;
#pragma unroll
      for (int k = 0; k < kJ; ++k) f.b[k] = Wide::read_bt(smem + now, ob[k]);
#pragma unroll
      for (int i = 0; i < kI; ++i) f.a[i] = Wide::read_bt(smem + now, oa[i]);
      Wide::template mfmas<true>(acc, f);
      ahead = now;
      now = now == 2 * kStage ? 0u : now + kStage;
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");  // (the zeros past K too)
    Wide::PP::barrier();
    char* cq[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) cq[q] = smem + q * 16384;
    // (the staging area has a place for each wave, whose index also counts 64
    // columns: the tile's are moved back by those of the waves above)
    TileJob out = j;
    out.n0 -= 128 * wm;
    out.n_valid += 128 * wm;
    Wide::template epilogue_lds_t<SG_NONE, BF ? SG_BF16 : SG_F16>(acc, out, cq, D, ldd, lane, wm,
                                                                  wave);
  }
};

}  // namespace sg
