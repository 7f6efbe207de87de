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
// counterparts in the same cycles, so large products run the mainloop of
// pingpong16.h (Elem = kElemI8) at twice the operations per byte.  Middle
// sizes run i8_mid_kernel, products of few rows, bound by reading B once,
// i8_stream_kernel.
#pragma once

#include "i8_params.h"
#include "pingpong16.h"

namespace sg {

// The panels of the tile at D row row0 (m_valid rows) and column n0 (bn wide).
// A 16-bit D of 256x256 tiles goes past the caches when grouped, whose tiles
// come from many B (us alone / with a quantiser that reads D next, past |
// through: 8192 x 2048 x 2048 of 64 groups 80.5 / 94.4 | 86.0 / 94.2; 32768 x
// 4096 x 1024 of 32 180 / 242 | 193 / 253; x 2048, gathered 305 / 349 | 310 /
// 357).  A dense product's reader finds it in the caches, and one of few K
// tiles is faster itself (8192 x 8192 x 1024 82 / 115 | 74 / 104; x 8192 366 /
// 415 | 375 / 405; 4096 x 16384 x 4096 204 / 255 | 207 / 241).  An fp32 D is
// stored 16 bytes a lane, in parts of lines that the caches put together
// (8192 x 4096 x 1024 72 / 99 | 51 / 76; 32768 x 4096 x 2048 of 32 groups 407 /
// 528 | 357 / 487).
template <bool Rows>
__device__ __forceinline__ TileJob i8_job(const I8Params& p, int64_t row0, int m_valid,
                                          int64_t n0, int bn, int g, bool past) {
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
  j.past = past;
  return j;
}

template <int BM>
__device__ __forceinline__ TileJob i8_dense_job(const I8Params& p, int wg, int bn) {
  const int t = xcd_remap(wg, p.tiles_m * p.tiles_n);
  int tm, tn;
  raster(t, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
  const int64_t m0 = (int64_t)tm * BM;
  return i8_job<false>(p, m0, (int)min<int64_t>(BM, p.M - m0), (int64_t)tn * bn, bn, 0,
                       false);
}

// The tile of workgroup `wg` among the groups' tiles, found from the offsets
// in device memory: lane l adds up the row tiles of groups 4l .. 4l+3, a scan
// over the wave places them, and the lane whose range holds the tile names
// the group.  About a microsecond of latency against a host round trip for
// the offsets.  Offsets outside [0, M] are clamped and a decreasing pair is
// an empty group, so no offsets make the kernel leave its buffers; tiles that
// such offsets add beyond the grid are not computed.  (Nor do they overflow
// the counts: the host keeps R / BM below 2^23, and of 256 groups at most 128
// can rise over all R rows.)  False: no tile.
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
  j = i8_job<Rows>(p, (int64_t)row0 + m0, min(BM, rows_g - m0), (int64_t)tn * bn, bn, g, true);
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

// Middle sizes, fewer 256x256 tiles than CUs: BM x BN tiles of eight waves in
// two groups of four, one wave of each group per SIMD.  Group g multiplies K
// tiles 2i + g, and the groups work one phase apart: in phase t one group
// reads K tile t from LDS into registers while the other runs its MFMAs over
// tile t - 1, so the LDS, the matrix cores and the loads are all busy in every
// phase.  (With both groups in the same phase, or with one group of four, the
// units wait for each other: a 128x128x128-byte step took 0.53 us instead of
// the 0.33 us its LDS traffic needs.)  The groups' integer sums are added in
// the epilogue, exactly.
//
// One ring of kStages K tiles serves both groups.  Every wave loads an eighth
// of tile t + kStages - 1 in phase t, into the stage whose tile t - 1 was read
// in the phase before; a phase ends when the wave's part of tile t + 1 has
// landed, and its barrier makes that tile whole.
template <int BM, int BN, bool Rows>
struct I8MidTile {
  static constexpr int kWM = BM / 2, kWN = BN / 2;        // a wave's block
  static constexpr int kFM = kWM / 32, kFN = kWN / 32;    // 32x32 blocks of it
  // K tiles are kSub times 128 bytes wide: 64x64 tiles take two at a time,
  // which halves the barriers of their short phases.
  static constexpr int kSub = BM * BN <= 64 * 64 ? 2 : 1;
  static constexpr int kABytes = BM * 128, kSubBytes = (BM + BN) * 128;
  static constexpr int kStageBytes = kSub * kSubBytes;
  static constexpr int kStages = 163840 / kStageBytes;    // 5 or 6
  static constexpr int kLdsBytes = kStages * kStageBytes;
  static constexpr int kSubLoads = (BM + BN) / 64;
  static constexpr int kLoads = kSub * kSubLoads;         // a wave's loads per K tile
  static constexpr int kSteps = 4 * kSub;                 // 32-byte K steps of a tile
  static_assert(kStages >= 3 && (kStages - 2) * kLoads < 64, "the ring");
  using ALoader = typename std::conditional<Rows, RowsHalfLoader<kSwzDefault>,
                                            HalfLoader<kSwzDefault>>::type;

  struct Frags {
    u32x4 a[kSteps][kFM], b[kSteps][kFN];
  };

  // The end of a phase.
  __device__ __forceinline__ static void end_phase() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"((kStages - 2) * kLoads) : "memory");
    PingPongTile<kElemI8, kSwzDefault>::barrier();
  }

  __device__ __forceinline__ static void run(char* smem, const TileJob& j, const I8Params& p) {
    const int tid = threadIdx.x;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = wave >> 2, w4 = wave & 3, wm = w4 >> 1, wn = w4 & 1;
    const int lrow = lane & 31, lhalf = lane >> 5;
    const u32x4 ra = rsrc_words(j.a, j.a_bytes), rb = rsrc_words(j.b, j.b_bytes);
    const uint32_t kbytes = (uint32_t)p.K;
    const int T = (int)((p.K + 128 * kSub - 1) / (128 * kSub)), Tg = (T + 1) / 2;
    // The half-tile loaders with eight waves: wave w fills regions 8q + w, the
    // loaders' load 2q of "wave" w.
    ALoader la;
    HalfLoader<kSwzDefault> lb;
    if constexpr (Rows)
      la.init(wave, lane, j.a_pitch, j.rows, j.m_valid, j.a_total);
    else
      la.init(wave, lane, j.a_pitch);
    lb.init(wave, lane, j.b_pitch);
    const uint32_t ring = lds_addr(smem);
    const Scales sc = load_scales(j, lane, g, wm, wn);

    // Load q of the wave's part of K tile t; past K every chunk reads as zero.
    auto issue1 = [&](int t, int q) {
      const int sub = q / kSubLoads, l = q % kSubLoads;
      const uint32_t stage = ring + (uint32_t)((t % kStages) * kStageBytes + sub * kSubBytes);
      const uint32_t k0 = (uint32_t)(kSub * t + sub) * 128u;
      if (l < BM / 64)
        la.issue(ra, stage, wave, 2 * l, j.m_valid, k0, kbytes);
      else
        lb.issue(rb, stage + kABytes, wave, 2 * (l - BM / 64), j.n_valid, k0, kbytes);
    };
    auto issue = [&](int t) {
#pragma unroll
      for (int q = 0; q < kLoads; ++q) issue1(t, q);
    };
    uint32_t oa[4], ob[4];  // fragment 0 of each step of 128 bytes; the next ones 4 KiB on
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      oa[s] = lds_offset<128, kSwzDefault>(wm * kWM + lrow, 2 * s + lhalf);
      ob[s] = kABytes + lds_offset<128, kSwzDefault>(wn * kWN + lrow, 2 * s + lhalf);
    }
    f32x16 acc[kFM][kFN];
#pragma unroll
    for (int m = 0; m < kFM; ++m)
#pragma unroll
      for (int n = 0; n < kFN; ++n) acc[m][n] = f32x16{};

#pragma unroll
    for (int t = 0; t < kStages - 1; ++t) issue(t);
    end_phase();  // tile 0 has landed (its newer loads are those of a phase's end)
    if (g) {      // group 1 is one phase behind
      issue(kStages - 1);
      end_phase();
    }
    for (int i = 0; i < Tg; ++i) {
      const int t = 2 * i + g;  // the phase, and the tile it reads
      Frags f;
      const char* st = smem + (t % kStages) * kStageBytes;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
#pragma unroll
        for (int m = 0; m < kFM; ++m)
          f.a[s][m] = lds_read16(st, oa[s & 3] + (s >> 2) * kSubBytes + m * 4096);
#pragma unroll
        for (int n = 0; n < kFN; ++n)
          f.b[s][n] = lds_read16(st, ob[s & 3] + (s >> 2) * kSubBytes + n * 4096);
      }
      issue(t + kStages - 1);
      end_phase();
      constexpr int kMfma = kSteps * kFM * kFN, kEvery = kMfma / kLoads;
#pragma unroll
      for (int q = 0; q < kMfma; ++q) {
        const int s = q / (kFM * kFN), b = q % (kFM * kFN);
        const int m = b / kFN, n = (m & 1) ? kFN - 1 - b % kFN : b % kFN;
        acc[m][n] = mfma32x32x16<kElemI8>(f.b[s][n], f.a[s][m], acc[m][n]);
        if (q % kEvery == kEvery - 1 && q / kEvery < kLoads) {
          __builtin_amdgcn_sched_barrier(0);
          issue1(t + kStages, q / kEvery);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      end_phase();
    }
    wait_vmem();  // the loads past K
    PingPongTile<kElemI8, kSwzDefault>::barrier();
    if (!g) PingPongTile<kElemI8, kSwzDefault>::barrier();
    store(acc, smem, j, p, sc, lane, g, w4, wm, wn);
  }

  // The scales of the outputs that a lane stores, loaded before the mainloop:
  // after it, their latency (with gathered rows twice) added 3 us to a tile.
  static constexpr int kRowBytes = 128 * kFN, kWaveBytes = 32 * kFM * kRowBytes;
  static constexpr int kLanesPerRow = kRowBytes / 16, kRowsPerStep = 64 / kLanesPerRow;
  struct Scales {
    float a[kWaveBytes / 2048], b[4];
  };
  __device__ __forceinline__ static int out_row(int h, int lane, int g) {
    return kRowsPerStep * (2 * h + g) + lane / kLanesPerRow;
  }
  __device__ __forceinline__ static Scales load_scales(const TileJob& j, int lane, int g, int wm,
                                                       int wn) {
    Scales sc;
    const int nl = wn * kWN + 4 * (lane % kLanesPerRow);
#pragma unroll
    for (int h = 0; h < kWaveBytes / 2048; ++h)
      sc.a[h] = i8_row_scale<Rows>(j, wm * kWM + out_row(h, lane, g));
#pragma unroll
    for (int e = 0; e < 4; ++e) sc.b[e] = j.sb[min(nl + e, j.n_valid - 1)];
    return sc;
  }

  // Lane l of accumulator block (m, n) holds row 32m + l%32 of the wave's
  // block, columns 32n + 8q + 4(l/32) .. +3 in registers 4q .. 4q+3.  Every
  // wave puts its sums into LDS as rows of kRowBytes, chunk c of row r at c
  // XOR (r mod 8) (the 8 rows of a ds_write_b128 phase then fill a bank line);
  // the two waves of a block take alternate KiB of both groups' rows, add them,
  // scale them and store whole rows.
  static_assert(8 * kWaveBytes <= kLdsBytes, "staging fits the ring");
  __device__ __forceinline__ static void store(const f32x16 (&acc)[kFM][kFN], char* smem,
                                               const TileJob& j, const I8Params& p,
                                               const Scales& sc, int lane, int g, int w4, int wm,
                                               int wn) {
    char* const mine = smem + (4 * g + w4) * kWaveBytes;
#pragma unroll
    for (int m = 0; m < kFM; ++m)
#pragma unroll
      for (int n = 0; n < kFN; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4 v = {acc[m][n][4 * q], acc[m][n][4 * q + 1], acc[m][n][4 * q + 2],
                           acc[m][n][4 * q + 3]};
          const uint32_t r = (uint32_t)(32 * m + (lane & 31));
          const uint32_t c = (uint32_t)(8 * n + 2 * q + (lane >> 5));
          lds_write16(mine, r * kRowBytes + 16u * (c ^ (r & 7u)), __builtin_bit_cast(u32x4, v));
        }
    __syncthreads();
    const uint32_t cc = (uint32_t)(lane % kLanesPerRow);
    const int nl = wn * kWN + 4 * (int)cc, cols = j.n_valid - nl;
    if (cols <= 0) return;
#pragma unroll
    for (int h = 0; h < kWaveBytes / 2048; ++h) {
      const uint32_t r = (uint32_t)out_row(h, lane, g);
      const uint32_t off = r * kRowBytes + 16u * (cc ^ (r & 7u));
      const int ml = wm * kWM + (int)r;
      if (ml >= j.m_valid) continue;
      const i32x4 s = __builtin_bit_cast(i32x4, lds_read16(smem + w4 * kWaveBytes, off)) +
                      __builtin_bit_cast(i32x4, lds_read16(smem + (4 + w4) * kWaveBytes, off));
      const f32x4 v = i8_scale4(__builtin_bit_cast(f32x4, s), sc.a[h], sc.b);
      store_i8_chunk(v, p.D, p.d_dtype, (j.d_row0 + ml) * p.ldd + j.n0 + nl, cols, j.vec);
    }
  }
};

template <int BM, int BN, bool Grouped, bool Rows>
__global__ void __launch_bounds__(512, 1) i8_mid_kernel(const I8Params p) {
  using Tile = I8MidTile<BM, BN, Rows>;
  __shared__ __attribute__((aligned(4096))) char smem[Tile::kLdsBytes];
  const ClockStamp cs = clock_begin(p.clk);
  TileJob j;
  if constexpr (Grouped) {
    if (!i8_grouped_job<BM, Rows>(p, blockIdx.x, j, BN)) return;
  } else {
    j = i8_dense_job<BM>(p, blockIdx.x, BN);
  }
  Tile::run(smem, j, p);
  clock_end(p.clk, cs);
}

// ---- few rows

// 16*MT rows by BN = 16*NT*WN columns, for products that are bound by reading
// B.  Eight waves: WN along N, the other WK = 8 / WN split K.  A stage is 512
// bytes of K of both operands, loaded straight to LDS an eighth by each wave
// and kStages deep, so the loads in flight take no registers and every wave
// waits once per 512 bytes; wave (wn, wk) multiplies its 64*WN bytes of the
// stage.  The integer sums of the WK waves are added through LDS at the end.
// (Reading both operands into registers instead kept too few loads in flight:
// 16 x 8192 x 8192 took 20 us against 12 for the bytes.)
template <int MT, int NT, int WN, int Stages>
struct I8StreamTile {
  static constexpr int kBM = 16 * MT, kBN = 16 * NT * WN, kWK = 8 / WN;
  static constexpr int kSubBytes = (kBM + kBN) * 128;  // 128 bytes of K: A, then B
  static constexpr int kStageBytes = 4 * kSubBytes;
  static constexpr int kStages = Stages;
  static constexpr int kLoadsA = MT, kLoadsB = NT * WN, kLoads = kLoadsA + kLoadsB;
  static constexpr int kBlocks = MT * NT;
  static constexpr int kSumBytes = kWK > 1 ? 8 * kBlocks * 1024 : 0;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kLdsBytes = kRingBytes > kSumBytes ? kRingBytes : kSumBytes;
  static_assert(kStages >= 2 && (kStages - 1) * kLoads < 64 && kLdsBytes <= 163840, "the ring");

  // One wave's loads of one operand: load i fills 1 KiB region r = wave + 8i
  // of the stage's four 128-byte wide sub-tiles (Regions each, 8 rows).
  template <int Loads, int Regions>
  struct Loader {
    uint32_t voff[Loads], koff[Loads];  // byte of the operand; byte of K in the stage

    // source(row): the row of the operand, or -1.
    template <class Source>
    __device__ __forceinline__ void init(int wave, int lane, uint32_t pitch, Source source) {
#pragma unroll
      for (int i = 0; i < Loads; ++i) {
        const int idx = wave + 8 * i, sub = idx / Regions, r = idx % Regions;
        const uint32_t at = swz_bytes<kSwzDefault>((uint32_t)r * 1024u + 16u * (uint32_t)lane);
        const int src = source((int)(at >> 7));
        koff[i] = (uint32_t)sub * 128u + (at & 127u);
        voff[i] = src >= 0 ? (uint32_t)src * pitch + koff[i] : kOutOfRange;
      }
    }
    __device__ __forceinline__ void issue(u32x4 rsrc, uint32_t stage, int wave, uint32_t k0,
                                          uint32_t kbytes) const {
#pragma unroll
      for (int i = 0; i < Loads; ++i) {
        const int idx = wave + 8 * i, sub = idx / Regions, r = idx % Regions;
        dma16(rsrc, k0 + koff[i] < kbytes ? voff[i] + k0 : kOutOfRange,
              stage + (uint32_t)(sub * kSubBytes + r * 1024));
      }
    }
  };

  template <bool Rows>
  __device__ __forceinline__ static void run(char* smem, const TileJob& j, const I8Params& p) {
    const int tid = threadIdx.x;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, c = lane >> 4;
    const int wk = wave % kWK, wn = wave / kWK;
    const u32x4 ra = rsrc_words(j.a, j.a_bytes), rb = rsrc_words(j.b, j.b_bytes);
    Loader<kLoadsB, kBN / 8> lb;
    Loader<kLoadsA, kBM / 8> la;
    lb.init(wave, lane, j.b_pitch, [&](int n) { return n < j.n_valid ? n : -1; });
    la.init(wave, lane, j.a_pitch, [&](int m) {
      if (m >= j.m_valid) return -1;
      if (!Rows) return m;
      const int src = j.rows[m];
      return (uint32_t)src < (uint32_t)j.a_total ? src : -1;
    });
    const uint32_t kbytes = (uint32_t)p.K, ring = lds_addr(smem);
    const int T = (int)((p.K + 511) >> 9);
    auto issue = [&](int t) {
      const uint32_t stage = ring + (uint32_t)((t % kStages) * kStageBytes);
      lb.issue(rb, stage + kBM * 128, wave, (uint32_t)t * 512u, kbytes);
      la.issue(ra, stage, wave, (uint32_t)t * 512u, kbytes);
    };
#pragma unroll
    for (int t = 0; t < kStages - 1; ++t) issue(t);

    float sa[MT], sb[NT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) sa[mt] = i8_row_scale<Rows>(j, 16 * mt + r);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sb[nt][e] = j.sb[min(16 * (NT * wn + nt) + 4 * c + e, j.n_valid - 1)];
    f32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = f32x4{};
    uint32_t oa[WN], ob[WN];  // the wave's K steps: row block 0; the next 2 KiB on
#pragma unroll
    for (int s = 0; s < WN; ++s) {
      const int step = wk * WN + s;
      const uint32_t at = (uint32_t)((step >> 1) * kSubBytes);
      oa[s] = at + lds_offset<128, kSwzDefault>(r, 4 * (step & 1) + c);
      ob[s] = at + kBM * 128 + lds_offset<128, kSwzDefault>(16 * NT * wn + r, 4 * (step & 1) + c);
    }

    for (int t = 0; t < T; ++t) {
      // This wave's part of stage t has landed and its reads of stage t - 1
      // are done; after the barrier both hold for every wave.
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"((kStages - 2) * kLoads) : "memory");
      PingPongTile<kElemI8, kSwzDefault>::barrier();
      const char* st = smem + (t % kStages) * kStageBytes;
      u32x4 fa[WN][MT], fb[WN][NT];
#pragma unroll
      for (int s = 0; s < WN; ++s) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) fa[s][mt] = lds_read16(st, block_at(oa[s], mt));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) fb[s][nt] = lds_read16(st, block_at(ob[s], nt));
      }
      issue(t + kStages - 1);
#pragma unroll
      for (int s = 0; s < WN; ++s)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            acc[mt][nt] = mfma16x16x32<kElemI8>(fb[s][nt], fa[s][mt], acc[mt][nt]);
    }

    // Lane l of a block holds columns 4c .. 4c+3 of row l%16.  Block b's sums
    // over the WK waves are finished by wave b mod WK of them.
    wait_vmem();  // the loads past K
    if constexpr (kWK > 1) {
      __syncthreads();
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
        lds_write16(smem, (uint32_t)((wave * kBlocks + b) * 1024 + 16 * lane),
                    __builtin_bit_cast(u32x4, acc[b / NT][b % NT]));
      __syncthreads();
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      if (b % kWK != wk) continue;
      i32x4 v = __builtin_bit_cast(i32x4, acc[b / NT][b % NT]);
      if constexpr (kWK > 1) {
        v = i32x4{};
#pragma unroll
        for (int w = 0; w < kWK; ++w)
          v += __builtin_bit_cast(
              i32x4, lds_read16(smem, (uint32_t)(((kWK * wn + w) * kBlocks + b) * 1024 +
                                                 16 * lane)));
      }
      const int ml = 16 * (b / NT) + r, nl = 16 * (NT * wn + b % NT) + 4 * c;
      if (ml >= j.m_valid || nl >= j.n_valid) continue;
      const f32x4 d = i8_scale4(__builtin_bit_cast(f32x4, v), sa[b / NT], sb[b % NT]);
      store_i8_chunk(d, p.D, p.d_dtype, (j.d_row0 + ml) * p.ldd + j.n0 + nl, j.n_valid - nl,
                     j.vec);
    }
  }

  // The place of 16-row block b, from block 0's: rows 16 apart differ in bit 3
  // of the XOR key (the line index), rows 32 apart in none of it.
  __device__ __forceinline__ static uint32_t block_at(uint32_t first, int b) {
    return (first ^ ((uint32_t)(b & 1) << 7)) + (uint32_t)b * 2048u;
  }
};

template <int MT, int NT, int WN, int Stages, bool Grouped, bool Rows>
__global__ void __launch_bounds__(512, 1) i8_stream_kernel(const I8Params p) {
  using Tile = I8StreamTile<MT, NT, WN, Stages>;
  __shared__ __attribute__((aligned(4096))) char smem[Tile::kLdsBytes];
  const ClockStamp cs = clock_begin(p.clk);
  TileJob j;
  if constexpr (Grouped) {
    if (!i8_grouped_job<Tile::kBM, Rows>(p, blockIdx.x, j, Tile::kBN)) return;
  } else {
    j = i8_dense_job<Tile::kBM>(p, blockIdx.x, Tile::kBN);
  }
  Tile::template run<Rows>(smem, j, p);
  clock_end(p.clk, cs);
}

}  // namespace sg
