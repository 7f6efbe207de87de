// xent_plan.h -- the host side of the cross entropy's calls: their arguments,
// tiles, workspace and the runs of words of the backward pass.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "launch.h"

namespace sg {

struct XentCall {
  int64_t M, N, K;
  float alpha;
  const void* A;
  int64_t lda;
  const void* B;
  int64_t ldb;
  bool bf16;
  const void* targets;
  bool wide;                // 64-bit targets
  void* workspace;
  float* loss;              // forward
  float* lse;               // forward: written, backward: read
  const float* dloss;       // backward
  const float* dlse;        // or NULL
  void* dA;                 // or NULL
  int64_t ldda;
  void* dB;                 // or NULL
  int64_t lddb;
};

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t tile_side(TileShape t) { return t == kTile256 ? 256 : t == kTile128 ? 128 : 64; }

constexpr int64_t kXentCUs = 256;
constexpr int64_t kXentMaxLd = int64_t{1} << 22;   // a panel of 256 rows below 2^31 bytes
constexpr int64_t kXentMaxRows = int64_t{1} << 22; // 256 columns of the gradient below 2^31 bytes
constexpr int64_t kXentMaxTiles = int64_t{1} << 23;  // (of 512 threads: 2^32)

// Up to so many tokens the gradient of the logits is kept in two parts.
constexpr int64_t kXentFew = 64;

// The tiles of the product (both operands K-major).  Up to 64 tokens it is bound
// by reading B: 64x64 tiles with two workgroups a CU (us with B in memory, 64 |
// 128 | 256 tiles: 4 x 32768 x 2048 34.9 | 34.1 | 38.7; 64 x 65536 x 4096 110 |
// 127 | 130; 4 x 70000 x 2048 66 | 97; 64 x 131072 x 4096 207 | 210, 5.2 TB/s).
inline TileShape xent_tile(int64_t M, int64_t N) {
  if (M <= 64) return kTile64;
  return pick_dense_tile(M, N, true, true);
}

// Forward: a pair of floats for each token and column tile, then a float for
// each token.
inline int64_t xent_workspace(int64_t M, int64_t N) {
  return M * cdiv(N, tile_side(xent_tile(M, N))) * 8 + M * 4;
}

// The tiles of a gradient's product of rows x cols over `terms`, and how many
// workgroups share a tile's terms (`most` at most), whose sums a launch more
// adds up.  From measured times (us, all CUs busy): a workgroup takes 5, 4 or
// 2.5 and 0.95, 0.45 or 0.25 for 64 terms with 256x256, 128x128 and 64x64 tiles
// (1021 x 2056 over 32003, K- and MN-major operand, 256 | 128 | 64 alone: 476 |
// 222 | 358; 8192 x 1024 over 128, both MN-major: 10.2 | 14.3 | 24.3), the sums
// 3 and 4 MB a microsecond.
struct XentBack {
  TileShape tile;
  int64_t splits;
  bool fits;  // fewer than 2^23 workgroups
};
inline XentBack xent_back(int64_t rows, int64_t cols, int64_t terms, int64_t most) {
  static const double start[3] = {5.0, 4.0, 2.5}, step[3] = {0.95, 0.45, 0.25};
  const int64_t units = cdiv(terms, 64);
  XentBack best{kTile256, 1, false};
  double least = 0;
  for (int t = 0; t < 3; ++t) {
    const int64_t side = tile_side((TileShape)t);
    const int64_t tiles = cdiv(rows, side) * cdiv(cols, side);
    for (int64_t s = 1; s <= most && (s == 1 || 4 * s <= units); ++s) {
      if (tiles * s >= kXentMaxTiles) break;
      double us = (double)cdiv(tiles * s, kXentCUs) *
                  (start[t] + step[t] * (double)cdiv(units, s));
      if (s > 1) us += 3.0 + (double)s * (double)rows * (double)cols * 2e-6;
      if (least == 0 || us < least) {
        least = us;
        best = {(TileShape)t, s, true};
      }
    }
  }
  return best;
}

// dB of up to 512 terms: 256x128 tiles, two workgroups a CU, where the model says
// 256x256, one (us of all gradients, twin | one: 8 tokens of 131072 x 2048 357 |
// 398, 64 of 8192 x 1024 27.4 | 29.4, 128 of 32000 x 4096 222 | 237, 256 292 |
// 306, 384 of 50257 x 768 152 | 163, 512 of 32000 x 4096 383 | 390, 1024 678 |
// 668).
inline bool xent_twin(TileShape tile, int64_t terms) { return tile == kTile256 && terms <= 512; }

// Whether dA's `values` may be added up in the launch of dB's tiles, four a
// thread: a launch has fewer than 2^32 threads.
inline bool xent_joins(int64_t tiles, int64_t threads, int64_t values) {
  return (tiles + cdiv(values, 4 * threads)) * threads < (int64_t{1} << 32);
}

// Backward: the words go in runs of `words`, for which the gradient of the
// logits, 16 bits each (twice for few tokens), takes up to 512 MB, a row of it
// fewer than 2^22 values (dB's tiles look up to 96 rows past the last by 32-bit
// offsets) and an operand of a product stays below 2^31 bytes.  Workspace: the
// tokens' terms, the scale, the gradient of one run, A twice for few tokens, and
// the sums of dA: one for each split, and with several runs one more.
constexpr int kXentMostParts = 256;  // workgroups that look for the largest |dloss|
constexpr int64_t kXentMostSplits = 32;
struct XentPlan {
  int64_t words, ldg, rows;
  XentBack hidden;  // the product of dA
  bool parts;       // dA comes from parts that are added up
  bool fits;        // every product is one launch
  int64_t scale_at, most_at, g_at, twice_at, sum_at, parts_at, bytes;
};

inline XentPlan xent_plan(int64_t M, int64_t N, int64_t K, int64_t ldb) {
  XentPlan p{};
  const bool few = M <= kXentFew;
  p.rows = few ? 2 * M : M;
  int64_t most = std::max<int64_t>((int64_t{1} << 28) / p.rows, 256);
  most = std::min(most, ((int64_t{1} << 30) - 1) / ldb);
  most = std::min(most, kXentMaxLd - 256);  // (the pitch of g as that of A and B)
  most = std::max<int64_t>(most / 256 * 256, 256);
  p.words = cdiv(cdiv(N, cdiv(N, most)), 256) * 256;
  const int64_t run = std::min(p.words, N);
  // (a pitch of many KiB would put the rows of a tile on the same few memory
  // channels: 256 bytes more, 8192 x 4096 over 32768 1431 -> 1416 us)
  p.ldg = cdiv(run, 64) * 64;
  if (p.ldg % 2048 == 0) p.ldg += 128;
  p.hidden = xent_back(p.rows, K, run, kXentMostSplits);
  p.fits = p.hidden.fits && xent_back(run, K, p.rows, 1).fits;
  p.parts = few || p.hidden.splits > 1;
  p.scale_at = 16 * M;
  p.most_at = p.scale_at + 16;
  p.g_at = cdiv(p.most_at + 8 * kXentMostParts, 256) * 256;
  p.twice_at = p.g_at + 2 * p.rows * p.ldg;
  p.sum_at = p.twice_at + (few ? 2 * p.rows * K : 0);
  p.parts_at = p.sum_at + (p.words < N ? 4 * M * K : 0);
  p.bytes = p.parts_at + (p.parts ? 4 * p.hidden.splits * p.rows * K : 0);
  return p;
}

hipError_t launch_xent(const XentCall& c, hipStream_t s);
// `plan`: xent_plan's, not used where M or N is 0.
hipError_t launch_xent_backward(const XentCall& c, const XentPlan& plan, hipStream_t s);

}  // namespace sg
