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
constexpr int64_t kXentMaxTiles = int64_t{1} << 23;

// Up to so many tokens the product streams B past them (xent_few.h).
constexpr int64_t kXentFew = 64;
// Words of a workgroup then: 128 while that fills the CUs, up to 512.
inline int xent_few_blocks(int64_t N) {
  return N > 2 * 128 * kXentCUs ? 4 : N > 128 * kXentCUs ? 2 : 1;
}

// The tiles of the product (both operands K-major).
inline TileShape xent_tile(int64_t M, int64_t N) { return pick_dense_tile(M, N, true, true); }
// Words of a tile, few tokens or not.
inline int64_t xent_columns(int64_t M, int64_t N) {
  return M <= kXentFew ? 128 * xent_few_blocks(N) : tile_side(xent_tile(M, N));
}

// The tiles of the gradients' products (MN-major operands, K of them).
inline TileShape xent_back_tile(int64_t M, int64_t N, int64_t K) {
  return pick_dense_tile(M, N, K > 64, true);
}

// Forward: a pair of floats for each token and column tile, then a float for
// each token.
inline int64_t xent_workspace(int64_t M, int64_t N, int64_t K) {
  return M * cdiv(N, xent_columns(M, N)) * 8 + M * 4;
}

// Backward: the words go in runs of `words`, for which the gradient of the
// logits, 16 bits each (twice for few tokens), takes up to 512 MB and an operand
// of a product stays below 2^31 bytes.  Where dA has too few tiles for the CUs,
// `splits` workgroups a tile share a run's words.  Workspace: the tokens' terms,
// the scale, the gradient of one run, A twice for few tokens, and the sums of
// dA: one for each split, and with several runs one more.
constexpr int kXentMostParts = 256;  // workgroups that look for the largest |dloss|
struct XentPlan {
  int64_t words, ldg, rows, splits;
  int64_t scale_at, most_at, g_at, twice_at, sum_at, parts_at, bytes;
  TileShape a_tile;
};

inline XentPlan xent_plan(int64_t M, int64_t N, int64_t K, int64_t ldb) {
  XentPlan p{};
  const bool few = M <= kXentFew;
  p.rows = few ? 2 * M : M;
  int64_t most = std::max<int64_t>((int64_t{1} << 28) / p.rows, 256);
  most = std::min(most, ((int64_t{1} << 30) - 1) / ldb);
  most = std::max<int64_t>(most / 256 * 256, 256);
  p.words = cdiv(cdiv(N, cdiv(N, most)), 256) * 256;
  const int64_t run = std::min(p.words, N);
  p.ldg = cdiv(run, 64) * 64;
  // (for few tokens one tile holds them all, so that B is read once)
  p.a_tile = few ? (p.rows > 64 ? kTile128 : kTile64) : xent_back_tile(M, K, run);
  const int64_t side = tile_side(p.a_tile), tiles = cdiv(p.rows, side) * cdiv(K, side);
  p.splits = p.a_tile == kTile256
                 ? 1
                 : std::max<int64_t>(1, std::min(kXentCUs / tiles, cdiv(run, 512)));
  const bool parts = few || p.splits > 1, several = p.words < N;
  p.scale_at = 16 * M;
  p.most_at = p.scale_at + 16;
  p.g_at = cdiv(p.most_at + 8 * kXentMostParts, 256) * 256;
  p.twice_at = p.g_at + 2 * p.rows * p.ldg;
  p.sum_at = p.twice_at + (few ? 2 * p.rows * K : 0);
  p.parts_at = p.sum_at + (several ? 4 * M * K : 0);
  p.bytes = p.parts_at + (parts ? 4 * p.splits * p.rows * K : 0);
  return p;
}

hipError_t launch_xent(const XentCall& c, hipStream_t s);
hipError_t launch_xent_backward(const XentCall& c, hipStream_t s);

}  // namespace sg
