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

// The tiles of the product (both operands K-major).
inline TileShape xent_tile(int64_t M, int64_t N, int64_t K) {
  if (M <= 64) return kTile64;
  return pick_dense_tile(M, N, true, true);
}

// The tiles of the gradients' products (MN-major operands, K of them).
inline TileShape xent_back_tile(int64_t M, int64_t N, int64_t K) {
  return pick_dense_tile(M, N, K > 64, true);
}

// Forward: a pair of floats for each token and column tile, then a float for
// each token.
inline int64_t xent_workspace(int64_t M, int64_t N, int64_t K) {
  return M * cdiv(N, tile_side(xent_tile(M, N, K))) * 8 + M * 4;
}

// Backward: the words go in runs of `words`, for which the gradient of the
// logits, 16 bits each, takes up to 512 MB and an operand of a product stays
// below 2^31 bytes.  Workspace: the tokens' terms, the scale, the gradient of
// one run, and with several runs the sum of dA.
struct XentPlan {
  int64_t words, ldg, scale_at, g_at, sum_at, bytes;
};

inline XentPlan xent_plan(int64_t M, int64_t N, int64_t K, int64_t ldb) {
  XentPlan p{};
  const int64_t rows = std::max<int64_t>(M, 1), words = std::max<int64_t>(N, 1);
  int64_t most = std::max<int64_t>((int64_t{1} << 28) / rows, 256);
  most = std::min(most, ((int64_t{1} << 30) - 1) / std::max<int64_t>(ldb, 1));
  most = std::max<int64_t>(most / 256 * 256, 256);
  p.words = cdiv(cdiv(words, cdiv(words, most)), 256) * 256;
  p.ldg = std::min(p.words, cdiv(words, 64) * 64);
  p.scale_at = 16 * M;
  p.g_at = cdiv(p.scale_at + 4, 256) * 256;
  p.sum_at = p.g_at + 2 * M * p.ldg;
  p.bytes = p.sum_at + (p.words < N ? 4 * M * K : 0);
  return p;
}

hipError_t launch_xent(const XentCall& c, hipStream_t s);
hipError_t launch_xent_backward(const XentCall& c, hipStream_t s);

}  // namespace sg
