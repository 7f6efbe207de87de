// xent.hip -- the vocabulary's cross entropy (gemm_xent_run) and its gradients
// (gemm_xent_backward_run): instantiations, the kernels around the products,
// and the plan of both calls.
#include "xent.h"

#include "launch.h"
#include "twin16.h"
#include "xent_plan.h"

namespace sg {

namespace {

constexpr int kJoinThreads = 512;

// Joins the tiles' pairs of each token: R tokens a workgroup, whose threads
// split the tiles; every pair of partners is joined in a fixed order.  With p
// the target's logit, loss = (maximum - p) + log(sum): where the target holds
// the maximum, the sum is 1 + the rest and the small loss keeps its digits,
// which lse - p would lose.
template <int R>
__global__ void __launch_bounds__(kJoinThreads) xent_join_kernel(const XentRows p) {
  constexpr int kSegs = kJoinThreads / R;
  __shared__ float2 area[kSegs][R];
  const int r = threadIdx.x % R, seg = threadIdx.x / R;
  const int64_t row = block_index() * R + r;
  const bool live = row < p.M;
  float m = -__builtin_inff(), s = 0.0f;
  if (live) {
    const float2* part = reinterpret_cast<const float2*>(p.part) + row;
    int t = seg;
    for (; t + 3 * kSegs < p.tiles; t += 4 * kSegs) {
      float2 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = part[(int64_t)(t + i * kSegs) * p.M];
#pragma unroll
      for (int i = 0; i < 4; ++i) join_stats(m, s, v[i].x, v[i].y);
    }
    for (; t < p.tiles; t += kSegs) {
      const float2 v = part[(int64_t)t * p.M];
      join_stats(m, s, v.x, v.y);
    }
  }
  area[seg][r] = make_float2(m, s);
#pragma unroll
  for (int half = kSegs / 2; half > 0; half /= 2) {
    __syncthreads();
    if (seg < half) {
      const float2 a = area[seg][r], b = area[seg + half][r];
      m = a.x;
      s = a.y;
      join_stats(m, s, b.x, b.y);
      area[seg][r] = make_float2(m, s);
    }
  }
  if (seg != 0 || !live) return;
  const float log_sum = logf(s);
  p.lse[row] = m + log_sum;
  p.loss[row] =
      target_of(p.targets, p.wide, row, p.N) >= 0 ? (m - p.zt[row]) + log_sum : 0.0f;
}

constexpr int kRowsThreads = 1024;

// The largest a and b of a workgroup.
__device__ __forceinline__ float2 over_workgroup(float a, float b,
                                                 float2 (&area)[kRowsThreads / 64]) {
  a = lane_reduce<64>(a, OpMax{});
  b = lane_reduce<64>(b, OpMax{});
  if ((threadIdx.x & 63) == 0) area[threadIdx.x >> 6] = make_float2(a, b);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kRowsThreads / 64; ++w) {
    a = __builtin_fmaxf(a, area[w].x);
    b = __builtin_fmaxf(b, area[w].y);
  }
  return make_float2(a, b);
}

// The factors of token m's gradient: dloss (0 without a target) and with dlse.
__device__ __forceinline__ float2 factors_of(const XentRows& p, int64_t m, int t) {
  const float given = p.dloss[m], dl = t >= 0 ? given : 0.0f;
  return make_float2(dl, p.dlse ? dl + p.dlse[m] : dl);
}

// The largest |dloss| and the largest sum with the softmax's factor over tokens
// first, first + step, ..., then over the workgroup.
__device__ __forceinline__ float2 largest(const XentRows& p, int64_t first, int64_t step,
                                          float2 (&area)[kRowsThreads / 64]) {
  float most = 0.0f, top = 0.0f;
#pragma unroll 4
  for (int64_t m = first; m < p.M; m += step) {
    const float2 f = factors_of(p, m, target_of(p.targets, p.wide, m, p.N));
    const float2 size = weight_of(f.x, f.y);
    most = __builtin_fmaxf(most, size.x);
    top = __builtin_fmaxf(top, size.y);
  }
  return over_workgroup(most, top, area);
}

// Beyond 8192 tokens a launch looks for them first; each workgroup for itself
// takes as long until then.
__global__ void __launch_bounds__(kRowsThreads) xent_most_kernel(const XentRows p) {
  __shared__ float2 area[kRowsThreads / 64];
  const float2 v = largest(p, (int64_t)blockIdx.x * kRowsThreads + threadIdx.x,
                           (int64_t)gridDim.x * kRowsThreads, area);
  if (threadIdx.x == 0) p.most[blockIdx.x] = v;
}

// The terms of each token's gradient (XentGrad::Row).
__global__ void __launch_bounds__(kRowsThreads) xent_rows_kernel(const XentRows p) {
  __shared__ float2 area[kRowsThreads / 64];
  float2 found;
  if (p.parts == 0) {
    found = largest(p, threadIdx.x, kRowsThreads, area);
  } else {
    const float2 v = (int)threadIdx.x < p.parts ? p.most[threadIdx.x] : make_float2(0.0f, 0.0f);
    found = over_workgroup(v.x, v.y, area);
  }
  const XentScale f = scale_of(p.alpha, found.x, found.y);
  if (blockIdx.x == 0 && threadIdx.x == 0) p.scale[0] = f.down;
  const int64_t m = (int64_t)blockIdx.x * kRowsThreads + threadIdx.x;
  if (m >= p.M) return;
  const int t = target_of(p.targets, p.wide, m, p.N);
  const float2 w = factors_of(p, m, t);
  const float lse = p.lse[m];
  reinterpret_cast<f32x4*>(p.rows)[m] =
      f32x4{base_of(lse), softmax_factor(w.x, w.y, f.up, lse), w.x * f.up,
            __builtin_bit_cast(float, t)};
}

// Rows of 16-byte chunks set to zero (an empty vocabulary).
__global__ void __launch_bounds__(256) xent_zero_kernel(char* D, int64_t rows, int64_t chunks,
                                                        int64_t pitch) {
  const int64_t i = block_index() * 256 + threadIdx.x;
  if (i >= rows * chunks) return;
  *reinterpret_cast<u32x4*>(D + i / chunks * pitch + 16 * (i % chunks)) = u32x4{};
}

// Four values of dA, from i on, from its parts [splits][rows][K], rows M + m (with
// rows = 2 M) belonging to rows m, and the runs before: the last run's sum is
// rounded to dA's type.  Eight loads in flight a thread.
template <int DD>
__device__ __forceinline__ void sum_parts(const XentSum& p, int64_t i) {
  if (i >= p.M * p.K) return;
  f32x4 v = p.before ? *reinterpret_cast<const f32x4*>(p.before + i) : f32x4{};
  const float* const part = p.parts + i;
  if (p.rows > p.M) {
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
      v += *reinterpret_cast<const f32x4*>(part + (int64_t)(2 * s) * p.M * p.K);
      v += *reinterpret_cast<const f32x4*>(part + (int64_t)(2 * s + 1) * p.M * p.K);
    }
  } else {
#pragma unroll 8
    for (int s = 0; s < p.splits; ++s)
      v += *reinterpret_cast<const f32x4*>(part + (int64_t)s * p.M * p.K);
  }
  if constexpr (DD == SG_F32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(p.D) + i) = v;
  } else {
    v *= p.scale[0];
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.D) + i / p.K * p.ldd + i % p.K) =
        pack_d16<DD>(v);
  }
}

// Bound by reading the parts: small workgroups, so that all CUs read.
template <int DD>
__global__ void __launch_bounds__(64) xent_sum_kernel(const XentSum p) {
  sum_parts<DD>(p, (block_index() * 64 + threadIdx.x) * 4);
}

// dB on 256x256 tiles, and behind its tiles' workgroups those that add up dA's
// parts, which then overlap (a launch of them alone takes 4 us or more).
template <bool BF>
__global__ void __launch_bounds__(512, 1) xent_head_kernel(const DenseParams p, const XentSum q) {
  using Tile = PingPong16Tile<BF, kSwzDefault, true, true, true, false, void, true>;
  __shared__ __attribute__((aligned(4096))) char smem[Tile::kLdsBytes];
  const int tiles = p.tiles_m * p.tiles_n;
  if ((int)blockIdx.x >= tiles) {
    sum_parts<BF ? SG_BF16 : SG_F16>(q, ((int64_t)(blockIdx.x - tiles) * 512 + threadIdx.x) * 4);
    return;
  }
  const TileJob j = dense_tile_job<256, 256, true, true>(p, blockIdx.x);
  Tile::run(smem, j, p.K, nullptr, SG_NONE, p.D, p.d_dtype, p.ldd);
}

// The same on the 256x128 tiles of few tokens.  (Without a sum q.M is 0.)
template <bool BF>
__global__ void __launch_bounds__(256, 2) xent_twin_kernel(const DenseParams p, const XentSum q) {
  using Tile = TwinTile<BF>;
  __shared__ __attribute__((aligned(4096))) char smem[Tile::kLdsBytes];
  const int tiles = p.tiles_m * p.tiles_n;
  if ((int)blockIdx.x >= tiles) {
    sum_parts<BF ? SG_BF16 : SG_F16>(q, ((int64_t)(blockIdx.x - tiles) * 256 + threadIdx.x) * 4);
    return;
  }
  const TileJob j = dense_tile_job<256, 128, true, true>(p, blockIdx.x);
  Tile::run(smem, j, p.K, p.D, p.ldd);
}

// The gradient of the logits of few tokens, on 64x64 tiles; behind the tiles'
// workgroups those that write A twice.  One launch for what takes two otherwise
// (with the tokens' terms): a launch of them alone is 4 us of 33 (64 x 8192 x
// 1024).
template <bool BF>
__global__ void __launch_bounds__(256, 1) xent_few_kernel(const XentParams p, const XentTwice q) {
  using Tile = DeepTile<64, BF, false, false, XentGradFew<BF ? SG_BF16 : SG_F16>, 5>;
  __shared__ __attribute__((aligned(4096))) char smem[Tile::kLdsBytes];
  const int tiles = p.d.tiles_m * p.d.tiles_n;
  if ((int)blockIdx.x >= tiles) {
    const int64_t i = (int64_t)(blockIdx.x - tiles) * 256 + threadIdx.x, all = q.M * q.chunks;
    if (i >= all) return;
    const u32x4 v =
        *reinterpret_cast<const u32x4*>(q.A + i / q.chunks * q.pitch + 16 * (i % q.chunks));
    *reinterpret_cast<u32x4*>(q.D + 16 * i) = v;
    *reinterpret_cast<u32x4*>(q.D + 16 * (i + all)) = v;
    return;
  }
  const TileJob j = xent_job<64>(p, blockIdx.x);
  Tile::run(smem, j, p.d.K, nullptr, SG_NONE, p.d.D, p.d.d_dtype, p.d.ldd);
}

// One tile of dA over a share of the words: workgroup (x, y) of gridDim.y takes
// every share of whole 64 words, the last one to the end.
__device__ __forceinline__ void take_share(DenseParams& p) {
  const int64_t units = (p.K + 63) / 64;
  const int64_t first = 64 * (units * blockIdx.y / gridDim.y);
  const int64_t end = 64 * (units * (blockIdx.y + 1) / gridDim.y);
  p.A = static_cast<const char*>(p.A) + 2 * first;
  p.B = static_cast<const char*>(p.B) + 2 * first * p.ldb;
  p.D = static_cast<float*>(p.D) + (int64_t)blockIdx.y * p.M * p.N;
  p.K = min<int64_t>(end, p.K) - first;
}

template <int BM, bool BF>
__global__ void __launch_bounds__(256, 1) xent_split_kernel(DenseParams p) {
  using Tile = DeepTile<BM, BF, false, true>;
  __shared__ __attribute__((aligned(4096))) char smem[Tile::kLdsBytes];
  take_share(p);
  const TileJob j = dense_tile_job<BM, BM, false, true>(p, blockIdx.x);
  Tile::run(smem, j, p.K, nullptr, SG_NONE, p.D, SG_F32, p.N);
}

template <bool BF>
__global__ void __launch_bounds__(512, 1) xent_split_pingpong_kernel(DenseParams p) {
  using Tile = PingPong16Tile<BF, kSwzDefault, false, true, true, false, void, true>;
  __shared__ __attribute__((aligned(4096))) char smem[Tile::kLdsBytes];
  take_share(p);
  const TileJob j = dense_tile_job<256, 256, false, true>(p, blockIdx.x);
  Tile::run(smem, j, p.K, nullptr, SG_NONE, p.D, SG_F32, p.N);
}

template <bool BF, class Epi>
hipError_t go_product(TileShape tile, const XentParams& p, const char* epi, hipStream_t s) {
  const int grid = p.d.tiles_m * p.d.tiles_n;
  constexpr const char* kType = BF ? "bf16" : "f16";
  if (tile == kTile256 && p.d.K % 64) {
    static const char* const name = kernel_label("xent_pingpong_kernel", kType, epi, "tail");
    last_kernel() = name;
    hipLaunchKernelGGL((xent_pingpong_kernel<BF, Epi, true>), dim3(grid), dim3(512), 0, s, p);
  } else if (tile == kTile256) {
    static const char* const name = kernel_label("xent_pingpong_kernel", kType, epi);
    last_kernel() = name;
    hipLaunchKernelGGL((xent_pingpong_kernel<BF, Epi, false>), dim3(grid), dim3(512), 0, s, p);
  } else if (tile == kTile128 && grid > kXentCUs) {
    static const char* const name = kernel_label("xent_dense_kernel", kType, epi);
    last_kernel() = name;
    hipLaunchKernelGGL((xent_dense_kernel<BF, Epi>), dim3(grid), dim3(256), 0, s, p);
  } else if (tile == kTile128) {
    static const char* const name = kernel_label("xent_deep_kernel", "128", kType, epi);
    last_kernel() = name;
    hipLaunchKernelGGL((xent_deep_kernel<128, BF, Epi>), dim3(grid), dim3(256), 0, s, p);
  } else {
    static const char* const name = kernel_label("xent_deep_kernel", "64", kType, epi);
    last_kernel() = name;
    hipLaunchKernelGGL((xent_deep_kernel<64, BF, Epi>), dim3(grid), dim3(256), 0, s, p);
  }
  return hipGetLastError();
}

void set_product(DenseParams& d, int64_t M, int64_t N, int64_t K) {
  d = DenseParams{};
  d.M = M;
  d.N = N;
  d.K = K;
  d.alpha = 1.0f;
  d.group_m = 8;
}

void set_tiles(DenseParams& d, TileShape t) {
  const int64_t side = tile_side(t);
  d.tiles_m = (int)cdiv(d.M, side);
  d.tiles_n = (int)cdiv(d.N, side);
}

XentRows rows_of(const XentCall& c) {
  XentRows r{};
  r.M = c.M;
  r.N = c.N;
  r.alpha = c.alpha;
  r.targets = c.targets;
  r.wide = c.wide;
  return r;
}

template <int R>
void go_join(const XentRows& r, hipStream_t s) {
  hipLaunchKernelGGL((xent_join_kernel<R>), grid_of(cdiv(r.M, R)), dim3(kJoinThreads), 0, s, r);
}

template <int BM>
void go_split(const DenseParams& d, bool bf16, dim3 grid, hipStream_t s) {
  if (bf16)
    hipLaunchKernelGGL((xent_split_kernel<BM, true>), grid, dim3(256), 0, s, d);
  else
    hipLaunchKernelGGL((xent_split_kernel<BM, false>), grid, dim3(256), 0, s, d);
}

hipError_t go_head(const DenseParams& d, const XentSum& q, bool bf16, hipStream_t s) {
  static const char* const names[2] = {kernel_label("xent_head_kernel", "f16"),
                                       kernel_label("xent_head_kernel", "bf16")};
  last_kernel() = names[bf16];
  const dim3 grid((unsigned)(d.tiles_m * d.tiles_n + cdiv(q.M * q.K, 4 * 512)));
  if (bf16) hipLaunchKernelGGL((xent_head_kernel<true>), grid, dim3(512), 0, s, d, q);
  else hipLaunchKernelGGL((xent_head_kernel<false>), grid, dim3(512), 0, s, d, q);
  return hipGetLastError();
}

hipError_t go_few(const XentParams& p, const XentCall& c, char* twice, hipStream_t s) {
  static const char* const names[2] = {kernel_label("xent_few_kernel", "f16"),
                                       kernel_label("xent_few_kernel", "bf16")};
  last_kernel() = names[c.bf16];
  const XentTwice q{static_cast<const char*>(c.A), c.M, c.K / 8, 2 * c.lda, twice};
  const dim3 grid((unsigned)(p.d.tiles_m * p.d.tiles_n + (twice ? cdiv(q.M * q.chunks, 256) : 0)));
  if (c.bf16) hipLaunchKernelGGL((xent_few_kernel<true>), grid, dim3(256), 0, s, p, q);
  else hipLaunchKernelGGL((xent_few_kernel<false>), grid, dim3(256), 0, s, p, q);
  return hipGetLastError();
}

hipError_t go_twin(const DenseParams& d, const XentSum& q, bool bf16, hipStream_t s) {
  static const char* const names[2] = {kernel_label("xent_twin_kernel", "f16"),
                                       kernel_label("xent_twin_kernel", "bf16")};
  last_kernel() = names[bf16];
  const dim3 grid((unsigned)(d.tiles_m * d.tiles_n + cdiv(q.M * q.K, 4 * 256)));
  if (bf16) hipLaunchKernelGGL((xent_twin_kernel<true>), grid, dim3(256), 0, s, d, q);
  else hipLaunchKernelGGL((xent_twin_kernel<false>), grid, dim3(256), 0, s, d, q);
  return hipGetLastError();
}

// The sum of dA's parts over one run of words.
XentSum sum_of(const XentCall& c, const XentPlan& plan, int64_t v0, int64_t n) {
  char* const w = static_cast<char*>(c.workspace);
  float* const sum = reinterpret_cast<float*>(w + plan.sum_at);
  // (a last run may have fewer words than splits of 64)
  const int splits = (int)std::min(plan.hidden.splits, cdiv(n, 64));
  return {c.M, c.K, plan.rows, splits, reinterpret_cast<float*>(w + plan.parts_at),
          v0 == 0 ? nullptr : sum, reinterpret_cast<const float*>(w + plan.scale_at),
          v0 + n == c.N ? c.dA : sum, c.ldda};
}

// dA of one run of n words from v0 on: g B, in fp32 until the last run.  `alone`:
// with the sum of its parts.
hipError_t hidden_gradient(const XentCall& c, const XentPlan& plan, const char* G, const char* B,
                           int64_t v0, int64_t n, bool alone, hipStream_t s) {
  char* const w = static_cast<char*>(c.workspace);
  float* const sum = reinterpret_cast<float*>(w + plan.sum_at);
  const bool first = v0 == 0, last = v0 + n == c.N;
  const int dt = c.bf16 ? SG_BF16 : SG_F16;
  const TileShape tile = plan.hidden.tile;
  DenseParams d;
  set_product(d, plan.rows, c.K, n);
  d.A = G;
  d.lda = plan.ldg;
  d.B = B;
  d.ldb = c.ldb;
  set_tiles(d, tile);
  if (plan.parts) {
    const XentSum q = sum_of(c, plan, v0, n);
    d.D = w + plan.parts_at;
    d.d_dtype = SG_F32;
    d.ldd = c.K;
    const dim3 grid((unsigned)(d.tiles_m * d.tiles_n), (unsigned)q.splits);
    if (tile == kTile128) go_split<128>(d, c.bf16, grid, s);
    else if (tile == kTile64) go_split<64>(d, c.bf16, grid, s);
    else if (c.bf16)
      hipLaunchKernelGGL((xent_split_pingpong_kernel<true>), grid, dim3(512), 0, s, d);
    else
      hipLaunchKernelGGL((xent_split_pingpong_kernel<false>), grid, dim3(512), 0, s, d);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !alone) return e;
    const dim3 blocks = grid_of(cdiv(c.M * c.K, 256));
    if (!last) hipLaunchKernelGGL((xent_sum_kernel<SG_F32>), blocks, dim3(64), 0, s, q);
    else if (c.bf16) hipLaunchKernelGGL((xent_sum_kernel<SG_BF16>), blocks, dim3(64), 0, s, q);
    else hipLaunchKernelGGL((xent_sum_kernel<SG_F16>), blocks, dim3(64), 0, s, q);
    return hipGetLastError();
  }
  d.C = first ? nullptr : sum;
  d.c_dtype = first ? SG_NONE : SG_F32;
  d.ldc = c.K;
  d.beta = first ? 0.0f : 1.0f;
  d.D = last ? c.dA : sum;
  d.d_dtype = last ? dt : SG_F32;
  d.ldd = last ? c.ldda : c.K;
  // (the scale is undone run by run: the sum holds what it stands for)
  d.alpha_dev = reinterpret_cast<const float*>(w + plan.scale_at);
  return launch_dense_any_k(tile, c.bf16, false, true, d, s);
}

// dB of the words [v0, v0 + n): g^T A.
struct HeadProduct {
  DenseParams d;
  TileShape tile;
  bool twin;  // 256x128 tiles instead of 256x256
};
HeadProduct head_product(const XentCall& c, const XentPlan& plan, const char* G, int64_t v0,
                         int64_t n) {
  char* const w = static_cast<char*>(c.workspace);
  const bool twice = plan.rows > c.M;
  HeadProduct h;
  DenseParams& d = h.d;
  set_product(d, n, c.K, plan.rows);
  d.A = G;
  d.lda = plan.ldg;
  d.B = twice ? w + plan.twice_at : c.A;
  d.ldb = twice ? c.K : c.lda;
  d.c_dtype = SG_NONE;
  d.D = static_cast<char*>(c.dB) + v0 * c.lddb * 2;
  d.d_dtype = c.bf16 ? SG_BF16 : SG_F16;
  d.ldd = c.lddb;
  d.alpha_dev = reinterpret_cast<const float*>(w + plan.scale_at);
  d.group_m = 4;  // (8192 x 65536 x 4096, all gradients with 2 | 4 | 8 | 16 tile rows
                  // a group: 9080 | 9069 | 9150 | 9340 us; the others like 8 as well)
  h.tile = xent_back(d.M, d.N, d.K, 1).tile;
  set_tiles(d, h.tile);
  h.twin = xent_twin(h.tile, d.K);
  if (h.twin) {
    d.tiles_n = (int)cdiv(d.N, 128);
    d.group_m = 8;  // (128 x 32000 x 4096, all gradients: 222 us, 227 with 4)
  }
  return h;
}

}  // namespace

hipError_t launch_xent(const XentCall& c, hipStream_t s) {
  const TileShape tile = xent_tile(c.M, c.N);
  XentParams p{};
  set_product(p.d, c.M, c.N, c.K);
  p.d.A = c.A;
  p.d.lda = c.lda;
  p.d.B = c.B;
  p.d.ldb = c.ldb;
  p.d.alpha = c.alpha;
  set_tiles(p.d, tile);
  p.x.targets = c.targets;
  p.x.wide = c.wide;
  p.x.words = c.N;
  p.x.part = static_cast<float*>(c.workspace);
  p.x.zt = p.x.part + 2 * c.M * p.d.tiles_n;
  if (c.N > 0) {
    const hipError_t e = c.bf16 ? go_product<true, XentStats>(tile, p, "stats", s)
                                : go_product<false, XentStats>(tile, p, "stats", s);
    if (e != hipSuccess) return e;
  }
  XentRows r = rows_of(c);
  r.part = p.x.part;
  r.zt = p.x.zt;
  r.tiles = p.d.tiles_n;
  r.loss = c.loss;
  r.lse = c.lse;
  // Tokens of a workgroup: enough workgroups for the CUs, and up to 32 tokens,
  // whose pairs are one 256-byte piece of each tile's row.
  if (c.M > 4096) go_join<32>(r, s);
  else if (c.M > 1024) go_join<8>(r, s);
  else go_join<2>(r, s);
  return hipGetLastError();
}

hipError_t launch_xent_backward(const XentCall& c, const XentPlan& plan, hipStream_t s) {
  if (c.M == 0 || c.N == 0) {  // sums of nothing
    char* const D = static_cast<char*>(c.N == 0 ? c.dA : c.dB);
    const int64_t n = c.N == 0 ? c.M : c.N, chunks = c.K / 8;
    if (!D || n == 0) return hipSuccess;
    hipLaunchKernelGGL(xent_zero_kernel, grid_of(cdiv(n * chunks, 256)), dim3(256), 0, s, D, n,
                       chunks, 2 * (c.N == 0 ? c.ldda : c.lddb));
    return hipGetLastError();
  }
  const bool few = plan.rows > c.M;
  char* const w = static_cast<char*>(c.workspace);
  char* const G = w + plan.g_at;
  XentRows r = rows_of(c);
  r.lse = const_cast<float*>(c.lse);
  r.dloss = c.dloss;
  r.dlse = c.dlse;
  r.rows = reinterpret_cast<float*>(w);
  r.scale = reinterpret_cast<float*>(w + plan.scale_at);
  r.most = reinterpret_cast<float2*>(w + plan.most_at);
  r.parts = c.M > 8192 ? (int)std::min<int64_t>(cdiv(c.M, kRowsThreads), kXentMostParts) : 0;
  hipError_t e = hipSuccess;
  if (!few) {
    if (r.parts)
      hipLaunchKernelGGL(xent_most_kernel, dim3(r.parts), dim3(kRowsThreads), 0, s, r);
    hipLaunchKernelGGL(xent_rows_kernel, dim3((unsigned)cdiv(c.M, kRowsThreads)),
                       dim3(kRowsThreads), 0, s, r);
    e = hipGetLastError();
  }
  for (int64_t v0 = 0; v0 < c.N && e == hipSuccess; v0 += plan.words) {
    const int64_t n = std::min(plan.words, c.N - v0);
    const bool last = v0 + n == c.N;
    const char* const B = static_cast<const char*>(c.B) + v0 * c.ldb * 2;
    XentParams p{};
    set_product(p.d, c.M, n, c.K);
    p.d.A = c.A;
    p.d.lda = c.lda;
    p.d.B = B;
    p.d.ldb = c.ldb;
    p.d.alpha = c.alpha;
    p.d.D = G;
    p.d.ldd = plan.ldg;
    p.d.d_dtype = c.bf16 ? SG_BF16 : SG_F16;
    p.x.n_store = cdiv(n, 64) * 64;
    p.x.words = c.N;
    p.col0 = v0;
    const TileShape tile = xent_tile(c.M, n);
    set_tiles(p.d, tile);
    if (few) {
      p.x.targets = c.targets;
      p.x.wide = c.wide;
      p.x.dloss = c.dloss;
      p.x.dlse = c.dlse;
      p.x.lse = c.lse;
      p.x.scale = r.scale;
      p.x.low = c.M * plan.ldg;
      e = go_few(p, c, v0 == 0 && c.dB ? w + plan.twice_at : nullptr, s);
    } else {
      p.x.rows = r.rows;
      e = c.bf16 ? go_product<true, XentGrad<SG_BF16>>(tile, p, "grad", s)
                 : go_product<false, XentGrad<SG_F16>>(tile, p, "grad", s);
    }
    HeadProduct h{};
    if (c.dB) h = head_product(c, plan, G, v0, n);
    const bool both = c.dA && c.dB && plan.parts && last && h.tile == kTile256 &&
                      xent_joins((int64_t)h.d.tiles_m * h.d.tiles_n, h.twin ? 256 : 512,
                                 c.M * c.K);
    if (e == hipSuccess && c.dA) e = hidden_gradient(c, plan, G, B, v0, n, !both, s);
    if (e != hipSuccess) break;
    if (h.twin)
      e = go_twin(h.d, both ? sum_of(c, plan, v0, n) : XentSum{}, c.bf16, s);
    else if (both)
      e = go_head(h.d, sum_of(c, plan, v0, n), c.bf16, s);
    else if (c.dB)
      e = launch_dense_any_k(h.tile, c.bf16, true, true, h.d, s);
  }
  return e;
}

}  // namespace sg
