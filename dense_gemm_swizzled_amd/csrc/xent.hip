// xent.hip -- the vocabulary's cross entropy (gemm_xent_run) and its gradients
// (gemm_xent_backward_run): instantiations, the kernels around the products,
// and the plan of both calls.
#include "xent.h"

#include "launch.h"
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

// The terms of each token's gradient (XentGrad::Row).  fp16 holds 2^-24 to
// 2^16, less than the factors of a mean over many tokens times the softmax of a
// large vocabulary span: they are scaled by the power of two that brings the
// largest to [2^13, 2^14), found by every workgroup for itself, and the
// products undo it in fp32 (scale[0]).  bf16 has fp32's range.
__global__ void __launch_bounds__(256) xent_rows_kernel(const XentRows p) {
  float factor = 1.0f;
  if (p.scaled) {
    __shared__ float tops[4];
    float top = 0.0f;
    for (int64_t m = threadIdx.x; m < p.M; m += 256) {
      const float dl = target_of(p.targets, p.wide, m, p.N) >= 0 ? p.dloss[m] : 0.0f;
      const float whole = p.dlse ? dl + p.dlse[m] : dl;
      top = __builtin_fmaxf(top, __builtin_fabsf(dl) + __builtin_fabsf(whole));
    }
    top = lane_reduce<64>(top, OpMax{});
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    top = __builtin_fmaxf(__builtin_fmaxf(tops[0], tops[1]), __builtin_fmaxf(tops[2], tops[3])) *
          __builtin_fabsf(p.alpha);
    int e = 0;
    if (top > 0.0f && top < __builtin_inff()) {
      frexpf(top, &e);          // top in [2^(e-1), 2^e)
      e = min(max(14 - e, -100), 100);
      factor = ldexpf(1.0f, e);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.scale[0] = ldexpf(1.0f, -e * (factor != 1.0f));
  }
  const int64_t m = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (m >= p.M) return;
  const int t = target_of(p.targets, p.wide, m, p.N);
  const float dl = t >= 0 ? p.dloss[m] : 0.0f;
  const float whole = p.dlse ? dl + p.dlse[m] : dl;
  reinterpret_cast<f32x4*>(p.rows)[m] =
      f32x4{p.lse[m] * kLog2e, whole * p.alpha * factor, dl * p.alpha * factor,
            __builtin_bit_cast(float, t)};
}

// Rows of 16-byte chunks set to zero (an empty vocabulary).
__global__ void __launch_bounds__(256) xent_zero_kernel(char* D, int64_t rows, int64_t chunks,
                                                        int64_t pitch) {
  const int64_t i = block_index() * 256 + threadIdx.x;
  if (i >= rows * chunks) return;
  *reinterpret_cast<u32x4*>(D + i / chunks * pitch + 16 * (i % chunks)) = u32x4{};
}

template <bool BF, class Epi>
hipError_t go_product(TileShape tile, const XentParams& p, const char* epi, hipStream_t s) {
  const int grid = p.d.tiles_m * p.d.tiles_n;
  if (tile == kTile256) {
    static const char* const name = kernel_label("xent_pingpong_kernel", BF ? "bf16" : "f16", epi);
    last_kernel() = name;
    hipLaunchKernelGGL((xent_pingpong_kernel<BF, Epi>), dim3(grid), dim3(512), 0, s, p);
  } else if (tile == kTile128) {
    static const char* const name =
        kernel_label("xent_deep_kernel", "128", BF ? "bf16" : "f16", epi);
    last_kernel() = name;
    hipLaunchKernelGGL((xent_deep_kernel<128, BF, Epi>), dim3(grid), dim3(256), 0, s, p);
  } else {
    static const char* const name =
        kernel_label("xent_deep_kernel", "64", BF ? "bf16" : "f16", epi);
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

}  // namespace

hipError_t launch_xent(const XentCall& c, hipStream_t s) {
  const TileShape tile = xent_tile(c.M, c.N, c.K);
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

hipError_t launch_xent_backward(const XentCall& c, hipStream_t s) {
  const XentPlan plan = xent_plan(c.M, c.N, c.K, c.ldb);
  char* const w = static_cast<char*>(c.workspace);
  float* const rows = reinterpret_cast<float*>(w);
  float* const scale = reinterpret_cast<float*>(w + plan.scale_at);
  char* const G = w + plan.g_at;
  float* const sum = reinterpret_cast<float*>(w + plan.sum_at);

  if (c.M == 0 || c.N == 0) {  // sums of nothing
    char* const D = static_cast<char*>(c.N == 0 ? c.dA : c.dB);
    const int64_t n = c.N == 0 ? c.M : c.N, chunks = c.K / 8;
    if (!D || n == 0) return hipSuccess;
    hipLaunchKernelGGL(xent_zero_kernel, grid_of(cdiv(n * chunks, 256)), dim3(256), 0, s, D, n,
                       chunks, 2 * (c.N == 0 ? c.ldda : c.lddb));
    return hipGetLastError();
  }
  XentRows r = rows_of(c);
  r.lse = const_cast<float*>(c.lse);
  r.dloss = c.dloss;
  r.dlse = c.dlse;
  r.rows = rows;
  r.scale = scale;
  r.scaled = !c.bf16;
  hipLaunchKernelGGL(xent_rows_kernel, dim3((unsigned)cdiv(c.M, 256)), dim3(256), 0, s, r);
  hipError_t e = hipGetLastError();
  const int dt = c.bf16 ? SG_BF16 : SG_F16;
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
    p.d.d_dtype = dt;
    p.x.rows = rows;
    p.x.n_store = cdiv(n, 64) * 64;
    p.col0 = v0;
    const TileShape tile = xent_tile(c.M, n, c.K);
    set_tiles(p.d, tile);
    e = c.bf16 ? go_product<true, XentGrad<SG_BF16>>(tile, p, "grad", s)
               : go_product<false, XentGrad<SG_F16>>(tile, p, "grad", s);
    if (e != hipSuccess) return e;
    if (c.dA) {  // dA += g B, in fp32 until the last words
      DenseParams d;
      set_product(d, c.M, c.K, n);
      d.A = G;
      d.lda = plan.ldg;
      d.B = B;
      d.ldb = c.ldb;
      d.C = v0 > 0 ? sum : nullptr;
      d.c_dtype = v0 > 0 ? SG_F32 : SG_NONE;
      d.ldc = c.K;
      d.beta = v0 > 0 ? 1.0f : 0.0f;
      d.D = last ? c.dA : sum;
      d.d_dtype = last ? dt : SG_F32;
      d.ldd = last ? c.ldda : c.K;
      d.alpha_dev = c.bf16 ? nullptr : scale;
      const TileShape t = xent_back_tile(d.M, d.N, n);
      set_tiles(d, t);
      e = launch_dense_any_k(t, c.bf16, false, true, d, s);
      if (e != hipSuccess) return e;
    }
    if (c.dB) {
      DenseParams d;
      set_product(d, n, c.K, c.M);
      d.A = G;
      d.lda = plan.ldg;
      d.B = c.A;
      d.ldb = c.lda;
      d.c_dtype = SG_NONE;
      d.D = static_cast<char*>(c.dB) + v0 * c.lddb * 2;
      d.d_dtype = dt;
      d.ldd = c.lddb;
      d.alpha_dev = c.bf16 ? nullptr : scale;
      const TileShape t = xent_back_tile(d.M, d.N, c.M);
      set_tiles(d, t);
      e = launch_dense_any_k(t, c.bf16, true, true, d, s);
      if (e != hipSuccess) return e;
    }
  }
  return e;
}

}  // namespace sg
