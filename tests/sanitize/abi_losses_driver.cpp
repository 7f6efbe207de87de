// abi_losses_driver.cpp -- drives the validation paths of the cross entropy and
// of the routing's balance loss (include/swizzled_gemm.h) on the host, for an
// AddressSanitizer + UndefinedBehaviorSanitizer build of the library's host
// code, which it contains as source: so it also checks the plan of the gradient
// over many sizes, and the tiles that the sizes of the GPU tests take.  Every
// call is rejected (or is a no-op) before the library touches the GPU.  Exit
// status 0 = every return code and choice as documented and no report.
#include "../../dense_gemm_swizzled_amd/csrc/api.hip"

static int fails = 0;
#define EXPECT_RC(call, want)                                                          \
  do {                                                                                 \
    const long long rc_ = (call);                                                      \
    if (rc_ != (want)) {                                                               \
      std::fprintf(stderr, "%s:%d: %s returned %lld, expected %lld (%s)\n", __FILE__,  \
                   __LINE__, #call, rc_, (long long)(want), gemm_last_error());        \
      ++fails;                                                                         \
    }                                                                                  \
  } while (0)

// Fake device addresses: never dereferenced.
static char* const Pc = reinterpret_cast<char*>(uintptr_t{0x10000});
static void* const P = Pc;
static float* const F = reinterpret_cast<float*>(Pc);
static float* const F2 = reinterpret_cast<float*>(Pc + 2);
static int32_t* const I = reinterpret_cast<int32_t*>(Pc);
static const int64_t kBig = int64_t{1} << 62;

static void cross_entropy() {
  auto run = [](int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
                int64_t ldb, int dt, const void* t, int tt, float* loss, void* w, int64_t wb) {
    return gemm_xent_run(M, N, K, 1.0f, A, lda, B, ldb, dt, t, tt, loss, F, w, wb, nullptr);
  };
  EXPECT_RC(run(-1, 50, 64, P, 64, P, 64, SG_BF16, P, SG_I64, F, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(run(kBig, 50, 64, P, 64, P, 64, SG_BF16, P, SG_I64, F, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(run(33, kBig, 64, P, 64, P, 64, SG_BF16, P, SG_I64, F, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(run(33, 50, kBig, P, kBig, P, kBig, SG_BF16, P, SG_I64, F, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(run(33, 50, 60, P, 64, P, 64, SG_BF16, P, SG_I64, F, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(run(33, 50, 64, P, kBig, P, 64, SG_BF16, P, SG_I64, F, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(run(33, 50, 64, P, 64, P, kBig, SG_BF16, P, SG_I64, F, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(run(33, 50, 64, P, 68, P, 64, SG_BF16, P, SG_I64, F, P, kBig), SG_ERR_ALIGN);
  EXPECT_RC(run(33, 50, 64, P, 64, P, 64, SG_F32, P, SG_I64, F, P, kBig), SG_ERR_DTYPE);
  EXPECT_RC(run(33, 50, 64, P, 64, P, 64, SG_F16, P, SG_F32, F, P, kBig), SG_ERR_DTYPE);
  EXPECT_RC(run(33, 50, 64, nullptr, 64, P, 64, SG_F16, P, SG_I32, F, P, kBig), SG_ERR_NULL);
  EXPECT_RC(run(33, 50, 64, P, 64, P, 64, SG_F16, nullptr, SG_I32, F, P, kBig), SG_ERR_NULL);
  EXPECT_RC(run(33, 50, 64, P, 64, P, 64, SG_F16, Pc + 2, SG_I32, F, P, kBig), SG_ERR_ALIGN);
  EXPECT_RC(run(33, 50, 64, P, 64, P, 64, SG_F16, P, SG_I32, nullptr, P, kBig), SG_ERR_NULL);
  EXPECT_RC(run(33, 50, 64, P, 64, P, 64, SG_F16, P, SG_I32, F2, P, kBig), SG_ERR_ALIGN);
  EXPECT_RC(run(33, 50, 64, P, 64, P, 64, SG_F16, P, SG_I32, F, P, 7), SG_ERR_SHAPE);
  EXPECT_RC(run(33, 50, 64, P, 64, P, 64, SG_F16, P, SG_I32, F, nullptr, kBig), SG_ERR_NULL);
  EXPECT_RC(run(33, 50, 64, P, 64, P, 64, SG_F16, P, SG_I32, F, Pc + 8, kBig), SG_ERR_ALIGN);
  EXPECT_RC(run(1 << 22, 1 << 30, 64, P, 64, P, 64, SG_F16, P, SG_I32, F, P, kBig),
            SG_ERR_SHAPE);
  // 2^23 tiles, whose threads no launch counts
  EXPECT_RC(run(1 << 20, 1 << 19, 64, P, 64, P, 64, SG_F16, P, SG_I32, F, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(sg::xent_joins((1 << 23) - 1, 512, 2048), 0);
  EXPECT_RC(sg::xent_joins((1 << 23) - 2, 512, 2048), 1);
  EXPECT_RC(sg::xent_joins(1 << 22, 512, int64_t{1} << 33), 0);
  EXPECT_RC(sg::xent_twin(sg::kTile256, 512), 1);
  EXPECT_RC(sg::xent_twin(sg::kTile256, 513), 0);
  EXPECT_RC(sg::xent_twin(sg::kTile128, 64), 0);
  EXPECT_RC(run(0, 50, 64, nullptr, 64, P, 64, SG_F16, nullptr, SG_I32, nullptr, nullptr, 0),
            SG_OK);
  auto back = [](int64_t M, int64_t lda, const float* dl, const float* dlse, void* dA,
                 int64_t ldda, void* dB, int64_t lddb, void* w, int64_t wb) {
    return gemm_xent_backward_run(M, 50, 64, 1.0f, dl, dlse, P, lda, P, 64, SG_BF16, P, SG_I64, F,
                                  dA, ldda, dB, lddb, w, wb, nullptr);
  };
  EXPECT_RC(back(1 << 22, 64, F, F, P, 64, P, 64, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(back(1 << 21, 1 << 11, F, F, P, 64, P, 64, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(back(33, 64, F, F, P, 56, P, 64, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(back(33, 64, F, F, P, 64, P, 63, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(back(33, 64, F, F, P, 68, P, 64, P, kBig), SG_ERR_ALIGN);
  EXPECT_RC(back(33, 64, F, F, P, 64, Pc + 8, 64, P, kBig), SG_ERR_ALIGN);
  EXPECT_RC(back(33, 64, nullptr, F, P, 64, P, 64, P, kBig), SG_ERR_NULL);
  EXPECT_RC(back(33, 64, F, F2, P, 64, P, 64, P, kBig), SG_ERR_ALIGN);
  EXPECT_RC(back(33, 64, F, F, P, 64, P, 64, P, 100), SG_ERR_SHAPE);
  EXPECT_RC(back(33, 64, F, F, P, 64, P, 64, nullptr, kBig), SG_ERR_NULL);
  EXPECT_RC(back(33, 64, F, F, nullptr, 0, nullptr, 0, nullptr, 0), SG_OK);
  EXPECT_RC(gemm_xent_workspace_bytes(kBig, 5, 8), SG_ERR_SHAPE);
  EXPECT_RC(gemm_xent_backward_workspace_bytes(5, 5, 8, kBig), SG_ERR_SHAPE);
  EXPECT_RC(gemm_xent_backward_workspace_bytes(5, 5, kBig, kBig), SG_ERR_SHAPE);
}

// The plan of the gradient: runs that cover the words, operands below 2^31
// bytes, areas that follow each other on 16-byte borders, launches of fewer than
// 2^23 workgroups.
static void plans() {
  for (int64_t M = 1; M < sg::kXentMaxRows; M = 3 * M + 5)
    for (int64_t N = 1; N < kMaxExtent; N = 7 * N + 11)
      for (int64_t ldb = 8; ldb < sg::kXentMaxLd; ldb = 24 * ldb + 8) {
        const int64_t K = ldb;
        const sg::XentPlan p = sg::xent_plan(M, N, K, ldb);
        const int64_t run = p.words < N ? p.words : N;
        EXPECT_RC(p.words > 0 && p.words % 256 == 0 && p.ldg >= run && p.ldg % 64 == 0 &&
                      p.ldg >= cdiv(run, 64) * 64, 1);
        EXPECT_RC(p.rows * p.ldg * 2 < kMaxExtent && (run - 1) * ldb * 2 + 2 * K < kMaxExtent, 1);
        EXPECT_RC((p.scale_at | p.most_at | p.g_at | p.twice_at | p.sum_at | p.parts_at) % 16, 0);
        EXPECT_RC(16 * M <= p.scale_at && p.scale_at < p.most_at && p.most_at < p.g_at &&
                      p.g_at + 2 * p.rows * p.ldg <= p.twice_at && p.twice_at <= p.sum_at &&
                      p.sum_at <= p.parts_at && p.parts_at <= p.bytes, 1);
        EXPECT_RC(p.hidden.splits >= 1 && p.hidden.splits <= sg::kXentMostSplits, 1);
        if (p.hidden.splits > 1) EXPECT_RC(4 * p.hidden.splits <= cdiv(run, 64), 1);
        const int64_t side = sg::tile_side(p.hidden.tile);
        const int64_t d = sg::tile_side(sg::xent_back(run, K, p.rows, 1).tile);
        // (a gradient of more tiles than a launch has is refused)
        EXPECT_RC(cdiv(p.rows, side) * cdiv(K, side) * p.hidden.splits < sg::kXentMaxTiles &&
                      cdiv(run, d) * cdiv(K, d) < sg::kXentMaxTiles, p.fits);
        // (fewer than 2^32 threads, with half the width of a tile too)
        if (p.fits && d == 256) EXPECT_RC(cdiv(run, 256) * cdiv(K, 128) * 256 < kMaxExtent * 2, 1);
        if (!p.fits)
          EXPECT_RC(gemm_xent_backward_run(M, N, K, 1.0f, F, nullptr, P, K, P, ldb, SG_BF16, P,
                                           SG_I64, F, P, K, nullptr, K, P, kBig, nullptr),
                    SG_ERR_SHAPE);
        EXPECT_RC(gemm_xent_backward_workspace_bytes(M, N, K, ldb), p.bytes);
      }
}

// The tiles of the GPU tests' sizes: every kernel runs.
static void choices() {
  struct Choice {
    int64_t M, N, K;
    sg::TileShape product, hidden;
    int64_t splits;
    sg::TileShape head;
  };
  const sg::TileShape A = sg::kTile256, B = sg::kTile128, C = sg::kTile64;
  const Choice list[] = {{17, 129, 40, C, C, 1, C},         {65, 257, 200, C, C, 1, C},
                         {130, 8190, 320, B, C, 16, B},     {700, 7001, 64, B, C, 16, C},
                         {2000, 8200, 192, A, B, 8, B},     {4099, 4100, 200, A, B, 3, B},
                         {40, 66001, 72, C, C, 32, A},      {2049, 20000, 1032, A, A, 5, A},
                         {2048, 20032, 1024, A, A, 8, A},   {8192, 300, 1032, B, A, 1, C},
                         {3000, 70, 520, C, B, 1, C},       {100, 300, 4096, C, C, 1, B},
                         {5000, 100003, 72, A, B, 6, B}};
  for (const Choice& c : list) {
    const sg::XentPlan p = sg::xent_plan(c.M, c.N, c.K, c.K);
    EXPECT_RC(sg::xent_tile(c.M, c.N), c.product);
    EXPECT_RC(p.hidden.tile, c.hidden);
    EXPECT_RC(p.hidden.splits, c.splits);
    EXPECT_RC(sg::xent_back(p.words < c.N ? p.words : c.N, c.K, p.rows, 1).tile, c.head);
  }
}

static void balance() {
  auto run = [](int64_t T, int E, int k, int64_t ldl, const int32_t* ids, float* loss, void* w,
                int64_t wb) {
    return moe_balance_run(T, E, k, P, ldl, SG_F32, ids, SG_SCORE_SOFTMAX, loss, I, I, w, wb,
                           nullptr);
  };
  EXPECT_RC(run(-1, 40, 4, 40, I, F, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(run(kBig, 40, 4, 40, I, F, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(run(900, 257, 4, 257, I, F, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(run(900, 40, 41, 40, I, F, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(run(1 << 30, 40, 2, 40, I, F, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(run(900, 40, 4, 39, I, F, P, kBig), SG_ERR_SHAPE);
  EXPECT_RC(run(900, 40, 4, 40, nullptr, F, P, kBig), SG_ERR_NULL);
  EXPECT_RC(run(900, 40, 4, 40, I, nullptr, P, kBig), SG_ERR_NULL);
  EXPECT_RC(run(900, 40, 4, 40, I, F2, P, kBig), SG_ERR_ALIGN);
  EXPECT_RC(run(900, 40, 4, 40, I, F, P, 100), SG_ERR_SHAPE);
  EXPECT_RC(run(900, 40, 4, 40, I, F, nullptr, kBig), SG_ERR_NULL);
  EXPECT_RC(run(900, 40, 4, 40, I, F, Pc + 4, kBig), SG_ERR_ALIGN);
  auto back = [](int64_t T, int E, const float* d, void* out, int64_t ldo, int score) {
    return moe_balance_backward_run(T, E, d, P, 40, SG_BF16, I, I, score, out, ldo, nullptr);
  };
  EXPECT_RC(back(900, 40, F, P, 39, 0), SG_ERR_SHAPE);
  EXPECT_RC(back(900, 41, F, P, 41, 0), SG_ERR_SHAPE);
  EXPECT_RC(back(900, 40, nullptr, P, 40, 0), SG_ERR_NULL);
  EXPECT_RC(back(900, 40, F2, P, 40, 0), SG_ERR_ALIGN);
  EXPECT_RC(back(900, 40, F, Pc + 1, 40, 0), SG_ERR_ALIGN);
  EXPECT_RC(back(900, 40, F, P, 40, 7), SG_ERR_DTYPE);
  EXPECT_RC(back(0, 40, nullptr, nullptr, 40, 0), SG_OK);
  EXPECT_RC(moe_balance_workspace_bytes(kBig, 8), SG_ERR_SHAPE);
  for (int64_t T = 1; T < kMaxExtent; T += 1 + T / 2) {
    const int64_t chunk = balance_chunk(T), parts = cdiv(T, chunk);
    EXPECT_RC(chunk % 16 == 0 && parts >= 1 && parts <= 256 && (T > 256 || parts == 1), 1);
  }
}

int main() {
  cross_entropy();
  plans();
  choices();
  balance();
  if (fails) {
    std::fprintf(stderr, "%d check(s) failed\n", fails);
    return 1;
  }
  std::puts("losses ABI sanitizer run clean");
  return 0;
}
