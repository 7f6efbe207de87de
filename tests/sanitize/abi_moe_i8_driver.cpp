// abi_moe_i8_driver.cpp -- drives the validation paths of the expert-routing
// and 8-bit entry points (include/swizzled_gemm.h) on the host, for an
// AddressSanitizer + UndefinedBehaviorSanitizer build of the library's host
// code, which it contains as source: so it also checks which kernel the tile
// choice takes for each size that the GPU tests run every kernel with.  Every
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
static int32_t* const I = reinterpret_cast<int32_t*>(Pc);
static const float* const F2 = reinterpret_cast<const float*>(Pc + 2);
static int32_t* const I2 = reinterpret_cast<int32_t*>(Pc + 2);
static const int64_t kBig = int64_t{1} << 62;

static int gemm(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const float* SA,
                const void* B, int64_t ldb, const float* SB, void* D, int64_t ldd, int dt) {
  return i8_gemm_run(M, N, K, A, lda, SA, B, ldb, SB, D, ldd, dt, nullptr);
}

static void products() {
  EXPECT_RC(gemm(-1, 40, 64, P, 64, F, P, 64, F, P, 40, SG_BF16), SG_ERR_SHAPE);
  EXPECT_RC(gemm(33, -1, 64, P, 64, F, P, 64, F, P, 40, SG_BF16), SG_ERR_SHAPE);
  EXPECT_RC(gemm(33, 40, -16, P, 64, F, P, 64, F, P, 40, SG_BF16), SG_ERR_SHAPE);
  EXPECT_RC(gemm(33, 40, 72, P, 80, F, P, 80, F, P, 40, SG_BF16), SG_ERR_SHAPE);
  EXPECT_RC(gemm(33, 40, 131072, P, 131072, F, P, 131072, F, P, 40, SG_BF16), SG_ERR_SHAPE);
  EXPECT_RC(gemm(33, 40, 64, P, 48, F, P, 64, F, P, 40, SG_BF16), SG_ERR_SHAPE);
  EXPECT_RC(gemm(33, 40, 64, P, 64, F, P, 64, F, P, 39, SG_BF16), SG_ERR_SHAPE);
  EXPECT_RC(gemm(33, 40, 64, P, kBig, F, P, 64, F, P, 40, SG_BF16), SG_ERR_SHAPE);
  EXPECT_RC(gemm(33, 40, 64, P, 64, F, P, kBig, F, P, 40, SG_BF16), SG_ERR_SHAPE);
  EXPECT_RC(gemm(33, 40, 64, P, 1 << 30, F, P, 64, F, P, 40, SG_BF16), SG_ERR_SHAPE);
  EXPECT_RC(gemm(kBig, 40, 64, P, 64, F, P, 64, F, P, 40, SG_BF16), SG_ERR_SHAPE);
  EXPECT_RC(gemm(33, kBig, 64, P, 64, F, P, 64, F, P, kBig, SG_BF16), SG_ERR_SHAPE);
  EXPECT_RC(gemm(1, 1 << 29, 16, P, 16, F, P, 16, F, P, 1 << 29, SG_BF16), SG_ERR_SHAPE);
  EXPECT_RC(gemm(33, 40, 64, P, 64, F, P, 64, F, P, 40, SG_E4M3), SG_ERR_DTYPE);
  EXPECT_RC(gemm(33, 40, 64, nullptr, 64, F, P, 64, F, P, 40, SG_F32), SG_ERR_NULL);
  EXPECT_RC(gemm(33, 40, 64, P, 64, nullptr, P, 64, F, P, 40, SG_F32), SG_ERR_NULL);
  EXPECT_RC(gemm(33, 40, 64, P, 64, F, P, 64, nullptr, P, 40, SG_F32), SG_ERR_NULL);
  EXPECT_RC(gemm(33, 40, 64, P, 64, F, P, 64, F, nullptr, 40, SG_F32), SG_ERR_NULL);
  EXPECT_RC(gemm(33, 40, 64, Pc + 8, 64, F, P, 64, F, P, 40, SG_F32), SG_ERR_ALIGN);
  EXPECT_RC(gemm(33, 40, 64, P, 72, F, P, 64, F, P, 40, SG_F32), SG_ERR_ALIGN);
  EXPECT_RC(gemm(33, 40, 64, P, 64, F2, P, 64, F, P, 40, SG_F32), SG_ERR_ALIGN);
  EXPECT_RC(gemm(33, 40, 64, P, 64, F, P, 64, F, Pc + 2, 40, SG_F32), SG_ERR_ALIGN);
  EXPECT_RC(gemm(0, 40, 64, nullptr, 64, nullptr, P, 64, F, nullptr, 40, SG_F32), SG_OK);
  EXPECT_RC(gemm(33, 0, 64, P, 64, F, nullptr, 64, nullptr, nullptr, 0, SG_F32), SG_OK);

  auto grouped = [](int G, int64_t R, const int32_t* off, int64_t lda, int64_t a_rows,
                    const int32_t* rows, const void* A, const float* SA) {
    return i8_grouped_gemm_run(G, R, 40, 64, off, A, lda, a_rows, rows, SA, P, F, P, 40, SG_F16,
                               nullptr);
  };
  EXPECT_RC(grouped(0, 33, I, 64, 33, I, P, F), SG_ERR_GROUPS);
  EXPECT_RC(grouped(257, 33, I, 64, 33, I, P, F), SG_ERR_GROUPS);
  EXPECT_RC(grouped(4, -1, I, 64, 33, I, P, F), SG_ERR_SHAPE);
  EXPECT_RC(grouped(4, 33, I, 64, 32, nullptr, P, F), SG_ERR_SHAPE);
  EXPECT_RC(grouped(4, 33, I, 64, -1, I, P, F), SG_ERR_SHAPE);
  EXPECT_RC(grouped(4, 33, I, 64, 1 << 26, I, P, F), SG_ERR_SHAPE);
  EXPECT_RC(grouped(4, 33, I, kBig, 33, I, P, F), SG_ERR_SHAPE);
  EXPECT_RC(grouped(4, 33, nullptr, 64, 33, I, P, F), SG_ERR_NULL);
  EXPECT_RC(grouped(4, 33, I, 64, 33, I, nullptr, F), SG_ERR_NULL);
  EXPECT_RC(grouped(4, 33, I2, 64, 33, I, P, F), SG_ERR_ALIGN);
  EXPECT_RC(grouped(4, 33, I, 64, 33, I2, P, F), SG_ERR_ALIGN);
  EXPECT_RC(grouped(4, 0, I, 64, 0, I, nullptr, nullptr), SG_OK);

  auto quant = [](int64_t R, int64_t K, const void* X, int64_t ldx, int dt, void* Q, int64_t ldq,
                  float* S) { return i8_quant_run(R, K, X, ldx, dt, Q, ldq, S, nullptr); };
  EXPECT_RC(quant(-1, 50, P, 50, SG_F32, P, 64, F), SG_ERR_SHAPE);
  EXPECT_RC(quant(3, kBig, P, kBig, SG_F32, P, kBig, F), SG_ERR_SHAPE);
  EXPECT_RC(quant(3, 50, P, 49, SG_F32, P, 64, F), SG_ERR_SHAPE);
  EXPECT_RC(quant(3, 50, P, 50, SG_F32, P, 48, F), SG_ERR_SHAPE);
  EXPECT_RC(quant(3, 50, P, 50, SG_F32, P, 72, F), SG_ERR_ALIGN);
  EXPECT_RC(quant(3, 50, Pc + 2, 50, SG_F32, P, 64, F), SG_ERR_ALIGN);
  EXPECT_RC(quant(3, 50, P, 50, SG_E8M0, P, 64, F), SG_ERR_DTYPE);
  EXPECT_RC(quant(3, 50, nullptr, 50, SG_F16, P, 64, F), SG_ERR_NULL);
  EXPECT_RC(quant(3, 50, P, 50, SG_F16, P, 64, nullptr), SG_ERR_NULL);
  EXPECT_RC(quant(0, 50, nullptr, 50, SG_F16, nullptr, 64, nullptr), SG_OK);
}

static void routing() {
  auto route = [](int64_t T, int E, int k, const void* x, int64_t ldl, int dt, const float* bias,
                  int score, int groups, int top, int gs, float* w, int32_t* ids) {
    return moe_route_run(T, E, k, x, ldl, dt, bias, score, groups, top, gs, 1, 1.0f, w, ids,
                         nullptr);
  };
  EXPECT_RC(route(-1, 16, 2, P, 16, SG_F32, nullptr, 0, 1, 1, 0, F, I), SG_ERR_SHAPE);
  EXPECT_RC(route(kBig, 16, 2, P, 16, SG_F32, nullptr, 0, 1, 1, 0, F, I), SG_ERR_SHAPE);
  EXPECT_RC(route(3, 257, 2, P, 300, SG_F32, nullptr, 0, 1, 1, 0, F, I), SG_ERR_SHAPE);
  EXPECT_RC(route(3, 16, 17, P, 16, SG_F32, nullptr, 0, 1, 1, 0, F, I), SG_ERR_SHAPE);
  EXPECT_RC(route(3, 64, 33, P, 64, SG_F32, nullptr, 0, 1, 1, 0, F, I), SG_ERR_SHAPE);
  EXPECT_RC(route(3, 16, 2, P, 15, SG_F32, nullptr, 0, 1, 1, 0, F, I), SG_ERR_SHAPE);
  EXPECT_RC(route(3, 16, 2, P, 16, SG_E4M3, nullptr, 0, 1, 1, 0, F, I), SG_ERR_DTYPE);
  EXPECT_RC(route(3, 16, 2, P, 16, SG_F32, nullptr, 2, 1, 1, 0, F, I), SG_ERR_DTYPE);
  EXPECT_RC(route(3, 16, 2, P, 16, SG_F32, nullptr, 0, 3, 1, 0, F, I), SG_ERR_GROUPS);
  EXPECT_RC(route(3, 16, 2, P, 16, SG_F32, nullptr, 0, 0, 1, 0, F, I), SG_ERR_GROUPS);
  EXPECT_RC(route(3, 64, 2, P, 64, SG_F32, nullptr, 0, 64, 1, 0, F, I), SG_ERR_GROUPS);
  EXPECT_RC(route(3, 16, 2, P, 16, SG_F32, nullptr, 0, 4, 5, 0, F, I), SG_ERR_GROUPS);
  EXPECT_RC(route(3, 16, 5, P, 16, SG_F32, nullptr, 0, 4, 1, 0, F, I), SG_ERR_GROUPS);
  EXPECT_RC(route(3, 16, 2, P, 16, SG_F32, nullptr, 0, 4, 1, 2, F, I), SG_ERR_GROUPS);
  EXPECT_RC(route(3, 16, 2, nullptr, 16, SG_F32, nullptr, 0, 1, 1, 0, F, I), SG_ERR_NULL);
  EXPECT_RC(route(3, 16, 2, P, 16, SG_F32, nullptr, 0, 1, 1, 0, nullptr, I), SG_ERR_NULL);
  EXPECT_RC(route(3, 16, 2, P, 16, SG_F32, F2, 0, 1, 1, 0, F, I), SG_ERR_ALIGN);
  EXPECT_RC(route(3, 16, 2, P, 16, SG_F32, nullptr, 0, 1, 1, 0, F, I2), SG_ERR_ALIGN);
  EXPECT_RC(route(3, 16, 2, Pc + 1, 16, SG_F16, nullptr, 0, 1, 1, 0, F, I), SG_ERR_ALIGN);
  EXPECT_RC(route(0, 16, 2, nullptr, 16, SG_F32, nullptr, 0, 1, 1, 0, nullptr, nullptr), SG_OK);

  auto back = [](int64_t T, int k, const float* dw, const void* x, int dt, const int32_t* ids,
                 void* out, int64_t lddl) {
    return moe_route_backward_run(T, 16, k, dw, x, 16, dt, ids, 0, 1, 1.0f, out, lddl, nullptr);
  };
  EXPECT_RC(back(-1, 2, F, P, SG_F32, I, P, 16), SG_ERR_SHAPE);
  EXPECT_RC(back(3, 17, F, P, SG_F32, I, P, 16), SG_ERR_SHAPE);
  EXPECT_RC(back(3, 2, F, P, SG_F32, I, P, 15), SG_ERR_SHAPE);
  EXPECT_RC(back(3, 2, F, P, 0, I, P, 16), SG_ERR_DTYPE);
  EXPECT_RC(back(3, 2, nullptr, P, SG_F32, I, P, 16), SG_ERR_NULL);
  EXPECT_RC(back(3, 2, F, P, SG_F32, I, nullptr, 16), SG_ERR_NULL);
  EXPECT_RC(back(3, 2, F2, P, SG_F32, I, P, 16), SG_ERR_ALIGN);
  EXPECT_RC(back(3, 2, F, P, SG_F32, I, Pc + 2, 16), SG_ERR_ALIGN);
  EXPECT_RC(back(0, 2, nullptr, nullptr, SG_F32, nullptr, nullptr, 16), SG_OK);

  auto plan = [](int64_t T, int E, int k, const int32_t* ids, int32_t* off, void* ws, int64_t n) {
    return moe_plan_run(T, E, k, ids, off, I, I, ws, n, nullptr);
  };
  EXPECT_RC(plan(-1, 16, 2, I, I, nullptr, 0), SG_ERR_SHAPE);
  EXPECT_RC(plan(3, 257, 2, I, I, nullptr, 0), SG_ERR_SHAPE);
  EXPECT_RC(plan(3, 16, 257, I, I, nullptr, 0), SG_ERR_SHAPE);
  EXPECT_RC(plan(1 << 30, 16, 2, I, I, nullptr, 0), SG_ERR_SHAPE);
  EXPECT_RC(plan(3, 16, 2, nullptr, I, nullptr, 0), SG_ERR_NULL);
  EXPECT_RC(plan(3, 16, 2, I, nullptr, nullptr, 0), SG_ERR_NULL);
  EXPECT_RC(plan(9000, 16, 2, I, I, nullptr, 1 << 20), SG_ERR_NULL);
  EXPECT_RC(plan(9000, 16, 2, I, I, P, 16), SG_ERR_SHAPE);
  EXPECT_RC(plan(3, 16, 2, I, I, Pc + 2, 0), SG_ERR_ALIGN);
  EXPECT_RC(plan(3, 16, 2, I2, I, nullptr, 0), SG_ERR_ALIGN);

  EXPECT_RC(moe_plan_workspace_bytes(-1, 8), SG_ERR_SHAPE);
  EXPECT_RC(moe_plan_workspace_bytes(8, 257), SG_ERR_SHAPE);
  EXPECT_RC(moe_plan_workspace_bytes(int64_t{1} << 31, 8), SG_ERR_SHAPE);
  EXPECT_RC(moe_plan_workspace_bytes(kPlanAlone, 256), 0);
  // Chunks cover the pairs, in whole steps of every wave, with few counts.
  for (int E = 1; E <= SG_MAX_GROUPS; E = 2 * E + 1 - E % 2)
    for (int64_t n = kPlanAlone + 1; n < kMaxExtent; n += n / 3) {
      const int64_t chunk = plan_chunk(n, E), blocks = cdiv(n, chunk);
      EXPECT_RC(chunk % 1024 == 0 && blocks * chunk >= n && blocks <= 256, 1);
      EXPECT_RC(moe_plan_workspace_bytes(n, E), blocks * E * 4);
    }
}

static void choices() {
  struct Choice {
    int64_t M, N, K;
    sg::I8Tile want;
  };
  const Choice dense[] = {
      {1, 4096, 1040, sg::kI8Stream16x16},   {7, 4500, 1040, sg::kI8Stream16x32},
      {16, 33000, 112, sg::kI8Stream16x64},  {20, 200, 528, sg::kI8Stream32x16},
      {29, 5001, 528, sg::kI8Stream32x32},   {32, 9000, 272, sg::kI8Stream32x32x2},
      {50, 2900, 1040, sg::kI8Stream64x32},  {64, 9000, 272, sg::kI8Mid64x64},
      {333, 4104, 1040, sg::kI8Mid64x128},   {768, 4096, 1040, sg::kI8Mid128x128},
      {4096, 4096, 128, sg::kI8PingPong256}};
  for (const Choice& c : dense)
    EXPECT_RC(pick_i8_dense(c.M, c.N, c.K, true), c.want);
  // Panels that 256 rows would push past 32-bit offsets never take 256x256.
  for (int64_t M = 1; M < (1 << 24); M = 3 * M + 1)
    for (int64_t N = 16; N < (1 << 20); N = 5 * N + 3) {
      EXPECT_RC(pick_i8_dense(M, N, 4096, false) == sg::kI8PingPong256, 0);
      EXPECT_RC(pick_i8_grouped(M, 8, N, 4096, false) == sg::kI8PingPong256, 0);
    }
}

int main() {
  products();
  routing();
  choices();
  if (fails) {
    std::fprintf(stderr, "%d check(s) failed\n", fails);
    return 1;
  }
  std::puts("routing and 8-bit ABI sanitizer run clean");
  return 0;
}
