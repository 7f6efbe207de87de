// xent_plans.cpp -- the plan of the cross entropy's gradient (xent_plan.h) on the
// host: what its kernels take for granted of a run of words, and the runs of the
// GPU tests' sizes.  Exit status 0 = all as stated.
#include <cstdio>

#include "../../dense_gemm_swizzled_amd/csrc/xent_plan.h"

static int fails = 0;
#define EXPECT(what)                                                                  \
  do {                                                                                \
    if (!(what)) {                                                                    \
      if (++fails <= 20)                                                              \
        std::fprintf(stderr, "%s:%d: %s (M=%lld N=%lld ldb=%lld)\n", __FILE__,        \
                     __LINE__, #what, (long long)M, (long long)N, (long long)ldb);    \
    }                                                                                 \
  } while (0)

// The products of dB take the gradient of the logits row by row, up to 96 rows
// past its last, by 32-bit offsets: its pitch is below 2^22 values like those of
// A and B, however many words there are.
static void pitches() {
  for (int64_t M : {1, 2, 31, 32, 33, 64, 65, 512, 8192, 100003})
    for (int64_t N : {1LL, 255LL, 131072LL, (1LL << 22) - 255, 1LL << 22, (1LL << 22) + 1,
                      10000000LL, 100000000LL, (1LL << 31) - 1})
      for (int64_t ldb : {8LL, 4096LL, (1LL << 22) - 8}) {
        const sg::XentPlan p = sg::xent_plan(M, N, ldb, ldb);
        const int64_t run = p.words < N ? p.words : N;
        EXPECT(p.ldg >= run && p.ldg < sg::kXentMaxLd);
        EXPECT(p.rows * p.ldg * 2 + 96 * p.ldg * 2 < int64_t{1} << 32);
        EXPECT(p.words % 256 == 0 && p.words > 0);
      }
}

// Few tokens in several runs of words: dA's parts, the last run of a single word
// and of fewer shares than the others.
static void runs() {
  const int64_t N = 10753, K = 136, ldb = int64_t{1} << 19;
  for (int64_t M : {1, 33, 64}) {
    const sg::XentPlan p = sg::xent_plan(M, N, K, ldb);
    EXPECT(p.words == 1792 && sg::cdiv(N, p.words) == 7 && N - 6 * p.words == 1);
    EXPECT(p.parts && p.rows == 2 * M && p.hidden.splits > 1);
  }
}

int main() {
  pitches();
  runs();
  if (fails) {
    std::fprintf(stderr, "%d check(s) failed\n", fails);
    return 1;
  }
  std::puts("plans as stated");
  return 0;
}
