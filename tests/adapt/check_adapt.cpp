// Host-only checks of the choice of kernels for products with adapters (csrc/adapt_plan.h), built with
// AddressSanitizer and UndefinedBehaviorSanitizer by tests/test_adapt_plan.py.
#include <stdio.h>
#include <stdlib.h>

#include "adapt_plan.h"

static int g_fail = 0;
#define CHECK(cond, ...)                                        \
  do {                                                          \
    if (!(cond)) {                                              \
      fprintf(stderr, "FAIL %s:%d: ", __FILE__, __LINE__);      \
      fprintf(stderr, __VA_ARGS__);                             \
      fputc('\n', stderr);                                      \
      if (++g_fail > 25) exit(1);                               \
    }                                                           \
  } while (0)

// The kernel that takes a size: the GPU tests take these to reach every one.
static void check_choice(int M, int N, int K, int shape, int parts) {
  const AdaptPlan p = plan_adapt(M, N, K, 256);
  CHECK(p.shape == shape && p.parts == parts, "%d x %d x %d: shape %d of %d workgroups", M, N, K, p.shape, p.parts);
}

static void check_refused(int M, int N, int K) {
  CHECK(!adapt_fits(plan_adapt(M, N, K, 256), M, N, K), "%d x %d x %d: said to fit", M, N, K);
}

// What the kernels and their launches assume.
static void check_limits(int M, int N, int K) {
  const AdaptPlan p = plan_adapt(M, N, K, 256);
  CHECK(p.shape >= 0 && p.shape <= 5 && (p.shape == 0) == (M <= 128), "%d x %d x %d: shape %d", M, N, K, p.shape);
  CHECK(p.parts >= 1 && p.parts <= 8 && (p.parts == 1 || p.shape == 1 || p.shape == 2) && (p.shape != 2 || p.parts == 2),
        "%d x %d x %d: shape %d of %d workgroups", M, N, K, p.shape, p.parts);
  CHECK(p.slots >= 1 && p.slots <= 32 && p.slots <= M && p.splits >= 1 && p.splits <= 4, "%d rows, K %d: %d slots, %d shares", M, K,
        p.slots, p.splits);
  static const int side[6][2] = {{0, 0}, {64, 64}, {128, 128}, {128, 128}, {128, 256}, {256, 256}};
  const int threads = p.shape == 1 ? 256 : 512;
  bool small = (N + 15LL) / 16 * 512 < 1LL << 32;
  if (p.shape) {
    const long long tiles = ((long long)M + side[p.shape][0] - 1) / side[p.shape][0] *
                            (((long long)N + side[p.shape][1] - 1) / side[p.shape][1]);
    small = tiles * p.parts * threads < 1LL << 32;
    CHECK(adapt_tiles(p, M, N) == (p.parts > 1 ? (size_t)tiles : 0), "%d x %d x %d: %zu counts", M, N, K, adapt_tiles(p, M, N));
    CHECK(adapt_part(p, M, N) == adapt_tiles(p, M, N) * p.parts * side[p.shape][0] * side[p.shape][1] * 4 &&
              adapt_done(p, M, N) == adapt_tiles(p, M, N) * 4,
          "%d x %d x %d: %zu bytes of sums", M, N, K, adapt_part(p, M, N));
  }
  const long long steps = K / 32, per = (steps + 15) / 16;
  const long long first = ((long long)M + 31) / 32 * p.splits * p.slots + ((p.shape ? N : M) + 15LL) / 16 * per;
  small = small && first * 256 < 1LL << 32;
  CHECK(adapt_fits(p, M, N, K) == small, "%d x %d x %d: said to %s", M, N, K, small ? "be too large" : "fit");
  // the weights as bf16 and Y take up to 200 GB
  const long long bytes = (p.shape ? 2LL * N * K : 0) + 4LL * M * N;
  CHECK(small || bytes > 200LL << 30, "%d x %d x %d: does not fit", M, N, K);
}

int main() {
  // every tile, and rows of few outputs
  check_choice(150, 300, 96, 1, 1);
  check_choice(500, 3990, 4128, 2, 2);
  check_choice(1000, 4000, 96, 3, 1);
  check_choice(2048, 4090, 96, 4, 1);
  check_choice(4090, 4096, 160, 5, 1);
  // 64 x 64 tiles of one to eight workgroups
  check_choice(640, 900, 4448, 1, 2);
  check_choice(333, 1500, 2080, 1, 2);
  check_choice(300, 500, 2048, 1, 3);
  check_choice(141, 303, 3968, 1, 4);
  check_choice(200, 260, 6176, 1, 5);
  check_choice(131, 70, 8192, 1, 6);
  check_choice(129, 64, 12320, 1, 7);
  check_choice(131, 70, 16384, 1, 8);
  // the sizes of the tests of every kernel
  check_choice(3, 40, 32, 0, 1);
  check_choice(30, 200, 64, 0, 1);
  check_choice(60, 333, 160, 0, 1);
  check_choice(100, 500, 32, 0, 1);
  check_choice(128, 2100, 96, 0, 1);
  check_choice(200, 700, 64, 1, 1);
  check_choice(200, 700, 2048, 1, 3);
  check_choice(500, 4090, 1280, 2, 2);
  check_choice(700, 3000, 32, 3, 1);
  check_choice(2000, 3800, 32, 4, 1);
  check_choice(2500, 4000, 32, 5, 1);
  // the refused ones of the GPU tests
  check_refused(1000, 1 << 26, 0);
  check_refused(200, 1 << 20, 1 << 17);
  check_refused(16384, 1 << 20, 1 << 17);
  check_refused(16384, 1 << 26, 32);
  for (int M : {1, 2, 16, 17, 100, 128, 129, 200, 999, 2048, 4096, 10000, 16384})
    for (int N : {1, 15, 64, 300, 2049, 4096, 11008, 14336, 128256, 1 << 20, 1 << 23, 1 << 26})
      for (int K : {0, 32, 96, 1024, 2048, 4096, 14336, 1 << 17, 1 << 22})
        check_limits(M, N, K);
  if (g_fail) return 1;
  printf("adapter checks passed\n");
  return 0;
}
