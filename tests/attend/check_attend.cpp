// Host-only checks of the attention's launch shapes (csrc/attend_plan.h), built
// with AddressSanitizer and UndefinedBehaviorSanitizer by tests/test_attend_plan.py.
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "attend_plan.h"

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

// The threads of a joining workgroup: every (row, four values, share run) has
// one, and the first of a group finds its partners inside the shared array.
static void check_join(int dim, int shares) {
  const JoinPlan j = plan_join(dim, shares);
  const int q4 = dim / 4;
  CHECK(j.rows >= 1 && j.threads <= 256, "dim %d shares %d: %d rows, %d threads", dim, shares, j.rows, j.threads);
  std::vector<int> hit((size_t)j.rows * q4 * j.G, 0);
  for (int tid = 0; tid < j.threads; ++tid) {
    const JoinThread t = join_thread(tid, dim, j.G);
    CHECK(t.k >= 0 && t.k < j.G && t.d >= 0 && t.d + 3 < dim, "dim %d thread %d", dim, tid);
    if (t.i < j.rows) ++hit[((size_t)t.i * j.G + t.k) * q4 + t.d / 4];
    if (t.k != 0) continue;
    for (int e = 1; e < j.G; ++e) {
      const int other = tid + e * q4;
      CHECK(other < 256, "dim %d shares %d: thread %d reads sum %d of 256", dim, shares, tid, other);
      const JoinThread o = join_thread(other, dim, j.G);
      CHECK(other < j.threads && o.i == t.i && o.k == e && o.d == t.d, "dim %d: thread %d's partner %d", dim, tid, e);
    }
  }
  for (size_t i = 0; i < hit.size(); ++i) CHECK(hit[i] == 1, "dim %d: part %zu has %d threads", dim, i, hit[i]);
}

int main() {
  for (int dim : {64, 96, 128, 192, 256})
    for (int shares : {2, 3, 8, 9, 15, 16, 17, 64, 512}) check_join(dim, shares);
  if (g_fail) return 1;
  printf("attention checks passed\n");
  return 0;
}
