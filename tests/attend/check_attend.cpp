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

// A plan that is said to fit: no number of it has overflowed, and the launches' threads are fewer than 2^32; one
// that is said not to: they are not.
static void check_limits(long long R, int seqs, int kv_heads, int dim, long long hold) {
  const AttnPlan p = plan_attention(R, seqs, kv_heads, dim, hold, 256);
  const __int128 rows = (__int128)R * seqs * kv_heads;
  const int block = p.wide ? (p.nb == 1 ? 64 : 128) : 16 * p.nb;
  CHECK((long long)p.nrb * block >= R && (long long)(p.nrb - 1) * block < R, "R %lld: %d blocks of %d", R, p.nrb, block);
  CHECK(p.nb >= 1 && p.nb <= (p.wide ? (dim <= 128 ? 2 : 1) : dim <= 128 ? 3 : 2), "R %lld dim %d: nb %d", R, dim, p.nb);
  CHECK(p.units >= (long long)seqs * kv_heads && p.kept >= 0 && p.fit >= 1, "seqs %d heads %d: %d units", seqs, kv_heads, p.units);
  const JoinPlan j = plan_join(dim, p.shares);
  // k_tree_attn: four waves for up to 16 rows and for heads above 128, else eight; k_tree_attn_wide: four
  const int waves = p.wide || p.nb == 1 || dim > 128 ? 4 : 8;
  const __int128 attn = ((__int128)p.units + 7) / 8 * 8 * p.nrb * waves * 64;
  const __int128 join = p.most > 1 ? (rows + j.rows - 1) / j.rows * j.threads : 0;
  const bool small = attn < (__int128)1 << 32 && join < (__int128)1 << 32;
  CHECK(attention_fits(p, (long long)rows, dim) == small, "R %lld seqs %d heads %d dim %d", R, seqs, kv_heads, dim);
}

// The kernel that takes a call of R rows a key head: the GPU tests take these row counts to reach every one.
static void check_choice(int dim, long long R, int wide, int nb, int nrb) {
  const AttnPlan p = plan_attention(R, 1, 1, dim, 2, 256);
  CHECK(!!p.wide == !!wide && p.nb == nb && p.nrb == nrb, "dim %d rows %lld: wide %d, nb %d, %d blocks", dim, R, p.wide, p.nb, p.nrb);
}

int main() {
  for (int dim : {64, 96, 128}) {
    check_choice(dim, 10, 0, 1, 1);
    check_choice(dim, 20, 0, 2, 1);
    check_choice(dim, 40, 0, 3, 1);
    check_choice(dim, 64, 1, 1, 1);
    check_choice(dim, 80, 0, 3, 2);
    check_choice(dim, 128, 1, 2, 1);
  }
  for (int dim : {192, 256}) {
    check_choice(dim, 10, 0, 1, 1);
    check_choice(dim, 20, 0, 2, 1);
    check_choice(dim, 64, 1, 1, 1);
    check_choice(dim, 80, 0, 2, 3);
  }
  for (int dim : {64, 96, 128, 192, 256})
    for (long long R : {1LL, 16LL, 17LL, 48LL, 49LL, 64LL, 65LL, 128LL, 129LL, 1000LL, 1LL << 20, 1LL << 26})
      for (int heads : {1, 3, 8, 64, 65535})
        for (int seqs : {1, 2, 65, 4096, 1 << 18, 1 << 20, 1 << 24, 1 << 28})
          for (long long hold : {0LL, 1LL, 64LL, 1LL << 21})
            if ((__int128)R * heads <= 1 << 26 && (__int128)R * heads * seqs <= 1 << 30) check_limits(R, seqs, heads, dim, hold);
  for (int dim : {64, 96, 128, 192, 256})
    for (int shares : {2, 3, 8, 9, 15, 16, 17, 64, 512}) check_join(dim, shares);
  if (g_fail) return 1;
  printf("attention checks passed\n");
  return 0;
}
