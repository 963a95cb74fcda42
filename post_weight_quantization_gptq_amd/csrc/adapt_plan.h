// Which kernels take a quantised product with adapters, from the call's sizes alone (no
// HIP: the tests build this for the host).
#pragma once
#include <algorithm>
#include <cmath>
#include <cstddef>

struct AdaptPlan {
  int shape;  // of the product: 0 few rows, 1 .. 5 its tiles
  int parts;  // workgroups of a tile, shapes 1 and 2
  int splits, slots;  // of the first launch: shares of k, workgroups for the adapters of the same 32 rows
};

// The kernels for M rows, N outputs and K inputs on ncu compute units.
inline AdaptPlan plan_adapt(int M, int N, int K, int ncu) {
  AdaptPlan p{};
  // Few rows: up to 128 the weights are unpacked where they are used (128 rows of a
  // 4096 x 4096 layer 34 us in all, 41 through bf16 weights in memory; 192 rows 53 and 39).
  // Else the tiles whose rounds over the CUs take least.  us of a round at K = 4096, of which
  // 5 do not grow with K, and beside it: two 64 x 64 share a CU, halves are joined.  In
  // all, with rank 32 and 4096 outputs, in this order: 256 rows 41, 43, 54, 76, 111; 512 rows
  // 55, 45, 53, 73, 108; 1024 rows 79, 66, 58, 75, 108; 2048 rows 137, 112, 97, 85, 109; 3000
  // rows 196, 159, 137, 140, 117.  A 64 x 64 tile has as many workgroups as pay: 300 rows of 500
  // outputs (40 tiles), K = 4096, rank 16: 24 us with 1, 19, 17, 16, 16, 18 with 2, 3, 4, 6,
  // 8; K = 1024, 140 rows of 1024: 13.7, 12.7, 12.5, 13.5 with 1 to 4.
  struct Tile {
    int m, n;
    double round, more;
  };
  static const Tile tile[5] = {{64, 64, 24, 0}, {128, 128, 20, 5}, {128, 128, 40, 0}, {128, 256, 62, 0}, {256, 256, 105, 0}};
  const double fixed = 5.3;
  p.shape = 0;
  p.parts = 1;
  double best = 0.0;
  for (int i = 0; i < 5 && M > 128; ++i) {
    const double n = (double)((M + tile[i].m - 1) / tile[i].m) * ((N + tile[i].n - 1) / tile[i].n) / ncu;
    for (int parts = 1; parts <= (i == 0 ? std::min(8, std::max(K / 256, 1)) : 1); ++parts) {
      const double rounds = i == 0 ? std::max(1.0, 0.85 * n * parts) : std::ceil(i == 1 ? 2 * n : n);
      const double t = fixed + (tile[i].round * rounds - fixed) / parts * K / 4096 + tile[i].more +
                       (parts > 1 ? 1.7 + 1.1 * parts : 0.0);
      if (!p.shape || t < best) {
        p.shape = i + 1;
        p.parts = i == 1 ? 2 : parts;
        best = t;
      }
    }
  }
  // The first launch: workgroups for every adapter of 32 rows where there are few rows (64
  // rows with 48 adapters, 4096 x 4096: 9 us, 137 with one), else one that takes them in
  // turn (4096 rows with five: 20, with two 22, with four 33); two shares of k (24 us
  // with one), four where there are few workgroups.  Each share is read again in the
  // second launch (64 rows: 20, 21, 24, 30 us with 1, 2, 4, 8).
  const int groups = (M + 31) / 32;
  p.slots = std::min(std::max(ncu / (2 * groups), 1), std::min(M, 32));
  p.splits = K < 1024 ? 1 : K >= 2048 && groups * p.slots < ncu / 8 ? 4 : 2;
  return p;
}

// Tiles that several workgroups have (0: none do), and the bytes that those need for their
// sums and for their counts.
inline size_t adapt_tiles(const AdaptPlan& p, int M, int N) {
  const int side = p.shape == 1 ? 64 : 128;
  return p.parts > 1 ? (size_t)((M + side - 1) / side) * ((N + side - 1) / side) : 0;
}
inline size_t adapt_part(const AdaptPlan& p, int M, int N) {
  return adapt_tiles(p, M, N) * p.parts * (p.shape == 1 ? 64 * 64 : 128 * 128) * sizeof(float);
}
inline size_t adapt_done(const AdaptPlan& p, int M, int N) { return adapt_tiles(p, M, N) * sizeof(int); }

// Whether the threads of every launch can be counted in 32 bits.
inline bool adapt_fits(const AdaptPlan& p, int M, int N, int K) {
  static const struct {
    int m, n, threads;
  } tile[5] = {{64, 64, 256}, {128, 128, 512}, {128, 128, 512}, {128, 256, 512}, {256, 256, 512}};
  const long long per = (K / 32 + 15) / 16;  // workgroups of 16 rows of X or of the weights
  const long long down = (M + 31LL) / 32 * p.splits * p.slots + ((p.shape ? N : M) + 15LL) / 16 * per;
  long long product = (N + 15LL) / 16 * 512;
  if (p.shape) {
    const auto& t = tile[p.shape - 1];
    product = ((long long)M + t.m - 1) / t.m * (((long long)N + t.n - 1) / t.n) * p.parts * t.threads;
  }
  return down * 256 < 1LL << 32 && product < 1LL << 32;
}
