// Descriptor of the quantised product with adapters (internal to the library).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "adapt_plan.h"

struct AdaptProb : AdaptPlan {
  const uint16_t* X;  // bf16 bits, row pitch ldx
  const uint32_t* P;  // [N][K bits / 32] row bitstreams
  const float* S;     // [N][G]
  const uint8_t* Z;   // [N][G]
  const uint16_t* down;  // [count][rank][K]
  const uint16_t* up;    // [count][N][rank]
  const float* alpha;    // [count] or null: 1
  const int* ids;        // [M]; outside 0 .. count - 1: no adapter
  float* T;              // workspace [splits][M][rank]: shares of X down^T
  uint16_t* XB;          // workspace, shape 0: X in blocks, M up to 16 and K up to 128
  uint16_t* W;           // workspace, shape > 0: the weights as bf16, ((N + 15) / 16) 16 K
  float* part;           // workspace, parts > 1: the sums of every tile
  int* done;             // one for every tile, 0 between calls
  float* Y;              // row pitch ldy
  long long ldx, ldy;
  int M, N, K, G;
  int gshift;  // group = 2^gshift (31: one group a row)
  int count, rank;
  int wdown, wrows;  // workgroups of the first launch's first two kinds
};

hipError_t launch_adapt_down(const AdaptProb& p, int bits, hipStream_t st);
hipError_t launch_adapt_product(const AdaptProb& p, int bits, hipStream_t st);
