// Descriptors of the serving operators' kernels: rotary positions and the
// key/value cache on low-precision grids (internal to the library).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attend_plan.h"

// One rotary call.  Strides count elements; table is [length][2][rot / 2].
struct RopeProb {
  const void* x;
  void* y;
  const int* pos;
  const float* table;
  long long tokens, xt, xh, yt, yh;
  int heads, dim, rot, length;
  float sign;  // +1: rotate; -1: rotate back
};

// Frequencies (radians per position) of a rotary table: 1 KB of kernel
// arguments instead of an upload.
struct RopeFreq {
  double f[128];
};

// The paged cache.  Per (page, head): k_codes [page][rb], v_codes [rb][page],
// rb = dim bits / 8; scales and zeros [page].
struct KvPool {
  uint8_t* kc;
  float* ks;
  uint8_t* kz;
  uint8_t* vc;
  float* vs;
  uint8_t* vz;
  int pages, heads, dim, rb;
  int pshift;  // tokens per page = 2^pshift
};

struct KvWriteProb {
  KvPool c;
  const void* k;
  const void* v;
  const int* slots;
  long long tokens, kt, kh, vt, vh;  // strides in elements
};

struct KvReadProb {
  KvPool c;
  void* k;
  void* v;
  const int* slots;
  long long tokens, kt, kh, vt, vh;
  int wide;    // rows are aligned to eight values
  int stream;  // stored past the caches
};

// Attention of seqs x tokens query tokens over the cache.
struct AttnProb : AttnPlan {
  KvPool c;
  const uint16_t* q;  // bf16 bits
  uint16_t* o;
  const int* tables;  // [seqs][width] page numbers
  const int* lengths; // [seqs] tokens before the drafted ones
  const uint32_t* mask;  // [seqs][tokens][words] or null: a chain
  long long qb, qt, qh, ob, ot, oh;
  int seqs, tokens, heads, group;  // group = heads / c.heads
  int width, words;
  float scale;  // of the scores, times log2(e)
  // workspace: unnormalised rows [unit][row][dim] with their {M, l}, and of each
  // sequence {first unit of head 0, shares}
  float* part;
  float* ml;
  int* info;
  int* count;  // one for each row block of a (sequence, key head), 0 between calls; null: k_attn_join follows
};

hipError_t launch_rope_table(const RopeFreq& f, int length, int half, double mag, float* table, hipStream_t st);
// types: 0 bf16, 1 float32; layout: 0 halves, 1 interleaved
hipError_t launch_rope(const RopeProb& p, int xtype, int ytype, int layout, hipStream_t st);
hipError_t launch_kv_write(const KvWriteProb& p, int type, int bits, hipStream_t st);
hipError_t launch_kv_read(KvReadProb p, int type, int bits, hipStream_t st);
void plan_tree_attn(AttnProb& p, int ncu);
hipError_t launch_attn_join(const AttnProb& p, hipStream_t st);
hipError_t launch_tree_attn(const AttnProb& p, int bits, hipStream_t st);
