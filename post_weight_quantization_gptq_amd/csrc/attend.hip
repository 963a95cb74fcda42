// Attention of drafted tokens over the quantised cache (gfx950).
#include "common.h"
#include "serve.h"

#include <algorithm>

// running maximum of a row that has seen nothing (finite: its product with a zero scale is 0)
#define NONE (-3.402823466e38f)

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

namespace {

// Codes enter the matrix unit as float16 without a conversion: 0x6400 | c is
// 1024 + c.  Two bytes of w, at bit 0 and 8 (half 0) or 16 and 24 (half 1):
__device__ __forceinline__ uint32_t bytes2(uint32_t w, int half) {
  return __builtin_amdgcn_perm(0x64646464u, w, half ? 0x04030402u : 0x04010400u);
}
// the nibbles at bits 0 and 16 as 1024 + c, and those at bits 4 and 20 as 1024
// + 16 c: one instruction each with both constants in registers (the compiler
// takes two, with literals)
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask) {
  uint32_t r;
  asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(w), "s"(mask), "v"(0x64006400u));
  return r;
}
__device__ __forceinline__ uint32_t nib_lo(uint32_t w) { return and_or(w, 0x000F000Fu); }
__device__ __forceinline__ uint32_t nib_hi(uint32_t w) { return and_or(w, 0x00F000F0u); }

__device__ __forceinline__ uint32_t sub16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, a) - __builtin_bit_cast(f16x2, b));
}
// float16 pair c minus float16 pair z as a bfloat16 pair (exact for integers up to 256)
__device__ __forceinline__ uint32_t diff_bf16(uint32_t c, uint32_t z) {
  uint32_t lo, hi;
  asm("v_fma_mix_f32 %0, %1, 1.0, -%2 op_sel_hi:[1,0,1]" : "=v"(lo) : "v"(c), "v"(z));
  asm("v_fma_mix_f32 %0, %1, 1.0, -%2 op_sel:[1,0,1] op_sel_hi:[1,0,1]" : "=v"(hi) : "v"(c), "v"(z));
  return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}
// Two floats as the sum of two bfloat16 pairs: each to the nearest (ties to
// even), then what that left (exact in float32) to the nearest.  As many
// instructions as cutting both off, which would leave every weight, and so every
// result, too small by 2^-17 on average.
__device__ __forceinline__ uint32_t near16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ void split16(float a, float b, uint32_t& lead, uint32_t& next) {
  lead = near16(a, b);
  next = near16(a - __uint_as_float(lead << 16), b - __uint_as_float(lead & 0xFFFF0000u));
}

// largest value (sum) of the four lanes that differ in lane / 16
__device__ __forceinline__ float max_groups(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_groups(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// A value that is the same in all lanes, as such.
__device__ __forceinline__ size_t uniform(size_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (size_t)hi << 32 | lo;
}
// Entry of a table that nothing writes during the launch, at an address that is
// the same in all lanes: read through the scalar cache.
__device__ __forceinline__ int scalar_load(const int* p) {
  typedef const __attribute__((address_space(4))) int cint;
  return *(cint*)uniform((size_t)p);
}
// A load that asks the caches not to keep what is read once (32 contexts of
// 8192 tokens: 83.4 against 85.7 us; where blocks share the codes it costs: 108
// rows of 4000 positions 48 against 45 us).
template <bool ONCE, class V>
__device__ __forceinline__ V fetch(const V* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(glb(p));
  return *glb(p);
}

__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_bf(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

// One tile of TP positions as a lane holds it: see k_tree_attn.
template <int DIM, int BITS, int TP>
struct Tile {
  static constexpr int CH = TP / 4;          // positions whose weights a lane has: a chunk
  static constexpr int NI = CH / 4;          // blocks of 16 key rows
  static constexpr int NS = CH / 8;          // steps of 32 positions of the second product
  static constexpr int RB = DIM * BITS / 8;  // bytes of a key row; byte rows of a value block
  static constexpr int NW = RB / 16;         // words of a key row per lane
  static constexpr int NF = RB / 64;         // ... whole 64-byte pieces
  static constexpr bool R32 = RB % 64 >= 32, R16 = RB % 32 != 0;
  static constexpr int NMB = RB / 16;        // blocks of 16 byte rows of values
  typedef uint32_t Chunk __attribute__((ext_vector_type(NI)));  // a byte for each position of a chunk
  uint32_t k[NI][NW];
  Chunk v[NMB];
  f32x4 ks[NI], vs[NI];
  Chunk kz, vz;  // of the lane's key rows' chunk, of its own
  bool bad;

  // byte offset in a key row of word w of lane group g
  static __device__ __forceinline__ constexpr int off(int w, int g) {
    if (w < 4 * NF) return 64 * (w / 4) + 16 * g + 4 * (w % 4);
    if (R32 && w < 4 * NF + 2) return 64 * NF + 8 * g + 4 * (w - 4 * NF);
    return 64 * NF + (R32 ? 32 : 0) + 4 * g;
  }
};

// Positions of a call's sequence b: `len` before the drafted tokens, npos in all.
struct Span {
  int b, len, npos;
};
__device__ __forceinline__ Span span_of(const AttnProb& p, int b) {
  const int cap = p.width << p.c.pshift, len = min(p.lengths[b], cap);  // (cap is at most 2^29)
  return Span{b, len, len < 0 ? 0 : min(len + p.tokens, cap)};
}
// A workgroup's share of the work: the positions of sequence b, key head h, are
// cut into `shares` runs of tiles of nearly the same number, this is run
// `split`.  first: number of the sequence's first share of head 0 in the
// workspace, which holds those of sequences with more than one.
struct Share {
  int b, h, split, shares, first;
  // of its row rr, of R: the shares of a row lie side by side
  __device__ __forceinline__ long long place(int rr, int R) const {
    return ((long long)first + (long long)h * shares) * R + (long long)rr * shares + split;
  }
};
// Sums over the lanes up to each one; the last lane's.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // from one lane below, in rows of 16
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);  // two
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);  // four
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);  // eight
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // the last lane of the row below
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // the last lane of the lower half
  return v;
}
__device__ __forceinline__ int wave_sum(int v) { return __builtin_amdgcn_readlane(wave_scan(v), 63); }
// Quotient rounded up, of numbers under 2^24.
__device__ __forceinline__ int ceil_div(int a, int b) {
  int q = (int)((float)a * __builtin_amdgcn_rcpf((float)b));
  q -= q * b >= a ? 1 : 0;  // the product may be off by one either way
  q += q * b < a ? 1 : 0;
  q += q * b < a ? 1 : 0;
  return q;
}
// Workgroups go to sequences by their lengths, which only the device knows:
// the fewest tiles for each, at least LEAST, such that no more of them (p.fit for
// a key head and row block) are made than run at once.  The longest
// share is what a call takes: eight trees over 0 to 4093 positions 43 us, 47
// with equally many shares for each sequence.  The whole wave takes part.  Every
// workgroup reads all lengths, 64 at a time and up to eight times, which grows with
// the square of the sequences: calls of 32, 128, 256, 512 and 1024 sequences without
// positions (8 heads, one token) take 5, 13, 29, 79 and 246 us.
template <int TP, int LEAST>
__device__ __forceinline__ bool find_share(const AttnProb& p, int unit, Share& o) {
  static_assert(LEAST * TP >= 256, "the host's bounds count shares of 256 positions or more");
  const int lane = threadIdx.x & 63, H = p.c.heads, fit = p.fit;
  auto tiles = [&](int b) { return b < p.seqs ? (span_of(p, b).npos + TP - 1) / TP : 0; };
  if (p.seqs == 1) {
    const int t = tiles(0);
    o.b = o.first = 0;
    o.shares = max(ceil_div(t, max(LEAST, ceil_div(t, fit))), 1);
    o.h = unit / o.shares;
    o.split = unit % o.shares;
    return o.h < H;
  }
  const int mine = tiles(lane);
  auto tiles_at = [&](int b) { return b == 0 ? mine : tiles(b + lane); };
  float total = 0.f;
  for (int b = 0; b < p.seqs; b += 64) total += (float)wave_sum(tiles_at(b));
  // (a sequence rounds its shares up, so that some more than total / fit are needed)
  int lo = max(LEAST, (int)min(total * __builtin_amdgcn_rcpf((float)fit), 16777215.f) + 1), hi = 2 * lo;
  for (int k = 0; k < 6 && lo < hi; ++k) {
    const int mid = (lo + hi) >> 1;
    int n = 0;
    for (int b = 0; b < p.seqs; b += 64)
      n += wave_sum(b + lane < p.seqs ? max(ceil_div(tiles_at(b), mid), 1) : 0);
    if (n <= fit)
      hi = mid;
    else
      lo = mid + 1;
  }
  const int per = hi;
  int run = 0, kept = 0;  // shares before; of those, in the workspace
  for (int b = 0; b < p.seqs; b += 64) {
    const int sh = b + lane < p.seqs ? max(ceil_div(tiles_at(b), per), 1) : 0;
    const int in = wave_scan(sh), in2 = wave_scan(sh > 1 ? sh : 0);
    const long long first = (long long)H * (run + in - sh), last = (long long)H * (run + in);
    const uint64_t hit = __ballot(unit >= first && unit < last);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      o.b = b + at;
      o.shares = __builtin_amdgcn_readlane(sh, at);
      const int local = unit - H * (run + __builtin_amdgcn_readlane(in, at) - o.shares);
      o.h = local / o.shares;
      o.split = local % o.shares;
      o.first = H * (kept + __builtin_amdgcn_readlane(in2, at) - (o.shares > 1 ? o.shares : 0));
      return true;
    }
    run += __builtin_amdgcn_readlane(in, 63);
    kept += __builtin_amdgcn_readlane(in2, 63);
  }
  return false;
}

// Which of the positions j0 .. j0 + CH - 1 drafted token t sees.
template <int CH>
__device__ __forceinline__ uint32_t seen(const AttnProb& p, const Span& a, int j0, int t) {
  const int below = min(max(a.len - j0, 0), CH);
  uint32_t bits;
  if (p.mask) {
    bits = 0;
    const int i0 = max(j0 - a.len, 0), wd = i0 >> 5;
    const uint32_t* m = p.mask + ((size_t)a.b * p.tokens + t) * p.words;
    if (below < CH) {
      const uint64_t lo = wd < p.words ? m[wd] : 0u, hi = wd + 1 < p.words ? m[wd + 1] : 0u;
      bits = (uint32_t)((hi << 32 | lo) >> (i0 & 31));
    }
    bits = bits << below | ((1u << below) - 1u);
  } else {
    bits = (1u << min(max(a.len + t + 1 - j0, 0), CH)) - 1u;
  }
  return bits & ((1u << min(max(a.npos - j0, 0), CH)) - 1u);
}

// Query row rr of (sequence b, key head h) as operands for NK steps of 32
// dimensions, and the factor that turns its scores, times their positions'
// scales, into powers of two.  off(ks, j): dimension of the j-th four values of
// step ks (8 bits), off(ks, 0) of its eight (4 bits).
template <int NK, int BITS, class Off>
__device__ __forceinline__ float query_row(const AttnProb& p, int b, int h, int rr, Off off, u32x4* out) {
  const int R = p.tokens * p.group, rc = min(rr, R - 1);
  const uint16_t* q = p.q + b * p.qb + (rc / p.group) * p.qt + (h * p.group + rc % p.group) * p.qh;
  float v[NK][8];
  float mx = 0.f;
#pragma unroll
  for (int ks = 0; ks < NK; ++ks) {
    uint32_t u[4];
    if constexpr (BITS == 8) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const u32x2 a = *glb((const u32x2*)(q + off(ks, j)));
        u[2 * j] = a[0];
        u[2 * j + 1] = a[1];
      }
    } else {
      const u32x4 a = *glb((const u32x4*)(q + off(ks, 0)));
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = a[j];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // 4 bits: elements 0, 4, 1, 5, 2, 6, 3, 7 of the eight
      const int i = BITS == 8 ? e : (e >> 1) + 4 * (e & 1);
      const float f = __uint_as_float(i & 1 ? u[i >> 1] & 0xFFFF0000u : u[i >> 1] << 16);
      v[ks][e] = rr < R ? f : 0.f;
      mx = fmaxf(mx, fabsf(v[ks][e]));
    }
  }
  mx = max_groups(mx);
  const int ex = (int)(__float_as_uint(mx) >> 23);
  // 2^up mx in [2^14, 2^15), or less where the factor would fall under 2^-118: a
  // position that is not seen has the score NONE, and NONE times the factor (-2^10)
  // has to lie far below every other score
  const int es = (int)(__float_as_uint(fabsf(p.scale)) >> 23) - 127;
  const int up = ex == 0 || ex == 255 ? 0 : min(141 - ex, min(100, 118 + es));
  float f = __uint_as_float((uint32_t)(127 + up) << 23);
  if (p.scale < 0.f) f = -f;
  if (p.scale == 0.f) f = 0.f;
#pragma unroll
  for (int ks = 0; ks < NK; ++ks) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // 4 bits: the odd codes of a word arrive times 16
      const float fj = BITS == 4 && (j & 1) ? f * 0.0625f : f;
      out[ks][j] = pack16(v[ks][2 * j] * fj, v[ks][2 * j + 1] * fj);
    }
  }
  // (less only for a scale of 0, or for one under 2^-118 with queries under 2^-126)
  return fmaxf(fabsf(p.scale) * __uint_as_float((uint32_t)(127 - up) << 23), 0x1p-118f);
}

// Eight key codes as an operand, less their zero point: zl = 1024 + z twice, zh
// = 1024 + 16 z twice.
template <int BITS>
__device__ __forceinline__ u32x4 key_operand(uint32_t w0, uint32_t w1, uint32_t zl, uint32_t zh) {
  if constexpr (BITS == 8)
    return u32x4{sub16(bytes2(w0, 0), zl), sub16(bytes2(w0, 1), zl), sub16(bytes2(w1, 0), zl), sub16(bytes2(w1, 1), zl)};
  const uint32_t w8 = w0 >> 8;
  return u32x4{sub16(nib_lo(w0), zl), sub16(nib_hi(w0), zh), sub16(nib_lo(w8), zl), sub16(nib_hi(w8), zh)};
}
// The value codes of eight positions (two words) as operands, less their zero
// points z0, z1: at 8 bits lo, at 4 bits lo and (times 16) hi.
template <int BITS>
__device__ __forceinline__ void value_operand(const uint32_t* w, const uint32_t* z, u32x4& lo, u32x4& hi) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if constexpr (BITS == 8) {
      lo[2 * j] = diff_bf16(bytes2(w[j], 0), bytes2(z[j], 0));
      lo[2 * j + 1] = diff_bf16(bytes2(w[j], 1), bytes2(z[j], 1));
    } else {
      lo[2 * j] = diff_bf16(nib_lo(w[j]), nib_lo(z[j]));
      lo[2 * j + 1] = diff_bf16(nib_lo(w[j] >> 8), nib_lo(z[j] >> 8));
      hi[2 * j] = diff_bf16(nib_hi(w[j]), nib_hi(z[j] << 4));
      hi[2 * j + 1] = diff_bf16(nib_hi(w[j] >> 8), nib_hi(z[j] >> 4));
    }
  }
}

// The rows of a wave: running reference M (NONE: nothing seen), sum l, factor
// cq, and the unnormalised result.
template <int NB, int NO>
struct Rows {
  f32x4 acc[NB][NO];
  float M[NB], l[NB], cq[NB];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      M[nb] = NONE;
      l[nb] = 0.f;
#pragma unroll
      for (int i = 0; i < NO; ++i) acc[nb][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
};

// Scores S of a lane's CH positions (before their scales ks) to weights P times
// the scales vs, for row block nb: [leading, next][step].
template <int BITS, int CH, int NB, int NO>
__device__ __forceinline__ void weigh(Rows<NB, NO>& r, int nb, const f32x4* S, const f32x4* ks, const f32x4* vs,
                                      bool masked, uint32_t see, u32x4 (*P)[CH / 8]) {
  float xs[CH], mx = NONE;
#pragma unroll
  for (int i = 0; i < CH; ++i) xs[i] = S[i >> 2][i & 3] * ks[i >> 2][i & 3];
  if (masked) {
#pragma unroll
    for (int i = 0; i < CH; ++i) xs[i] = (see >> i) & 1u ? xs[i] : NONE;
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) mx = fmaxf(mx, xs[i]);
  // M moves only when a score passes it by 2^8 (its weight): most tiles then
  // need neither the maximum over the lanes nor a pass over the sums.
  if (__any((mx - r.M[nb]) * r.cq[nb] > 8.f)) {
    const float Mn = fmaxf(r.M[nb], max_groups(mx));
    const float al = Mn > r.M[nb] ? __builtin_amdgcn_exp2f((r.M[nb] - Mn) * r.cq[nb]) : 1.f;
    r.l[nb] *= al;
#pragma unroll
    for (int i = 0; i < NO; ++i) r.acc[nb][i] *= al;
    r.M[nb] = Mn;
  }
  // (nothing seen yet: NONE cq is far below every score's product with cq, and its weights are 0)
  const float ref = r.M[nb] == NONE ? 0.f : r.M[nb] * r.cq[nb];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(xs[i], r.cq[nb], -ref));
    r.l[nb] += e;
    xs[i] = e * vs[i >> 2][i & 3];
  }
  if (masked) {
#pragma unroll
    for (int i = 0; i < CH; ++i) xs[i] = (see >> i) & 1u ? xs[i] : 0.f;
  }
#pragma unroll
  for (int s = 0; s < CH / 8; ++s) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // 4 bits: positions (0, 2), (1, 3) of every four, as their bytes come apart
      const float a = xs[8 * s + (BITS == 8 ? 2 * j : 4 * (j >> 1) + (j & 1))];
      const float b = xs[8 * s + (BITS == 8 ? 2 * j + 1 : 4 * (j >> 1) + (j & 1) + 2)];
      uint32_t lead, next;
      split16(a, b, lead, next);
      P[0][s][j] = lead;
      P[1][s][j] = next;
    }
  }
  __builtin_amdgcn_sched_barrier(0);
}

// End of a wave's positions: sums over the four lanes of a row, M in powers of
// two (-INFINITY: nothing seen), 4 bits: the upper half's codes came times 16.
template <int BITS, int NB, int NO>
__device__ __forceinline__ void settle(Rows<NB, NO>& r) {
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    r.l[nb] = sum_groups(r.l[nb]);
    r.M[nb] = r.M[nb] == NONE ? -INFINITY : r.M[nb] * r.cq[nb];
    if constexpr (BITS == 4) {
#pragma unroll
      for (int i = NO / 2; i < NO; ++i) r.acc[nb][i] *= 0.0625f;
    }
  }
}

// Rows that another workgroup of the same launch reads, perhaps on another
// XCD: stored through and loaded past the L2 (agent-scope accesses), so that no
// cache has to be written back or emptied for them.  (A fence pair, which does
// that, took 90 us of a 180 us call.)
__device__ __forceinline__ void put_shared(float* p, float a, float b) {
  const uint64_t v = (uint64_t)__float_as_uint(b) << 32 | __float_as_uint(a);
  __hip_atomic_store((uint64_t*)p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <bool SHARED>
__device__ __forceinline__ f32x2 get2(const float* p) {
  if (!SHARED) return *(const f32x2*)p;
  const uint64_t v = __hip_atomic_load((const uint64_t*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return f32x2{__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32))};
}

// Joins the shares of row rr of sequence me.b, key head me.h, dimensions d .. d
// + 3: sum of exp2(M_s - max M) (O_s, l_s).  G threads take every G-th share
// each (k says which) and are added in order; !on: takes part only.
template <int G>
struct JoinLds {
  f32x4 o[G > 1 ? 256 : 1];
  float l[G > 1 ? 256 : 1];
};
template <int G, bool SHARED>
__device__ __forceinline__ void join_row(const AttnProb& p, bool on, Share me, int rr, int d, int k, JoinLds<G>* s) {
  const int dim = p.c.dim, R = p.tokens * p.group;
  f32x4 a = {0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
  if (on) {
    me.split = 0;
    const long long row = me.place(rr, R);
    const float* ml = p.ml + 2 * row;
    float mx = -INFINITY;
#pragma unroll 8
    for (int e = 0; e < me.shares; ++e) mx = fmaxf(mx, get2<SHARED>(ml + 2 * e)[0]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float* part = p.part + row * dim + d;
#pragma unroll 4
    for (int e = k; e < me.shares; e += G) {
      const f32x2 o0 = get2<SHARED>(part + (size_t)e * dim), o1 = get2<SHARED>(part + (size_t)e * dim + 2);
      const f32x2 m = get2<SHARED>(ml + 2 * e);
      const float f = __builtin_amdgcn_exp2f(m[0] - ref);
      l += f * m[1];
      a += f * f32x4{o0[0], o0[1], o1[0], o1[1]};
    }
  }
  if constexpr (G > 1) {
    s->o[threadIdx.x] = a;
    s->l[threadIdx.x] = l;
    __syncthreads();
    if (k != 0) return;
    for (int e = 1; e < G; ++e) {
      a += s->o[threadIdx.x + e * (dim >> 2)];
      l += s->l[threadIdx.x + e * (dim >> 2)];
    }
  }
  if (!on) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *(bf16x4*)(p.o + me.b * p.ob + (rr / p.group) * p.ot + (me.h * p.group + rr % p.group) * p.oh + d) =
      __builtin_convertvector(a * inv, bf16x4);
}

// The rows of a share from row0 on: the result (one share), or the unnormalised
// rows to the workspace.
template <int NB, int NO>
__device__ __forceinline__ void put_rows(const AttnProb& p, const Rows<NB, NO>& r, const Share& me, int row0) {
  const int b = me.b, h = me.h;
  const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15, R = p.tokens * p.group;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int rr = row0 + 16 * nb + n;
    if (rr >= R) continue;
    if (me.shares == 1) {
      const float inv = r.l[nb] == 0.f ? 0.f : 1.f / r.l[nb];
      uint16_t* o = p.o + b * p.ob + (rr / p.group) * p.ot + (h * p.group + rr % p.group) * p.oh;
#pragma unroll
      for (int i = 0; i < NO; ++i) *(bf16x4*)(o + 16 * i + 4 * g) = __builtin_convertvector(r.acc[nb][i] * inv, bf16x4);
    } else {
      const size_t row = (size_t)me.place(rr, R);
#pragma unroll
      for (int i = 0; i < NO; ++i) {
        float* o = p.part + row * (16 * NO) + 16 * i + 4 * g;
        if (p.count) {
          put_shared(o, r.acc[nb][i][0], r.acc[nb][i][1]);
          put_shared(o + 2, r.acc[nb][i][2], r.acc[nb][i][3]);
        } else {
          *(f32x4*)o = r.acc[nb][i];
        }
      }
      if (g == 0) put_shared(p.ml + 2 * row, r.M[nb], r.l[nb]);
    }
  }
}

}  // namespace

// Softmax attention in one pass over the cache with a running reference near the
// maximum and a running sum.
//
// A wave takes 16 NB query rows (token, head of the group) of one sequence and
// key head, and TP = 64 or 32 positions at a time, and works with both products
// transposed, so that nothing moves between lanes:
//   S^T = K Q^T: 16 positions x 16 rows per MFMA, the key rows ordered so that
//     the lane (g = lane / 16, n = lane % 16) receives row n's scores at
//     chunk g of the tile (TP/4 consecutive positions), four for each MFMA;
//   O^T = V^T P^T: the same lane's weights of those positions are its part of
//     the P^T operand as they are, and the V^T operand is as many consecutive
//     bytes of a dimension's row, which is why values lie dimension by
//     dimension in a page.  Every register of the sum belongs to row n.
// Codes enter as c - z: 1024 + c is made with one byte permutation or mask for
// two codes, and 1024 + z taken from it; float16 in the first product, bfloat16
// in the second, both exact, as all products are in float32.  Scores times
// their position's scale are then relative to the row's factor cq.
// Queries are scaled by a power of two per row to just below 2^15 (exact for
// elements within 2^-29 of the largest) and exact in float16 (bf16 has 8 bits);
// they wait in LDS in operand order.
//
// Weights enter the second product times their position's scale, as two
// bfloat16 numbers, the nearest to it and the nearest to what is left, within 2^-16
// of it and without a bias: with one of them the weights' rounding would be as
// large as the result's, and float16's range would lose the weights under 2^-29 of
// the largest, which are all there is where the others' values are zero.
//
// In a tile that reaches past the context or a page outside the pool,
// invisible positions are taken out of scores and weights by selection,
// whatever their scales hold.
//
// The WV waves of a workgroup take every WV-th tile of its share of the
// positions and are joined in LDS in a fixed order; of several shares
// the unnormalised rows go to the workspace.  The shares of a row are
// joined, in their order, by the workgroup that comes last (p.count, which it
// sets back to 0), or where they are many by k_attn_join.
//
// Up to 16 rows it is bound by reading the codes: 32 contexts of 4096 to 8192
// tokens, 8 heads of 128 at 8 bits, 423 MB in 85 us, 5.0 TB/s, what a large copy
// moves (at 4 bits 220 MB in 65 us, vector instructions issued 55% of the time, 38%
// at 8: unpacking does not halve); 64 positions a tile, so that 17 KB a wave are on
// their way.  With more rows by its vector instructions, about ten for a score and
// two for a code: 40 rows of 131071 positions, 4 heads at 4 bits, 39 us, issued 56%
// of the time; 32 positions a tile, so that two waves fit a SIMD without spills.
template <int DIM, int BITS, int NB, int TP, int WV, int OCC>
__global__ __launch_bounds__(64 * WV, OCC) void k_tree_attn(const AttnProb p) {
  typedef Tile<DIM, BITS, TP> T;
  typedef typename T::Chunk Chunk;
  constexpr int CH = T::CH, NI = T::NI, NS = T::NS;
  constexpr int NK = DIM / 32, NO = DIM / 16, NMB = T::NMB;
  constexpr bool ONCE = NB == 1;  // up to 16 rows: one block, so that the codes are read once
  __shared__ float sm[WV][16 * NB], sl[WV][16 * NB], scq[16 * NB];
  __shared__ union {
    u32x4 q[NB][NK][64];
    f32x4 o[WV / 2][NB * NO][64];
  } sh;
  const KvPool& c = p.c;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Blocks of one (sequence, key head, share) are eight apart: on one XCD,
  // whose L2 then holds the share's codes for all of them.
  const int x = blockIdx.x / (8 * p.nrb), rem = blockIdx.x % (8 * p.nrb);
  const int rb = rem >> 3, unit = 8 * x + (rem & 7);
  Share me;
  if (!find_share<TP, (WV * TP > 256 ? WV : 256 / TP)>(p, unit, me)) return;
  const int b = __builtin_amdgcn_readfirstlane(me.b), h = __builtin_amdgcn_readfirstlane(me.h);
  const int split = __builtin_amdgcn_readfirstlane(me.split), shares = __builtin_amdgcn_readfirstlane(me.shares);
  if (h == 0 && split == 0 && rb == 0 && tid == 0) {  // for the join
    p.info[2 * b] = me.first;
    p.info[2 * b + 1] = shares;
  }
  const int R = p.tokens * p.group;

  const Span sp = span_of(p, b);
  const int npos = sp.npos;
  const int ntile = (npos + TP - 1) / TP;
  const int per = (ntile + shares - 1) / shares;
  const int t1 = min(ntile, (split + 1) * per);
  int tile = split * per + w;

  const int pm = (1 << c.pshift) - 1, lastchunk = max(npos - 1, 0) / CH;
  const int* table = p.tables + (size_t)b * p.width;
  // A tile that lies in one page (pages of TP positions or more) is found by one
  // scalar load, and its addresses are scalar but for a constant of the lane;
  // otherwise every lane looks up the pages of the two chunks that it reads, of
  // its key rows and of its scores and values (the last chunk there is for those
  // past the end).
  const bool one = (1 << c.pshift) >= TP;
  struct Place {
    int k, v, ok, ov;
    bool bad;
  };
  auto inside = [&](int pg) { return (unsigned)pg < (unsigned)c.pages; };
  auto find = [&](int tl) {
    Place q;
    if (one) {
      const int at = min(tl * TP, max(npos - 1, 0)), pg = scalar_load(table + (at >> c.pshift));
      q.bad = !inside(pg);
      q.k = q.v = q.bad ? 0 : pg;
      q.ok = q.ov = tl * TP & pm;
    } else {
      const int ck = min(4 * tl + (n >> 2), lastchunk) * CH, cv = min(4 * tl + g, lastchunk) * CH;
      const int pk = glb(table)[ck >> c.pshift], pv = glb(table)[cv >> c.pshift];
      q.bad = !inside(pv);
      q.k = inside(pk) ? pk : 0;
      q.v = q.bad ? 0 : pv;
      q.ok = ck & pm;
      q.ov = cv & pm;
    }
    return q;
  };
  // slot of the chunk's first position, counted over all heads: of the tile (one
  // page; uniform) and the lane's chunk in it, or of the lane's chunk
  auto slot = [&](int pg, int off, int chunk, size_t& base) {
    base = (((size_t)pg * c.heads + h) << c.pshift) + off;
    if (one) base = uniform(base);
    return one ? CH * chunk : 0;
  };
  auto load_k = [&](T& t, const Place& q) {
    size_t at;
    const int in = slot(q.k, q.ok, n >> 2, at);
    const uint8_t* kr = c.kc + at * T::RB + (in + (n & 3)) * T::RB;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint8_t* r = kr + 4 * i * T::RB;
#pragma unroll
      for (int s = 0; s < T::NF; ++s) {
        const u32x4 u = fetch<ONCE>((const u32x4*)(r + 64 * s + 16 * g));
#pragma unroll
        for (int e = 0; e < 4; ++e) t.k[i][4 * s + e] = u[e];
      }
      if constexpr (T::R32) {
        const u32x2 u = fetch<ONCE>((const u32x2*)(r + 64 * T::NF + 8 * g));
        t.k[i][4 * T::NF] = u[0];
        t.k[i][4 * T::NF + 1] = u[1];
      }
      if constexpr (T::R16) t.k[i][T::NW - 1] = *glb((const uint32_t*)(r + T::RB - 16 + 4 * g));
    }
    t.kz = *glb((const Chunk*)(c.kz + at + in));
  };
  auto load_g = [&](T& t, const Place& q) {
    t.bad = q.bad;
    size_t at;
    const int in = slot(q.v, q.ov, g, at);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      t.ks[i] = *glb((const f32x4*)(c.ks + at + in + 4 * i));
      t.vs[i] = *glb((const f32x4*)(c.vs + at + in + 4 * i));
    }
    t.vz = *glb((const Chunk*)(c.vz + at + in));
  };
  auto load_v = [&](T& t, const Place& q) {
    const size_t blk = (((size_t)q.v * c.heads + h) * T::RB << c.pshift) + q.ov;
    const uint8_t* vr = c.vc + (one ? uniform(blk) : blk) + (n << c.pshift) + (one ? CH * g : 0);
#pragma unroll
    for (int i = 0; i < NMB; ++i) t.v[i] = fetch<ONCE>((const Chunk*)(vr + ((size_t)(16 * i) << c.pshift)));
  };

  const bool work = tile < t1;
  T t;
  Place at{};
  if (work) {
    at = find(tile);
    load_k(t, at);
    load_g(t, at);
    load_v(t, at);
  }

  // queries: row n of block nb, in the order of the key codes' words
#pragma unroll 1
  for (int nb = w; nb < NB; nb += WV) {
    u32x4 q[NK];
    const float f = query_row<NK, BITS>(
        p, b, h, 16 * (NB * rb + nb) + n,
        [&](int ks, int j) { return BITS == 8 ? T::off(2 * ks + j, g) : 2 * T::off(ks, g); }, q);
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) sh.q[nb][ks][lane] = q[ks];
    if (g == 0) scq[16 * nb + n] = f;
  }
  __syncthreads();

  Rows<NB, NO> r;
  r.clear();
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) r.cq[nb] = scq[16 * nb + n];

  f32x4 S[NB][NI];
  u32x4 P[NB][2][NS];  // [leading, next][step]
  auto scores = [&](const T& t) {
    uint32_t zl[NI], zh[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint32_t z = (t.kz[i] >> (8 * (n & 3))) & 255u;
      zl[i] = z * 0x00010001u + 0x64006400u;
      zh[i] = z * 0x00100010u + 0x64006400u;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) S[nb][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
      u32x4 q[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) q[nb] = sh.q[nb][ks][lane];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const u32x4 a = BITS == 8 ? key_operand<BITS>(t.k[i][2 * ks % T::NW], t.k[i][(2 * ks + 1) % T::NW], zl[i], zh[i])
                                  : key_operand<BITS>(t.k[i][ks], 0, zl[i], zh[i]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) S[nb][i] = mfma(a, q[nb], S[nb][i]);
      }
    }
  };
  auto weights = [&](const T& t, int tl) {
    const bool masked = TP * (tl + 1) > min(sp.len, npos) || __any(t.bad);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      uint32_t see = 0;
      if (masked && !t.bad)
        see = seen<CH>(p, sp, TP * tl + CH * g, min(16 * (NB * rb + nb) + n, R - 1) / p.group);
      weigh<BITS, CH>(r, nb, S[nb], t.ks, t.vs, masked, see, P[nb]);
    }
  };
  // vector instructions a product: what unpacking takes, over the products
  constexpr int VPM = NB == 1 ? 8 : NB == 2 ? 4 : 3;
  auto values = [&](const T& t, const uint32_t* vz) {
#pragma unroll
    for (int i = 0; i < NMB; ++i) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        u32x4 a, e;
        const uint32_t v[2] = {t.v[i][2 * s], t.v[i][2 * s + 1]};
        value_operand<BITS>(v, vz + 2 * s, a, e);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            r.acc[nb][i] = mfma_bf(a, P[nb][k][s], r.acc[nb][i]);
            if constexpr (BITS == 4) r.acc[nb][i + NMB] = mfma_bf(e, P[nb][k][s], r.acc[nb][i + NMB]);
          }
        }
      }
    }
    // the next codes are unpacked between the products: a product keeps its
    // unit busy for four further instructions' time
#pragma unroll
    for (int i = 0; i < 2 * NB * NO * NS; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x002, VPM, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
  };

  // A part of the next tile is asked for as soon as this tile's has been used.
  if (work) {
    at = find(tile + WV);
    while (true) {
      const bool more = tile + WV < t1;
      scores(t);
      __builtin_amdgcn_sched_barrier(0);
      if (more) load_k(t, at);
      __builtin_amdgcn_sched_barrier(0);
      weights(t, tile);
      uint32_t vz[NI];
#pragma unroll
      for (int i = 0; i < NI; ++i) vz[i] = t.vz[i];
      __builtin_amdgcn_sched_barrier(0);
      if (more) load_g(t, at);
      __builtin_amdgcn_sched_barrier(0);
      values(t, vz);
      __builtin_amdgcn_sched_barrier(0);
      if (!more) break;
      load_v(t, at);
      tile += WV;
      at = find(tile + WV);
    }
  }

  settle<BITS>(r);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    if (g == 0) {
      sm[w][16 * nb + n] = r.M[nb];
      sl[w][16 * nb + n] = r.l[nb];
    }
  }
  __syncthreads();
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    float mx = -INFINITY, s = 0.f;
#pragma unroll
    for (int k = 0; k < WV; ++k) mx = fmaxf(mx, sm[k][16 * nb + n]);
    const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
    for (int k = 0; k < WV; ++k) s += sl[k][16 * nb + n] * __builtin_amdgcn_exp2f(sm[k][16 * nb + n] - ref);
    const float f = __builtin_amdgcn_exp2f(r.M[nb] - ref);
#pragma unroll
    for (int i = 0; i < NO; ++i) r.acc[nb][i] *= f;
    r.M[nb] = mx;
    r.l[nb] = s;
  }
  auto put = [&](int k) {
#pragma unroll
    for (int i = 0; i < NB * NO; ++i) sh.o[k][i][lane] = r.acc[i / NO][i % NO];
  };
  auto add = [&](int k) {
#pragma unroll
    for (int i = 0; i < NB * NO; ++i) r.acc[i / NO][i % NO] += sh.o[k][i][lane];
  };
#pragma unroll
  for (int half = WV / 2; half > 0; half /= 2) {
    if (w >= half && w < 2 * half) put(w - half);
    __syncthreads();
    if (w < half) add(w);
    __syncthreads();
  }
  if (w == 0) put_rows(p, r, me, 16 * NB * rb);
  if (!p.count || shares == 1) return;
  __shared__ int last;
  if (w == 0) {
    // this wave wrote the rows: they are in memory before the count says so
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (lane == 0) {
      int* ct = p.count + ((size_t)b * c.heads + h) * p.nrb + rb;
      last = __hip_atomic_fetch_add(ct, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == shares - 1;
      if (last) __hip_atomic_store(ct, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  __syncthreads();
  if (!last) return;
  const int r1 = min(16 * NB, R - 16 * NB * rb);
  for (int i = tid; i < r1 * (DIM / 4); i += 64 * WV)
    join_row<1, true>(p, true, me, 16 * NB * rb + i / (DIM / 4), 4 * (i % (DIM / 4)), 0, nullptr);
}

// The same attention for many rows: the four waves of a workgroup take 16 NB
// rows each and the same positions, so that codes are read and unpacked once
// for 64 NB rows.  Each wave unpacks its part of the next tile into LDS, as the
// operands are read (a lane's 16 bytes side by side), while the current one is
// used from the other half; one barrier a tile.  Nothing has to be joined in
// the workgroup.  The operand layout is that of k_tree_attn with dimension 32
// ks + 8 g + e in step ks.  Bound by vector instructions (issued 50% of the
// time) and the waits between them: 108 rows of 0 to 4093 positions, 64 heads of
// 128 in all at 4 bits, 38 us; 9.9 GFLOP.
template <int DIM, int BITS, int NB, int TP>
__global__ __launch_bounds__(256, 2) void k_tree_attn_wide(const AttnProb p) {
  typedef Tile<DIM, BITS, TP> T;
  typedef typename T::Chunk Chunk;
  constexpr int CH = T::CH, NI = T::NI, NS = T::NS, NMB = T::NMB;
  constexpr int NK = DIM / 32, NO = DIM / 16;
  constexpr int KS = NK * NI / 4;          // steps of a key block that a wave unpacks
  constexpr int VM = (NMB + 3) / 4;        // blocks of value rows that a wave unpacks, at most
  constexpr int KW = BITS == 8 ? 2 : 1;    // words of a lane per step
  struct Half {
    u32x4 k[NI][NK][64];
    u32x4 v[NO][NS][64];
    float sc[2][TP];
    int bad[4];
  };
  __shared__ Half lds[2];
  const KvPool& c = p.c;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int x = blockIdx.x / (8 * p.nrb), rem = blockIdx.x % (8 * p.nrb);
  const int rb = rem >> 3, unit = 8 * x + (rem & 7);
  Share me;
  if (!find_share<TP, 256 / TP>(p, unit, me)) return;
  const int b = __builtin_amdgcn_readfirstlane(me.b), h = __builtin_amdgcn_readfirstlane(me.h);
  const int split = __builtin_amdgcn_readfirstlane(me.split), shares = __builtin_amdgcn_readfirstlane(me.shares);
  if (h == 0 && split == 0 && rb == 0 && tid == 0) {  // for the join
    p.info[2 * b] = me.first;
    p.info[2 * b + 1] = shares;
  }
  const int R = p.tokens * p.group, row0 = 16 * NB * (4 * rb + w);

  const Span sp = span_of(p, b);
  const int npos = sp.npos;
  const int ntile = (npos + TP - 1) / TP;
  const int per = (ntile + shares - 1) / shares;
  const int t0 = split * per, t1 = min(ntile, t0 + per);
  const int pm = (1 << c.pshift) - 1, lastchunk = max(npos - 1, 0) / CH;
  const int* table = p.tables + (size_t)b * p.width;

  // What a wave brings of a tile: its steps of key block ki, its blocks of value
  // rows, and (waves 0 and 1) the scales of the keys and of the values.
  const int ki = w % NI, k0 = w / NI * KS;
  struct Raw {
    uint32_t k[KS][KW];
    Chunk v[VM];
    Chunk vz;
    uint32_t kz;
    float sc;
    bool bad;
  };
  struct Pages {
    int k, v, s;
  };
  auto chunk_of = [&](int chunk) { return min(chunk, lastchunk) * CH; };
  // page numbers are asked for a tile before the codes, ahead of the codes of the tile between
  auto find = [&](int tl) {
    Pages q;
    q.k = glb(table)[chunk_of(4 * tl + (n >> 2)) >> c.pshift];
    q.v = glb(table)[chunk_of(4 * tl + g) >> c.pshift];
    q.s = glb(table)[chunk_of(4 * tl + min(lane / CH, 3)) >> c.pshift];
    return q;
  };
  auto inside = [&](int pg) { return (unsigned)pg < (unsigned)c.pages; };
  auto load = [&](Raw& t, int tl, const Pages& q) {
    const size_t pk = (size_t)(inside(q.k) ? q.k : 0) * c.heads + h, pv = (size_t)(inside(q.v) ? q.v : 0) * c.heads + h;
    const size_t ps = (size_t)(inside(q.s) ? q.s : 0) * c.heads + h;
    const size_t at = (pk << c.pshift) + (chunk_of(4 * tl + (n >> 2)) & pm) + 4 * ki + (n & 3);
    typedef uint32_t KeyWords __attribute__((ext_vector_type(KW)));
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const KeyWords u = *glb((const KeyWords*)(c.kc + at * T::RB + 4 * KW * (4 * (k0 + ks) + g)));
#pragma unroll
      for (int e = 0; e < KW; ++e) t.k[ks][e] = u[e];
    }
    t.kz = *glb(c.kz + at);
    const int ov = chunk_of(4 * tl + g) & pm;
    const uint8_t* vr = c.vc + ((pv * T::RB + n) << c.pshift) + ov;
#pragma unroll
    for (int j = 0; j < VM; ++j)
      t.v[j] = *glb((const Chunk*)(vr + ((size_t)(16 * min(w + 4 * j, NMB - 1)) << c.pshift)));
    t.vz = *glb((const Chunk*)(c.vz + (pv << c.pshift) + ov));
    t.bad = !inside(q.s);
    if (w < 2)
      t.sc = *glb((w ? c.vs : c.ks) + (ps << c.pshift) + (chunk_of(4 * tl + min(lane / CH, 3)) & pm) + lane % CH);
  };
  auto unpack = [&](const Raw& t, Half& o) {
    const uint32_t zl = t.kz * 0x00010001u + 0x64006400u, zh = t.kz * 0x00100010u + 0x64006400u;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) o.k[ki][k0 + ks][lane] = key_operand<BITS>(t.k[ks][0], t.k[ks][KW - 1], zl, zh);
#pragma unroll
    for (int j = 0; j < VM; ++j) {
      const int mb = w + 4 * j;
      if (NMB % 4 != 0 && mb >= NMB) break;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const uint32_t v[2] = {t.v[j][2 * s], t.v[j][2 * s + 1]}, z[2] = {t.vz[2 * s], t.vz[2 * s + 1]};
        u32x4 lo, hi;
        value_operand<BITS>(v, z, lo, hi);
        o.v[mb][s][lane] = lo;
        if constexpr (BITS == 4) o.v[mb + NMB][s][lane] = hi;
      }
    }
    if (w < 2 && lane < TP) {
      o.sc[w][lane] = t.sc;
      if (w == 1 && lane % CH == 0) o.bad[lane / CH] = t.bad;
    }
  };
  // LDS written by the others can be read after it; loads in flight stay there
  auto meet = [&]() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  };

  u32x4 qf[NB][NK];
  Rows<NB, NO> r;
  r.clear();
  const bool rows = row0 < R;  // (a wave without rows still brings its part)
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    r.cq[nb] = query_row<NK, BITS>(
        p, b, h, row0 + 16 * nb + n, [&](int ks, int j) { return 32 * ks + 8 * g + 4 * j; }, qf[nb]);
    __builtin_amdgcn_sched_barrier(0);
  }

  auto use = [&](const Half& t, int tl) {
    f32x4 S[NB][NI], kv[2][NI];
    u32x4 P[NB][2][NS];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) S[nb][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const u32x4 a = t.k[i][ks][lane];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) S[nb][i] = mfma(a, qf[nb][ks], S[nb][i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      kv[0][i] = *(const f32x4*)&t.sc[0][CH * g + 4 * i];
      kv[1][i] = *(const f32x4*)&t.sc[1][CH * g + 4 * i];
    }
    const bool bad = t.bad[g], masked = TP * (tl + 1) > min(sp.len, npos) || __any(bad);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      uint32_t see = 0;
      if (masked && !bad) see = seen<CH>(p, sp, TP * tl + CH * g, min(row0 + 16 * nb + n, R - 1) / p.group);
      weigh<BITS, CH>(r, nb, S[nb], kv[0], kv[1], masked, see, P[nb]);
    }
#pragma unroll
    for (int i = 0; i < NO; ++i) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const u32x4 a = t.v[i][s][lane];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) r.acc[nb][i] = mfma_bf(a, P[nb][k][s], r.acc[nb][i]);
        }
      }
    }
  };

  if (t0 < t1) {
    Raw t;
    Pages q = find(t0), q1 = find(t0 + 1);
    load(t, t0, q);
    unpack(t, lds[0]);
    if (t0 + 1 < t1) {
      q = find(t0 + 2);
      load(t, t0 + 1, q1);
    }
    meet();
    for (int tl = t0; tl < t1; ++tl) {
      const int half = (tl - t0) & 1;
      if (tl + 1 < t1) {
        unpack(t, lds[half ^ 1]);
        __builtin_amdgcn_sched_barrier(0);
        if (tl + 2 < t1) {
          q1 = find(tl + 3);
          load(t, tl + 2, q);
          q = q1;
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (rows) use(lds[half], tl);
      meet();
    }
  }
  settle<BITS>(r);
  put_rows(p, r, me, row0);
}

// The shares of every row, where a launch of its own joins them: bound by
// reading them (13824 rows of up to 11 shares of 128 dimensions 7.5 us, 7 TB/s
// from the last-level cache) or by its latency (160 rows of 64 shares 5.8 us).
template <int G>
__global__ __launch_bounds__(256) void k_attn_join(const AttnProb p) {
  __shared__ JoinLds<G> s;
  const JoinThread t = join_thread(threadIdx.x, p.c.dim, G);
  const int rows = blockDim.x / (p.c.dim / 4 * G), R = p.tokens * p.group;
  const unsigned row = blockIdx.x * rows + t.i;  // (at most 2^30 of them)
  bool on = row < (unsigned)(p.seqs * p.c.heads * R);
  Share me{};
  if (on) {
    const int bh = (int)(row / R), b = bh / p.c.heads;
    me = Share{b, bh % p.c.heads, 0, p.info[2 * b + 1], p.info[2 * b]};
    on = me.shares > 1;  // a single share has written its result
  }
  join_row<G, false>(p, on, me, (int)(row % R), t.d, t.k, &s);
}

void plan_tree_attn(AttnProb& p, int ncu) {
  const long long hold = (((long long)p.width << p.c.pshift) + 255) / 256;
  (AttnPlan&)p = plan_attention((long long)p.tokens * p.group, p.seqs, p.c.heads, p.c.dim, hold, ncu);
}

namespace {
template <int DIM, int BITS>
void attn_nb(const AttnProb& p, dim3 grid, hipStream_t st) {
  constexpr int TP = DIM <= 128 ? 64 : 32;
  const dim3 block(attention_threads(p, DIM));
  if (p.wide) {
    if (p.nb == 1)
      hipLaunchKernelGGL((k_tree_attn_wide<DIM, BITS, 1, TP>), grid, block, 0, st, p);
    else if constexpr (DIM <= 128)
      hipLaunchKernelGGL((k_tree_attn_wide<DIM, BITS, 2, TP>), grid, block, 0, st, p);
  } else if (p.nb == 1) {
    hipLaunchKernelGGL((k_tree_attn<DIM, BITS, 1, TP, 4, 2>), grid, block, 0, st, p);
  } else if (p.nb == 2) {
    if constexpr (DIM <= 128)
      hipLaunchKernelGGL((k_tree_attn<DIM, BITS, 2, 32, 8, 2>), grid, block, 0, st, p);
    else
      hipLaunchKernelGGL((k_tree_attn<DIM, BITS, 2, 32, 4, 1>), grid, block, 0, st, p);
  } else if constexpr (DIM <= 128) {
    hipLaunchKernelGGL((k_tree_attn<DIM, BITS, 3, 32, 8, 2>), grid, block, 0, st, p);
  }
}
template <int BITS>
hipError_t attn_dim(const AttnProb& p, hipStream_t st) {
  const dim3 grid((unsigned)attention_blocks(p));
  switch (p.c.dim) {
    case 64: attn_nb<64, BITS>(p, grid, st); break;
    case 96: attn_nb<96, BITS>(p, grid, st); break;
    case 128: attn_nb<128, BITS>(p, grid, st); break;
    case 192: attn_nb<192, BITS>(p, grid, st); break;
    default: attn_nb<256, BITS>(p, grid, st); break;
  }
  return hipGetLastError();
}
}  // namespace

hipError_t launch_tree_attn(const AttnProb& p, int bits, hipStream_t st) {
  return bits == 8 ? attn_dim<8>(p, st) : attn_dim<4>(p, st);
}

hipError_t launch_attn_join(const AttnProb& p, hipStream_t st) {
  const JoinPlan j = plan_join(p.c.dim, p.shares);
  const long long n = (long long)p.seqs * p.c.heads * p.tokens * p.group;
  const dim3 grid((unsigned)((n + j.rows - 1) / j.rows)), block(j.threads);
  if (j.G == 8)
    hipLaunchKernelGGL(k_attn_join<8>, grid, block, 0, st, p);
  else if (j.G == 4)
    hipLaunchKernelGGL(k_attn_join<4>, grid, block, 0, st, p);
  else
    hipLaunchKernelGGL(k_attn_join<1>, grid, block, 0, st, p);
  return hipGetLastError();
}
