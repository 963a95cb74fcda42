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
// the leading 16 bits of two floats (their bfloat16 truncations), and those of what the truncation left
__device__ __forceinline__ uint32_t lead16(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ float rest16(float a) { return a - __uint_as_float(__float_as_uint(a) & 0xFFFF0000u); }

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

// Joins the shares of row `row` of (sequence, key head, row), dimensions d .. d
// + 3: sum of exp2(M_s - max M) (O_s, l_s).  G threads take every G-th share
// each (k says which) and are added in order; row < 0: takes part only.
template <int G>
struct JoinLds {
  f32x4 o[G > 1 ? 256 : 1];
  float l[G > 1 ? 256 : 1];
};
template <int G, bool SHARED>
__device__ __forceinline__ void join_row(const AttnProb& p, long long row, int d, int k, JoinLds<G>* s) {
  const int dim = p.c.dim, ns = p.nsplit;
  f32x4 a = {0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
  if (row >= 0) {
    const float* ml = p.ml + 2 * row * ns;
    float mx = -INFINITY;
#pragma unroll 8
    for (int e = 0; e < ns; ++e) mx = fmaxf(mx, get2<SHARED>(ml + 2 * e)[0]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float* part = p.part + row * ns * dim + d;
#pragma unroll 4
    for (int e = k; e < ns; e += G) {
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
  if (row < 0) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int R = p.tokens * p.group, bh = (int)(row / R), rr = (int)(row % R), b = bh / p.c.heads, h = bh % p.c.heads;
  *(bf16x4*)(p.o + b * p.ob + (rr / p.group) * p.ot + (h * p.group + rr % p.group) * p.oh + d) =
      __builtin_convertvector(a * inv, bf16x4);
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
// bfloat16 numbers, the leading 8 bits and the next 8: with one of them the
// weights' rounding would be as large as the result's, and float16's range
// would lose the weights under 2^-29 of the largest, which are all there is
// where the others' values are zero.
//
// In a tile that reaches past the context or a page outside the pool,
// invisible positions are taken out of scores and weights by selection,
// whatever their scales hold.
//
// The four waves of a workgroup take every fourth tile of its share of the
// positions and are joined in LDS in a fixed order; with several shares
// (nsplit) the unnormalised rows go to the workspace.  The shares of a row are
// joined, in their order, by the workgroup that comes last (p.count, which it
// sets back to 0), or where they are many by k_attn_join.
template <int DIM, int BITS, int NB, int TP, int OCC>
__global__ __launch_bounds__(256, OCC) void k_tree_attn(const AttnProb p) {
  typedef Tile<DIM, BITS, TP> T;
  typedef typename T::Chunk Chunk;
  constexpr int CH = T::CH, NI = T::NI, NS = T::NS;
  constexpr int NK = DIM / 32, NO = DIM / 16, NMB = T::NMB;
  constexpr bool ONCE = NB == 1;  // up to 16 rows: one block, so that the codes are read once
  __shared__ float sm[4][16 * NB], sl[4][16 * NB], scq[16 * NB];
  __shared__ union {
    u32x4 q[NB][NK][64];
    f32x4 o[2][NB * NO][64];
  } sh;
  const KvPool& c = p.c;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Blocks of one (sequence, key head, share) are eight apart: on one XCD,
  // whose L2 then holds the share's codes for all of them.
  const int x = blockIdx.x / (8 * p.nrb), rem = blockIdx.x % (8 * p.nrb);
  const int rb = rem >> 3, unit = 8 * x + (rem & 7);
  if (unit >= p.seqs * c.heads * p.nsplit) return;
  const int split = unit % p.nsplit, bh = unit / p.nsplit;
  const int h = bh % c.heads, b = bh / c.heads;
  const int R = p.tokens * p.group;

  const int len = p.lengths[b];
  const int cap = p.width << c.pshift;
  const int npos = len < 0 ? 0 : (int)min((long long)len + p.tokens, (long long)cap);
  const int ntile = (npos + TP - 1) / TP;
  const int per = (ntile + p.nsplit - 1) / p.nsplit;
  const int t1 = min(ntile, (split + 1) * per);
  int tile = split * per + w;

  const int pm = (1 << c.pshift) - 1, lastchunk = max(npos - 1, 0) / CH;
  const int* table = p.tables + (size_t)b * p.width;
  // page of a chunk (of the last one there is for those past the end)
  auto page_of = [&](int chunk, bool& bad) {
    const int pg = glb(table)[(min(chunk, lastchunk) * CH) >> c.pshift];
    bad = (unsigned)pg >= (unsigned)c.pages;
    return bad ? 0 : pg;
  };
  // (page, head) block and offset in it of the chunks of a tile that the lane
  // reads: of its key rows, of its scores and values
  struct Place {
    int k, v, ok, ov;
    bool bad;
  };
  auto find = [&](int tl) {
    Place q;
    bool bk;
    q.k = page_of(4 * tl + (n >> 2), bk);
    q.v = page_of(4 * tl + g, q.bad);
    q.ok = (min(4 * tl + (n >> 2), lastchunk) * CH) & pm;
    q.ov = (min(4 * tl + g, lastchunk) * CH) & pm;
    return q;
  };
  auto load_k = [&](T& t, const Place& q) {
    const size_t at = (((size_t)q.k * c.heads + h) << c.pshift) + q.ok;
    const uint8_t* kr = c.kc + (at + (n & 3)) * T::RB;
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
    t.kz = *glb((const Chunk*)(c.kz + at));
  };
  auto load_g = [&](T& t, const Place& q) {
    t.bad = q.bad;
    const size_t at = (((size_t)q.v * c.heads + h) << c.pshift) + q.ov;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      t.ks[i] = *glb((const f32x4*)(c.ks + at + 4 * i));
      t.vs[i] = *glb((const f32x4*)(c.vs + at + 4 * i));
    }
    t.vz = *glb((const Chunk*)(c.vz + at));
  };
  auto load_v = [&](T& t, const Place& q) {
    const uint8_t* vr = c.vc + ((((size_t)q.v * c.heads + h) * T::RB + n) << c.pshift) + q.ov;
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
  for (int nb = w; nb < NB; nb += 4) {
    const int rr = 16 * (NB * rb + nb) + n, rc = min(rr, R - 1);
    const uint16_t* q = p.q + b * p.qb + (rc / p.group) * p.qt + (h * p.group + rc % p.group) * p.qh;
    float v[NK][8];
    float mx = 0.f;
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
      uint32_t u[4];
      if constexpr (BITS == 8) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const u32x2 a = *glb((const u32x2*)(q + T::off(2 * ks + j, g)));
          u[2 * j] = a[0];
          u[2 * j + 1] = a[1];
        }
      } else {
        const u32x4 a = *glb((const u32x4*)(q + 2 * T::off(ks, g)));
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
    const int up = ex == 0 || ex == 255 ? 0 : min(141 - ex, 100);  // 2^up mx in [2^14, 2^15)
    float f = __uint_as_float((uint32_t)(127 + up) << 23);
    if (p.scale < 0.f) f = -f;
    if (p.scale == 0.f) f = 0.f;
    // (a factor under 2^-100 leaves every weight at 1, as 2^-100 does)
    if (g == 0) scq[16 * nb + n] = fmaxf(fabsf(p.scale) * __uint_as_float((uint32_t)(127 - up) << 23), 0x1p-100f);
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // 4 bits: the odd codes of a word arrive times 16
        const float fj = BITS == 4 && (j & 1) ? f * 0.0625f : f;
        o[j] = pack16(v[ks][2 * j] * fj, v[ks][2 * j + 1] * fj);
      }
      sh.q[nb][ks][lane] = o;
    }
  }
  __syncthreads();

  f32x4 acc[NB][NO];
  float M[NB], l[NB], cq[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    M[nb] = NONE;
    l[nb] = 0.f;
    cq[nb] = scq[16 * nb + n];
#pragma unroll
    for (int i = 0; i < NO; ++i) acc[nb][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // which of the positions j0 .. j0 + CH - 1 does the drafted token of row rr see
  auto seen = [&](int j0, int rr) -> uint32_t {
    const int below = min(max(len - j0, 0), CH), tk = min(rr, R - 1) / p.group;
    uint32_t bits;
    if (p.mask) {
      bits = 0;
      const int i0 = max(j0 - len, 0), wd = i0 >> 5;
      const uint32_t* m = p.mask + ((size_t)b * p.tokens + tk) * p.words;
      if (below < CH) {
        const uint64_t lo = wd < p.words ? m[wd] : 0u, hi = wd + 1 < p.words ? m[wd + 1] : 0u;
        bits = (uint32_t)((hi << 32 | lo) >> (i0 & 31));
      }
      bits = bits << below | ((1u << below) - 1u);
    } else {
      bits = (1u << min(max(len + tk + 1 - j0, 0), CH)) - 1u;
    }
    return bits & ((1u << min(max(npos - j0, 0), CH)) - 1u);
  };

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
        u32x4 a;
        if constexpr (BITS == 8) {
          const uint32_t w0 = t.k[i][2 * ks], w1 = t.k[i][2 * ks + 1];
          a = u32x4{sub16(bytes2(w0, 0), zl[i]), sub16(bytes2(w0, 1), zl[i]), sub16(bytes2(w1, 0), zl[i]),
                    sub16(bytes2(w1, 1), zl[i])};
        } else {
          const uint32_t w0 = t.k[i][ks], w8 = w0 >> 8;
          a = u32x4{sub16(nib_lo(w0), zl[i]), sub16(nib_hi(w0), zh[i]), sub16(nib_lo(w8), zl[i]),
                    sub16(nib_hi(w8), zh[i])};
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) S[nb][i] = mfma(a, q[nb], S[nb][i]);
      }
    }
  };
  auto weights = [&](const T& t, int tl) {
    const bool masked = TP * (tl + 1) > min(len, npos) || __any(t.bad);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float xs[CH], mx = NONE;
      uint32_t see = 0;
#pragma unroll
      for (int i = 0; i < CH; ++i) xs[i] = S[nb][i >> 2][i & 3] * t.ks[i >> 2][i & 3];
      if (masked) {
        see = t.bad ? 0u : seen(TP * tl + CH * g, 16 * (NB * rb + nb) + n);
#pragma unroll
        for (int i = 0; i < CH; ++i) xs[i] = (see >> i) & 1u ? xs[i] : NONE;
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) mx = fmaxf(mx, xs[i]);
      // M moves only when a score passes it by 2^8 (its weight): most tiles then
      // need neither the maximum over the lanes nor a pass over the sums.
      if (__any((mx - M[nb]) * cq[nb] > 8.f)) {
        const float Mn = fmaxf(M[nb], max_groups(mx));
        const float al = Mn > M[nb] ? __builtin_amdgcn_exp2f((M[nb] - Mn) * cq[nb]) : 1.f;
        l[nb] *= al;
#pragma unroll
        for (int i = 0; i < NO; ++i) acc[nb][i] *= al;
        M[nb] = Mn;
      }
      // (nothing seen yet: NONE cq is far below every score's product with cq, and its weights are 0)
      const float ref = M[nb] == NONE ? 0.f : M[nb] * cq[nb];
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(xs[i], cq[nb], -ref));
        l[nb] += e;
        xs[i] = e * t.vs[i >> 2][i & 3];
      }
      if (masked) {
#pragma unroll
        for (int i = 0; i < CH; ++i) xs[i] = (see >> i) & 1u ? xs[i] : 0.f;
      }
#pragma unroll
      for (int s = 0; s < NS; ++s) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // 4 bits: positions (0, 2), (1, 3) of every four, as their bytes come apart
          const float a = xs[8 * s + (BITS == 8 ? 2 * j : 4 * (j >> 1) + (j & 1))];
          const float b = xs[8 * s + (BITS == 8 ? 2 * j + 1 : 4 * (j >> 1) + (j & 1) + 2)];
          P[nb][0][s][j] = lead16(a, b);
          P[nb][1][s][j] = lead16(rest16(a), rest16(b));
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // zero points of the value operand's positions, in the form its codes have
  uint32_t zl[2 * NI], zh[BITS == 4 ? 2 * NI : 1];
  auto zeros = [&](const T& t) {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      if constexpr (BITS == 8) {
        zl[2 * j] = bytes2(t.vz[j], 0);
        zl[2 * j + 1] = bytes2(t.vz[j], 1);
      } else {
        zl[2 * j] = nib_lo(t.vz[j]);
        zl[2 * j + 1] = nib_lo(t.vz[j] >> 8);
        zh[2 * j] = nib_hi(t.vz[j] << 4);
        zh[2 * j + 1] = nib_hi(t.vz[j] >> 4);
      }
    }
  };
  // vector instructions a product: what unpacking takes, over the products
  constexpr int VPM = NB == 1 ? 8 : NB == 2 ? 4 : 3;
  auto values = [&](const T& t) {
#pragma unroll
    for (int i = 0; i < NMB; ++i) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        u32x4 a, e;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t u = t.v[i][2 * s + j];
          const uint32_t *lo = zl + 4 * s + 2 * j, *hi = zh + (BITS == 4 ? 4 * s + 2 * j : 0);
          if constexpr (BITS == 8) {
            a[2 * j] = diff_bf16(bytes2(u, 0), lo[0]);
            a[2 * j + 1] = diff_bf16(bytes2(u, 1), lo[1]);
          } else {
            a[2 * j] = diff_bf16(nib_lo(u), lo[0]);
            a[2 * j + 1] = diff_bf16(nib_lo(u >> 8), lo[1]);
            e[2 * j] = diff_bf16(nib_hi(u), hi[0]);
            e[2 * j + 1] = diff_bf16(nib_hi(u >> 8), hi[1]);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            acc[nb][i] = mfma_bf(a, P[nb][k][s], acc[nb][i]);
            if constexpr (BITS == 4) acc[nb][i + NMB] = mfma_bf(e, P[nb][k][s], acc[nb][i + NMB]);
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
    at = find(tile + 4);
    while (true) {
      const bool more = tile + 4 < t1;
      scores(t);
      __builtin_amdgcn_sched_barrier(0);
      if (more) load_k(t, at);
      __builtin_amdgcn_sched_barrier(0);
      weights(t, tile);
      zeros(t);
      __builtin_amdgcn_sched_barrier(0);
      if (more) load_g(t, at);
      __builtin_amdgcn_sched_barrier(0);
      values(t);
      __builtin_amdgcn_sched_barrier(0);
      if (!more) break;
      load_v(t, at);
      tile += 4;
      at = find(tile + 4);
    }
  }

  // one row's sum from its four lanes
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    l[nb] = sum_groups(l[nb]);
    M[nb] = M[nb] == NONE ? -INFINITY : M[nb] * cq[nb];
    if constexpr (BITS == 4) {  // the upper half's codes came times 16
#pragma unroll
      for (int i = NMB; i < NO; ++i) acc[nb][i] *= 0.0625f;
    }
    if (g == 0) {
      sm[w][16 * nb + n] = M[nb];
      sl[w][16 * nb + n] = l[nb];
    }
  }
  __syncthreads();
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    float mx = -INFINITY, s = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) mx = fmaxf(mx, sm[k][16 * nb + n]);
    const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
    for (int k = 0; k < 4; ++k) s += sl[k][16 * nb + n] * __builtin_amdgcn_exp2f(sm[k][16 * nb + n] - ref);
    const float f = __builtin_amdgcn_exp2f(M[nb] - ref);
#pragma unroll
    for (int i = 0; i < NO; ++i) acc[nb][i] *= f;
    M[nb] = mx;
    l[nb] = s;
  }
  auto put = [&](int k) {
#pragma unroll
    for (int i = 0; i < NB * NO; ++i) sh.o[k][i][lane] = acc[i / NO][i % NO];
  };
  auto add = [&](int k) {
#pragma unroll
    for (int i = 0; i < NB * NO; ++i) acc[i / NO][i % NO] += sh.o[k][i][lane];
  };
  if (w >= 2) put(w - 2);
  __syncthreads();
  if (w < 2) add(w);
  __syncthreads();
  if (w == 1) put(0);
  __syncthreads();
  if (w == 0) {
    add(0);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int rr = 16 * (NB * rb + nb) + n;
      if (rr >= R) continue;
      if (p.nsplit == 1) {
        const float inv = l[nb] == 0.f ? 0.f : 1.f / l[nb];
        uint16_t* o = p.o + b * p.ob + (rr / p.group) * p.ot + (h * p.group + rr % p.group) * p.oh;
#pragma unroll
        for (int i = 0; i < NO; ++i)
          *(bf16x4*)(o + 16 * i + 4 * g) = __builtin_convertvector(acc[nb][i] * inv, bf16x4);
      } else {
        const size_t row = ((size_t)bh * R + rr) * p.nsplit + split;
#pragma unroll
        for (int i = 0; i < NO; ++i) {
          float* o = p.part + row * DIM + 16 * i + 4 * g;
          put_shared(o, acc[nb][i][0], acc[nb][i][1]);
          put_shared(o + 2, acc[nb][i][2], acc[nb][i][3]);
        }
        if (g == 0) put_shared(p.ml + 2 * row, M[nb], l[nb]);
      }
    }
  }
  if (!p.count) return;
  __shared__ int last;
  if (w == 0) {
    // this wave wrote the rows: they are in memory before the count says so
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (lane == 0) {
      int* ct = p.count + (size_t)bh * p.nrb + rb;
      last = __hip_atomic_fetch_add(ct, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == p.nsplit - 1;
      if (last) __hip_atomic_store(ct, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  __syncthreads();
  if (!last) return;
  const int r1 = min(16 * NB, R - 16 * NB * rb);
  for (int i = tid; i < r1 * (DIM / 4); i += 256)
    join_row<1, true>(p, (long long)bh * R + 16 * NB * rb + i / (DIM / 4), 4 * (i % (DIM / 4)), 0, nullptr);
}

template <int G>
__global__ __launch_bounds__(256) void k_attn_join(const AttnProb p) {
  __shared__ JoinLds<G> s;
  const int q4 = p.c.dim >> 2, rows = max(256 / (q4 * G), 1);
  const int i = threadIdx.x / (q4 * G), k = threadIdx.x / q4 % G, d = 4 * (threadIdx.x % q4);
  const long long row = (long long)blockIdx.x * rows + i;
  join_row<G, false>(p, i < rows && row < (long long)p.seqs * p.c.heads * p.tokens * p.group ? row : -1, d, k, &s);
}

// Shares and row blocks of a call: as few blocks as blocks of up to 48 rows
// (32 for head sizes above 128, whose sums need the registers) allow, of equal size.
void plan_tree_attn(AttnProb& p, int ncu) {
  const long long R = (long long)p.tokens * p.group;
  const long long r16 = (R + 15) / 16, most = p.c.dim <= 128 ? 3 : 2;
  p.nrb = (int)((r16 + most - 1) / most);
  p.nb = (int)((r16 + p.nrb - 1) / p.nrb);
  const long long items = (long long)p.seqs * p.c.heads * p.nrb;
  const long long tiles = (((long long)p.width << p.c.pshift) + 63) / 64;
  long long s = (2LL * ncu + items - 1) / items;
  s = s < (tiles + 3) / 4 ? s : (tiles + 3) / 4;
  p.nsplit = (int)(s < 1 ? 1 : s > 128 ? 128 : s);
}

namespace {
template <int DIM, int BITS>
void attn_nb(const AttnProb& p, dim3 grid, hipStream_t st) {
  if (p.nb == 1)
    hipLaunchKernelGGL((k_tree_attn<DIM, BITS, 1, DIM <= 128 ? 64 : 32, 2>), grid, dim3(256), 0, st, p);
  else if (p.nb == 2)
    hipLaunchKernelGGL((k_tree_attn<DIM, BITS, 2, 32, DIM <= 128 ? 2 : 1>), grid, dim3(256), 0, st, p);
  else if constexpr (DIM <= 128)
    hipLaunchKernelGGL((k_tree_attn<DIM, BITS, 3, 32, 2>), grid, dim3(256), 0, st, p);
}
template <int BITS>
hipError_t attn_dim(const AttnProb& p, hipStream_t st) {
  const long long units = (long long)p.seqs * p.c.heads * p.nsplit;
  const dim3 grid((unsigned)((units + 7) / 8 * 8 * p.nrb));
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
  // eight threads for a value where there are many shares: 160 rows of 128
  // shares 8 us, 15 with one; 13824 rows of three shares 5 us, 11 with eight
  const int G = p.nsplit >= 16 && p.c.dim <= 128 ? 8 : p.nsplit >= 16 ? 4 : 1;
  const int rows = std::max(256 / (p.c.dim / 4 * G), 1);
  const long long n = (long long)p.seqs * p.c.heads * p.tokens * p.group;
  const dim3 grid((unsigned)((n + rows - 1) / rows));
  if (G == 8)
    hipLaunchKernelGGL(k_attn_join<8>, grid, dim3(256), 0, st, p);
  else if (G == 4)
    hipLaunchKernelGGL(k_attn_join<4>, grid, dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL(k_attn_join<1>, grid, dim3(256), 0, st, p);
  return hipGetLastError();
}
