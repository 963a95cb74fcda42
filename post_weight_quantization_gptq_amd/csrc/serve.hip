// Rotary positions and the key/value cache on low-precision grids (gfx950):
// what a served layer runs between its quantised products.
#include "common.h"
#include "serve.h"

#include <algorithm>

// Outputs from the last-level cache's size on are stored past the caches: what
// reads them next would not find them there, and they push out what is.  Smaller
// ones are left in the caches for it.  Past them, and ordinary, us:
//   read back           64 MB   128 MB   192 MB   256 MB   384 MB
//   alone               19, 19  33, 43   47, 63   79, 83   114, 119
//   and copied          45, 40  91, 86   142, 150 182, 187 266, 268
//   and its maximum     58, 54  94, 82   129, 109 162, 164 230, 238
//   rotary              64 MB   128 MB   192 MB   256 MB   384 MB
//   alone               34, 36  69, 71   102, 105 136, 138 201, 205
//   and copied          62, 56  124, 126 183, 181 243, 240 357, 358
//   and its maximum     62, 56  111, 101 161, 160 210, 211 310, 314
#define STREAM_BYTES (256LL << 20)

namespace {

__device__ __forceinline__ float bf_up(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
__device__ __forceinline__ uint16_t bf_down(float v) {  // nearest, ties to even
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// N consecutive values of either type, in 32 bits.
template <int N>
struct alignas(2 * N) Bf {
  uint16_t v[N];
};
template <int N>
struct alignas(4 * N) Fl {
  float v[N];
};
template <int N>
__device__ __forceinline__ void load_vals(const uint16_t* p, float* o) {
  const Bf<N> t = *(const Bf<N>*)p;
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = bf_up(t.v[i]);
}
template <int N>
__device__ __forceinline__ void load_vals(const float* p, float* o) {
  const Fl<N> t = *(const Fl<N>*)p;
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = t.v[i];
}
// STREAM: past the caches (see STREAM_BYTES)
template <int N, bool STREAM = false, class V>
__device__ __forceinline__ void store_bits(void* p, const V& t) {
  typedef uint32_t W __attribute__((ext_vector_type(sizeof(V) >= 16 ? 4 : sizeof(V) >= 8 ? 2 : 1)));
  if constexpr (STREAM && sizeof(V) % sizeof(W) == 0) {
    struct Parts {
      W w[sizeof(V) / sizeof(W)];
    };
    const Parts q = __builtin_bit_cast(Parts, t);
#pragma unroll
    for (unsigned i = 0; i < sizeof(V) / sizeof(W); ++i) __builtin_nontemporal_store(q.w[i], (W*)p + i);
  } else {
    *(V*)p = t;
  }
}
template <int N, bool STREAM = false>
__device__ __forceinline__ void store_vals(uint16_t* p, const float* v) {
  Bf<N> t;
#pragma unroll
  for (int i = 0; i < N; ++i) t.v[i] = bf_down(v[i]);
  store_bits<N, STREAM>(p, t);
}
template <int N, bool STREAM = false>
__device__ __forceinline__ void store_vals(float* p, const float* v) {
  Fl<N> t;
#pragma unroll
  for (int i = 0; i < N; ++i) t.v[i] = v[i];
  store_bits<N, STREAM>(p, t);
}

}  // namespace

// ---------------------------------------------------------------- rotary --
// table[p][0][i] = mag cos(p f_i), table[p][1][i] = mag sin(p f_i), rows from
// position `first` on: the angle and its cosine in fp64 (p f_i passes 1e5, where an
// fp32 angle would be off by 1e-2), rounded once.  Made once for a model; not tuned.
__global__ __launch_bounds__(256) void k_rope_table(const RopeFreq f, int first, int length, int half, double mag,
                                                    float* __restrict__ table) {
  const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
  if (idx >= (long long)length * half) return;
  const long long p = idx / half;
  const int i = (int)(idx % half);
  double s, c;
  sincos((double)(first + p) * f.f[i], &s, &c);
  table[p * 2 * half + i] = (float)(mag * c);
  table[p * 2 * half + half + i] = (float)(mag * s);
}

// (a, b) -> (a c - b s, b c + a s) on the pairs (i, i + rot/2) (halves) or
// (2i, 2i + 1) (interleaved) of the first rot values of every head; the other
// values are copied.  A thread takes V pairs of one (token, head); a position
// outside the table gives NaN.  Bound by HBM: 8192 tokens of 40 heads of 128
// from float32 to bf16, 256 MB in 43 us, 5.9 TB/s; a few tokens by the launch, 3.3 us.
template <class TX, class TY, int V, bool INTER, bool STREAM>
__global__ __launch_bounds__(256) void k_rope(const RopeProb p) {
  const int half = p.rot / 2;
  const int nrot = half / V, nth = nrot + (p.dim - p.rot) / (2 * V);  // threads of one head
  const unsigned idx = blockIdx.x * 256 + threadIdx.x, row = idx / nth;
  const int u = (int)(idx % nth);
  const long long t = row / (unsigned)p.heads;
  const int h = (int)(row % (unsigned)p.heads);
  if (t >= p.tokens) return;
  const TX* x = (const TX*)p.x + t * p.xt + h * p.xh;
  TY* y = (TY*)p.y + t * p.yt + h * p.yh;
  float a[V], b[V], r[V], q[V];
  if (u >= nrot) {
    const int i = p.rot + (u - nrot) * 2 * V;
    load_vals<V>(x + i, a);
    load_vals<V>(x + i + V, b);
    store_vals<V, STREAM>(y + i, a);
    store_vals<V, STREAM>(y + i + V, b);
    return;
  }
  const int i = u * V, pos = p.pos[t];
  const bool in = (unsigned)pos < (unsigned)p.length;
  const float* tab = p.table + (long long)(in ? pos : 0) * 2 * half + i;
  float c[V], s[V];
  load_vals<V>(tab, c);
  load_vals<V>(tab + half, s);
  if (INTER) {
    float w[2 * V];
    load_vals<2 * V>(x + 2 * i, w);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      a[j] = w[2 * j];
      b[j] = w[2 * j + 1];
    }
  } else {
    load_vals<V>(x + i, a);
    load_vals<V>(x + half + i, b);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float sj = p.sign * s[j];
    r[j] = in ? a[j] * c[j] - b[j] * sj : NAN;
    q[j] = in ? b[j] * c[j] + a[j] * sj : NAN;
  }
  if (INTER) {
    float w[2 * V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      w[2 * j] = r[j];
      w[2 * j + 1] = q[j];
    }
    store_vals<2 * V, STREAM>(y + 2 * i, w);
  } else {
    store_vals<V, STREAM>(y + i, r);
    store_vals<V, STREAM>(y + half + i, q);
  }
}

// ----------------------------------------------------------- cache write --
// Grid of one row (the dim values of a token's K or V in one head), every
// step in fp32: lo = min(v, 0), hi = max(v, 0), s = (hi - lo) fl32(1 / maxq),
// r = 1 / s, z = rne(-lo r).  A range under 2^-100 (r would overflow) is
// stored as zeros on s = 1; a row with a NaN or an infinity, or whose range
// overflows, gets s = NaN and so reads back as NaN.  The step is the product by
// definition.  The correctly rounded quotient (hi - lo) / maxq, which the weights'
// grids take, is up to one rounding apart; where -lo / s lies half way between two
// zero points (rows with hi = -lo, common in bf16) it may give the other one.  A
// product is what elementwise tensor code on this GPU makes of a division by a
// constant, so that a cache filled by such code holds the same codes.
struct KvGrid {
  float s, r, z;
};
__device__ __forceinline__ KvGrid kv_grid(float mn, float mx, bool bad, float maxq) {
  const float lo = fminf(mn, 0.f), hi = fmaxf(mx, 0.f), d = hi - lo;
  KvGrid g;
  if (bad || !(d <= 3.402823466e38f)) {
    g.s = NAN;
    g.r = g.z = 0.f;
  } else if (d < 0x1p-100f) {
    g.s = 1.f;
    g.r = 1.f;
    g.z = 0.f;
  } else {
    g.s = __fmul_rn(d, 1.f / maxq);
    g.r = 1.f / g.s;
    g.z = fminf(fmaxf(rintf(__fmul_rn(-lo, g.r)), 0.f), maxq);
  }
  return g;
}
__device__ __forceinline__ uint32_t kv_code(float v, const KvGrid& g, float maxq) {
  const float q = fminf(fmaxf(rintf(__fadd_rn(__fmul_rn(v, g.r), g.z)), 0.f), maxq);
  return (uint32_t)q;  // NaN: fmaxf gave 0
}

// Bytes of (page, head) blocks before slot's own.
__device__ __forceinline__ size_t kv_block(const KvPool& c, int slot, int h) {
  return (size_t)(slot >> c.pshift) * c.heads + h;
}

// Slots of the TW tokens from t0 on; -1: outside the pool, or no token.
template <int TW>
__device__ __forceinline__ void load_slots(const int* slots, long long t0, long long tokens, const KvPool& c, int* sl) {
  const int i = threadIdx.x;
  if (i < TW) {
    const int s = t0 + i < tokens ? slots[t0 + i] : -1;
    sl[i] = s >= 0 && s < (long long)c.pages << c.pshift ? s : -1;
  }
  __syncthreads();
}
// Whether four tokens lie side by side in one page.
__device__ __forceinline__ bool run_of_4(const int* s, int pm) {
  return s[0] >= 0 && s[1] == s[0] + 1 && s[2] == s[0] + 2 && s[3] == s[0] + 3 && (s[0] & pm) + 3 <= pm;
}
// Bytes e of the words w[0..3] become word e (a 4 x 4 transpose).
__device__ __forceinline__ void transpose4(uint32_t* w) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  w[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  w[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  w[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  w[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// Window of tokens, head and kind (0 keys, 1 values) of a workgroup: all of a
// window's on one XCD (workgroups go to the eight in turn), one after the other,
// so that the rows of its heads, which touch, meet in one L2.
__device__ __forceinline__ long long kv_window(const KvPool& c, int& h, int& kv) {
  const int xcd = blockIdx.x & 7, i = blockIdx.x >> 3;
  h = i % c.heads;
  kv = i / c.heads & 1;
  return (long long)(i / (2 * c.heads)) * 8 + xcd;
}

// A workgroup takes TW consecutive input tokens of one head, its keys or its
// values.  G lanes hold a row, eight neighbouring values
// each.  Key codes go straight to the pool; value codes through LDS, from where
// blocks of 4 tokens x 4 dimensions are transposed in registers, so that the
// tokens of a dimension, which lie side by side in the pool, leave as words
// where four slots follow each other inside a page.  Bound by HBM: 8194 tokens
// of 8 heads of 128 from float32 to 4 bits, 76 MB in 16 us, 4.6 TB/s (22 us with
// one byte of a dimension at a time); 16 tokens 5 us.
template <class T, int BITS, int D, int TW>
__global__ __launch_bounds__(256) void k_kv_write(const KvWriteProb p) {
  constexpr int G = D <= 64 ? 8 : D <= 128 ? 16 : 32, PITCH = D + 4, RB = D * BITS / 8;
  __shared__ __attribute__((aligned(16))) uint8_t vt[TW * PITCH];
  __shared__ int sl[TW];
  const KvPool& c = p.c;
  const int tid = threadIdx.x, lane = tid % G;
  int h, kv;
  const long long t0 = kv_window(c, h, kv) * TW;
  if (t0 >= p.tokens) return;
  const int pm = (1 << c.pshift) - 1;
  constexpr float maxq = (float)((1 << BITS) - 1);
  load_slots<TW>(p.slots, t0, p.tokens, c, sl);
  for (int i = tid / G; i < TW; i += 256 / G) {
    const int slot = sl[i];
    if (slot < 0) continue;
    const T* src = kv ? (const T*)p.v + (t0 + i) * p.vt + h * p.vh : (const T*)p.k + (t0 + i) * p.kt + h * p.kh;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (8 * lane < D) {
      load_vals<4>(src + 8 * lane, v);
      load_vals<4>(src + 8 * lane + 4, v + 4);
    }
    float mn = 0.f, mx = 0.f;
    int bad = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      mn = fminf(mn, v[e]);
      mx = fmaxf(mx, v[e]);
      bad |= !(fabsf(v[e]) <= 3.402823466e38f);
    }
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) {
      mn = fminf(mn, __shfl_xor(mn, o));
      mx = fmaxf(mx, __shfl_xor(mx, o));
      bad |= __shfl_xor(bad, o);
    }
    const KvGrid g = kv_grid(mn, mx, bad, maxq);
    const size_t at = (kv_block(c, slot, h) << c.pshift) + (slot & pm);
    if (lane == 0) {
      (kv ? c.vs : c.ks)[at] = g.s;
      (kv ? c.vz : c.kz)[at] = (uint8_t)g.z;
    }
    if (8 * lane >= D) continue;
    uint32_t q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = kv_code(v[e], g, maxq);
    const uint32_t lo = q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24, hi = q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24;
    if (kv) {
      *(uint32_t*)(vt + i * PITCH + 8 * lane) = lo;
      *(uint32_t*)(vt + i * PITCH + 8 * lane + 4) = hi;
    } else if (BITS == 8) {
      *(uint64_t*)(c.kc + at * RB + 8 * lane) = (uint64_t)hi << 32 | lo;
    } else {  // two codes a byte
      const uint32_t a = (lo | lo >> 4) & 0x00FF00FFu, b = (hi | hi >> 4) & 0x00FF00FFu;
      *(uint32_t*)(c.kc + at * RB + 4 * lane) = ((a | a >> 8) & 0xFFFFu) | (b | b >> 8) << 16;
    }
  }
  if (!kv) return;
  __syncthreads();
  constexpr int GW = TW / 4;
  for (int job = tid; job < RB / 4 * GW; job += 256) {
    const int r = 4 * (job / GW), i = 4 * (job % GW);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = *(const uint32_t*)(vt + (i + e) * PITCH + r);
    if (BITS == 4) {  // the dimensions D/2 on in the high halves (the bytes of skipped tokens hold anything)
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] |= (*(const uint32_t*)(vt + (i + e) * PITCH + r + D / 2) & 0x0F0F0F0Fu) << 4;
    }
    transpose4(w);
    if (run_of_4(sl + i, pm)) {
      uint8_t* dst = c.vc + ((kv_block(c, sl[i], h) * RB + r) << c.pshift) + (sl[i] & pm);
#pragma unroll
      for (int e = 0; e < 4; ++e) __builtin_memcpy(dst + ((size_t)e << c.pshift), &w[e], 4);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int s = sl[i + j];
        if (s < 0) continue;
        uint8_t* dst = c.vc + ((kv_block(c, s, h) * RB + r) << c.pshift) + (s & pm);
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[(size_t)e << c.pshift] = (uint8_t)(w[e] >> (8 * j));
      }
    }
  }
}

// ------------------------------------------------------------ cache read --
// The inverse, laid out the same: fl32(s (q - z)), rounded once to the output
// type; a slot outside the pool reads as zeros.  Bound by HBM: 32768 tokens of 8
// heads of 128, 8 bits to bf16, 204 MB in 41 us, 4.9 TB/s; 300 tokens 3.6 us.
template <class T, int BITS, int D, int TW>
__global__ __launch_bounds__(256) void k_kv_read(const KvReadProb p) {
  constexpr int RB = D * BITS / 8, PITCH = RB + 4, L = D / 8;
  __shared__ __attribute__((aligned(16))) uint8_t vt[TW * PITCH];
  __shared__ int sl[TW];
  const KvPool& c = p.c;
  const int tid = threadIdx.x;
  int h, kv;
  const long long t0 = kv_window(c, h, kv) * TW;
  if (t0 >= p.tokens) return;
  const int nt = (int)min((long long)TW, p.tokens - t0);
  const int pm = (1 << c.pshift) - 1;
  load_slots<TW>(p.slots, t0, p.tokens, c, sl);
  if (kv) {
    constexpr int GW = TW / 4;
    for (int job = tid; job < RB / 4 * GW; job += 256) {
      const int r = 4 * (job / GW), i = 4 * (job % GW);
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      if (run_of_4(sl + i, pm)) {
        const uint8_t* src = c.vc + ((kv_block(c, sl[i], h) * RB + r) << c.pshift) + (sl[i] & pm);
#pragma unroll
        for (int e = 0; e < 4; ++e) __builtin_memcpy(&w[e], src + ((size_t)e << c.pshift), 4);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int s = sl[i + j];
          if (s < 0) continue;
          const uint8_t* src = c.vc + ((kv_block(c, s, h) * RB + r) << c.pshift) + (s & pm);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] |= (uint32_t)src[(size_t)e << c.pshift] << (8 * j);
        }
      }
      transpose4(w);
#pragma unroll
      for (int e = 0; e < 4; ++e) *(uint32_t*)(vt + (i + e) * PITCH + r) = w[e];
    }
    __syncthreads();
  }
  for (int job = tid; job < nt * L; job += 256) {
    const int i = job / L, d = 8 * (job % L), slot = sl[i];
    T* dst = kv ? (T*)p.v + (t0 + i) * p.vt + h * p.vh : (T*)p.k + (t0 + i) * p.kt + h * p.kh;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (slot >= 0) {
      const size_t at = (kv_block(c, slot, h) << c.pshift) + (slot & pm);
      const float s = (kv ? c.vs : c.ks)[at], z = (float)(kv ? c.vz : c.kz)[at];
      uint32_t lo, hi;
      if (kv) {
        const int r = BITS == 8 || d < D / 2 ? d : d - D / 2, sh = BITS == 8 || d < D / 2 ? 0 : 4;
        lo = *(const uint32_t*)(vt + i * PITCH + r);
        hi = *(const uint32_t*)(vt + i * PITCH + r + 4);
        if (BITS == 4) {
          lo = (lo >> sh) & 0x0F0F0F0Fu;
          hi = (hi >> sh) & 0x0F0F0F0Fu;
        }
      } else if (BITS == 8) {
        const uint64_t u = *(const uint64_t*)(c.kc + at * RB + d);
        lo = (uint32_t)u;
        hi = (uint32_t)(u >> 32);
      } else {
        const uint32_t u = *(const uint32_t*)(c.kc + at * RB + d / 2);
        const uint32_t e = u & 0x0F0F0F0Fu, o = (u >> 4) & 0x0F0F0F0Fu;  // even and odd codes
        lo = __builtin_amdgcn_perm(o, e, 0x05010400u);
        hi = __builtin_amdgcn_perm(o, e, 0x07030602u);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = __fmul_rn(s, (float)((lo >> (8 * e)) & 255u) - z);
        v[e + 4] = __fmul_rn(s, (float)((hi >> (8 * e)) & 255u) - z);
      }
    }
    if (p.wide) {
      if (p.stream)
        store_vals<8, true>(dst + d, v);
      else
        store_vals<8>(dst + d, v);
    } else {
      store_vals<4>(dst + d, v);
      store_vals<4>(dst + d + 4, v + 4);
    }
  }
}

// ------------------------------------------------------------- launchers --
hipError_t launch_rope_table(const RopeFreq& f, int length, int half, double mag, float* table, hipStream_t st) {
  const long long most = (1LL << 31) / half;  // positions a launch: its threads are counted in 32 bits
  for (long long t = 0; t < length; t += most) {
    const int n = (int)std::min(most, length - t);
    const dim3 grid((unsigned)(((long long)n * half + 255) / 256));
    hipLaunchKernelGGL(k_rope_table, grid, dim3(256), 0, st, f, (int)t, n, half, mag, table + t * 2 * half);
  }
  return hipGetLastError();
}

namespace {

// V pairs per thread: the widest for which every access is aligned
template <class TX, class TY, bool INTER>
hipError_t rope_v(const RopeProb& p, hipStream_t st) {
  auto fits = [&](int v) {
    const int e = INTER ? 2 * v : v;  // values per access
    return (p.rot / 2) % v == 0 && (p.dim - p.rot) % (2 * v) == 0 && (INTER || (p.rot / 2) % e == 0) &&
           p.xt % e == 0 && p.xh % e == 0 && p.yt % e == 0 && p.yh % e == 0 &&
           (uintptr_t)p.x % (e * sizeof(TX)) == 0 && (uintptr_t)p.y % (e * sizeof(TY)) == 0 &&
           (uintptr_t)p.table % (4 * v) == 0;
  };
  // eight where the result is bf16, so that a store is 16 bytes (a prompt of
  // 8192 x 40 heads of 128 from float32: 43 to 45 us, 53 with four)
  const int v = sizeof(TY) == 2 && fits(8) ? 8 : fits(4) ? 4 : 1;
  const int nth = p.dim / (2 * v);
  const bool stream = p.tokens * p.heads * p.dim * (long long)sizeof(TY) >= STREAM_BYTES;
  // threads of a launch are counted in 32 bits
  const long long most = std::max((1LL << 31) / ((long long)p.heads * nth), 1LL);
  for (long long t = 0; t < p.tokens; t += most) {
    RopeProb q = p;
    q.tokens = std::min(most, p.tokens - t);
    q.x = (const TX*)p.x + t * p.xt;
    q.y = (TY*)p.y + t * p.yt;
    q.pos = p.pos + t;
    const dim3 grid((unsigned)((q.tokens * q.heads * nth + 255) / 256));
    if (v == 8) {
      if constexpr (sizeof(TY) == 2)
        hipLaunchKernelGGL((stream ? k_rope<TX, TY, 8, INTER, true> : k_rope<TX, TY, 8, INTER, false>), grid, dim3(256),
                           0, st, q);
    } else if (v == 4) {
      hipLaunchKernelGGL((stream ? k_rope<TX, TY, 4, INTER, true> : k_rope<TX, TY, 4, INTER, false>), grid, dim3(256), 0,
                         st, q);
    } else {
      hipLaunchKernelGGL((k_rope<TX, TY, 1, INTER, false>), grid, dim3(256), 0, st, q);
    }
  }
  return hipGetLastError();
}
template <class TX, class TY>
hipError_t rope_l(const RopeProb& p, int layout, hipStream_t st) {
  return layout ? rope_v<TX, TY, true>(p, st) : rope_v<TX, TY, false>(p, st);
}

// 64 tokens a workgroup where that makes 512 of them, else 16; as many tokens a
// launch as keep its threads under 2^32
template <class T, int BITS, int D, class P>
void kv_launch(const P& p, hipStream_t st, void (*wide)(P), void (*narrow)(P)) {
  const bool w = (p.tokens + 63) / 64 * p.c.heads >= 256;
  const long long tw = w ? 64 : 16, most = ((1LL << 24) - 1) / (2 * p.c.heads) / 8 * 8 * tw;
  for (long long t = 0; t < p.tokens; t += most) {
    P q = p;
    q.tokens = std::min(most, p.tokens - t);
    q.k = (decltype(q.k))((uintptr_t)p.k + t * p.kt * sizeof(T));
    q.v = (decltype(q.v))((uintptr_t)p.v + t * p.vt * sizeof(T));
    q.slots = p.slots + t;
    const dim3 grid((unsigned)(((q.tokens + tw - 1) / tw + 7) / 8 * 8 * p.c.heads * 2));
    hipLaunchKernelGGL(w ? wide : narrow, grid, dim3(256), 0, st, q);
  }
}
template <class T, int BITS, int D>
void kv_one(const KvWriteProb& p, hipStream_t st) {
  kv_launch<T, BITS, D>(p, st, k_kv_write<T, BITS, D, 64>, k_kv_write<T, BITS, D, 16>);
}
template <class T, int BITS, int D>
void kv_one(const KvReadProb& p, hipStream_t st) {
  kv_launch<T, BITS, D>(p, st, k_kv_read<T, BITS, D, 64>, k_kv_read<T, BITS, D, 16>);
}
template <class T, int BITS, class P>
hipError_t kv_dim(const P& p, hipStream_t st) {
  switch (p.c.dim) {
    case 64: kv_one<T, BITS, 64>(p, st); break;
    case 96: kv_one<T, BITS, 96>(p, st); break;
    case 128: kv_one<T, BITS, 128>(p, st); break;
    case 192: kv_one<T, BITS, 192>(p, st); break;
    default: kv_one<T, BITS, 256>(p, st); break;
  }
  return hipGetLastError();
}
template <class P>
hipError_t kv_any(const P& p, int type, int bits, hipStream_t st) {
  if (type) return bits == 8 ? kv_dim<float, 8>(p, st) : kv_dim<float, 4>(p, st);
  return bits == 8 ? kv_dim<uint16_t, 8>(p, st) : kv_dim<uint16_t, 4>(p, st);
}

}  // namespace

hipError_t launch_rope(const RopeProb& p, int xtype, int ytype, int layout, hipStream_t st) {
  if (xtype)
    return ytype ? rope_l<float, float>(p, layout, st) : rope_l<float, uint16_t>(p, layout, st);
  return ytype ? rope_l<uint16_t, float>(p, layout, st) : rope_l<uint16_t, uint16_t>(p, layout, st);
}

hipError_t launch_kv_write(const KvWriteProb& p, int type, int bits, hipStream_t st) {
  return kv_any(p, type, bits, st);
}

hipError_t launch_kv_read(KvReadProb p, int type, int bits, hipStream_t st) {
  p.wide = (p.kt | p.kh | p.vt | p.vh) % 8 == 0 && ((uintptr_t)p.k | (uintptr_t)p.v) % (type ? 32 : 16) == 0;
  p.stream = p.tokens * p.c.heads * p.c.dim * (type ? 8LL : 4LL) >= STREAM_BYTES;
  return kv_any(p, type, bits, st);
}
