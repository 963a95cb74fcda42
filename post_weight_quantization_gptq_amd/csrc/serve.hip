// Rotary positions and the key/value cache on low-precision grids (gfx950):
// what a served layer runs between its quantised products.
#include "common.h"
#include "serve.h"

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
template <int N>
__device__ __forceinline__ void store_vals(uint16_t* p, const float* v) {
  Bf<N> t;
#pragma unroll
  for (int i = 0; i < N; ++i) t.v[i] = bf_down(v[i]);
  *(Bf<N>*)p = t;
}
template <int N>
__device__ __forceinline__ void store_vals(float* p, const float* v) {
  Fl<N> t;
#pragma unroll
  for (int i = 0; i < N; ++i) t.v[i] = v[i];
  *(Fl<N>*)p = t;
}

}  // namespace

// ---------------------------------------------------------------- rotary --
// table[p][0][i] = mag cos(p f_i), table[p][1][i] = mag sin(p f_i): the angle
// and its cosine in fp64 (p f_i passes 1e5, where an fp32 angle would be off
// by 1e-2), rounded once.
__global__ __launch_bounds__(256) void k_rope_table(const RopeFreq f, int length, int half, double mag,
                                                    float* __restrict__ table) {
  const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
  if (idx >= (long long)length * half) return;
  const long long p = idx / half;
  const int i = (int)(idx % half);
  double s, c;
  sincos((double)p * f.f[i], &s, &c);
  table[p * 2 * half + i] = (float)(mag * c);
  table[p * 2 * half + half + i] = (float)(mag * s);
}

// (a, b) -> (a c - b s, b c + a s) on the pairs (i, i + rot/2) (halves) or
// (2i, 2i + 1) (interleaved) of the first rot values of every head; the other
// values are copied.  A thread takes V pairs of one (token, head); a position
// outside the table gives NaN.
template <class TX, class TY, int V, bool INTER>
__global__ __launch_bounds__(256) void k_rope(const RopeProb p) {
  const int half = p.rot / 2;
  const int nrot = half / V, nth = nrot + (p.dim - p.rot) / (2 * V);  // threads of one head
  const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long row = idx / nth;
  const int u = (int)(idx % nth);
  if (row >= p.tokens * p.heads) return;
  const long long t = row / p.heads;
  const int h = (int)(row % p.heads);
  const TX* x = (const TX*)p.x + t * p.xt + h * p.xh;
  TY* y = (TY*)p.y + t * p.yt + h * p.yh;
  float a[V], b[V], r[V], q[V];
  if (u >= nrot) {
    const int i = p.rot + (u - nrot) * 2 * V;
    load_vals<V>(x + i, a);
    load_vals<V>(x + i + V, b);
    store_vals<V>(y + i, a);
    store_vals<V>(y + i + V, b);
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
    store_vals<2 * V>(y + 2 * i, w);
  } else {
    store_vals<V>(y + i, r);
    store_vals<V>(y + half + i, q);
  }
}

// ----------------------------------------------------------- cache write --
// Grid of one row (the dim values of a token's K or V in one head), every
// step in fp32: lo = min(v, 0), hi = max(v, 0), s = (hi - lo) / maxq,
// r = 1 / s, z = rne(-lo r).  A range under 2^-100 (r would overflow) is
// stored as zeros on s = 1; a row with a NaN or an infinity, or whose range
// overflows, gets s = NaN and so reads back as NaN.
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
    g.s = d / maxq;
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

// A workgroup takes TW consecutive input tokens of one head.  Sixteen lanes
// hold a row, four neighbouring values each per 64; K codes go straight to
// the pool, V codes through LDS, so that the tokens of a dimension, which lie
// side by side in the pool, leave as 4-byte words where four slots follow
// each other inside a page.
template <class T, int BITS, int NCH, int TW>
__global__ __launch_bounds__(256) void k_kv_write(const KvWriteProb p) {
  constexpr int PITCH = TW + 4;  // bytes of an LDS row: an odd number of words
  __shared__ __attribute__((aligned(16))) uint8_t vt[64 * NCH * PITCH];
  __shared__ int sl[TW];
  const KvPool& c = p.c;
  const int tid = threadIdx.x, lane = tid & 15, sub = tid >> 4;
  const int h = blockIdx.y;
  const long long t0 = (long long)blockIdx.x * TW;
  const int nt = (int)min((long long)TW, p.tokens - t0);
  const int pm = (1 << c.pshift) - 1, D = c.dim;
  const long long nslot = (long long)c.pages << c.pshift;
  constexpr float maxq = (float)((1 << BITS) - 1);
  if (tid < TW) {
    const int s = tid < nt ? p.slots[t0 + tid] : -1;
    sl[tid] = s >= 0 && s < nslot ? s : -1;
  }
  __syncthreads();
  for (int job = sub; job < 2 * TW; job += 16) {
    const int kv = job >= TW, i = kv ? job - TW : job;
    const int slot = sl[i];
    if (slot < 0) continue;
    const T* src = kv ? (const T*)p.v + (t0 + i) * p.vt + h * p.vh : (const T*)p.k + (t0 + i) * p.kt + h * p.kh;
    float v[NCH][4];
    float mn = 0.f, mx = 0.f;
    int bad = 0;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int d = 64 * j + 4 * lane;
      if (d < D) load_vals<4>(src + d, v[j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (d >= D) v[j][e] = 0.f;
        mn = fminf(mn, v[j][e]);
        mx = fmaxf(mx, v[j][e]);
        bad |= !(fabsf(v[j][e]) <= 3.402823466e38f);
      }
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      mn = fminf(mn, __shfl_xor(mn, o));
      mx = fmaxf(mx, __shfl_xor(mx, o));
      bad |= __shfl_xor(bad, o);
    }
    const KvGrid g = kv_grid(mn, mx, bad, maxq);
    const size_t blk = kv_block(c, slot, h);
    if (lane == 0) {
      (kv ? c.vs : c.ks)[(blk << c.pshift) + (slot & pm)] = g.s;
      (kv ? c.vz : c.kz)[(blk << c.pshift) + (slot & pm)] = (uint8_t)g.z;
    }
    uint8_t* krow = c.kc + ((blk << c.pshift) + (slot & pm)) * c.rb;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int d = 64 * j + 4 * lane;
      if (d >= D) continue;
      uint32_t q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = kv_code(v[j][e], g, maxq);
      if (kv) {
#pragma unroll
        for (int e = 0; e < 4; ++e) vt[(d + e) * PITCH + i] = (uint8_t)q[e];
      } else if (BITS == 8) {
        *(uint32_t*)(krow + d) = q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24;
      } else {
        *(uint16_t*)(krow + (d >> 1)) = (uint16_t)(q[0] | q[1] << 4 | q[2] << 8 | q[3] << 12);
      }
    }
  }
  __syncthreads();
  constexpr int GW = TW / 4;
  for (int job = tid; job < c.rb * GW; job += 256) {
    const int r = job / GW, i = 4 * (job % GW);
    uint32_t w = *(const uint32_t*)(vt + r * PITCH + i);
    // (the bytes of skipped tokens hold anything)
    if (BITS == 4) w = (w & 0x0F0F0F0Fu) | (*(const uint32_t*)(vt + (r + (D >> 1)) * PITCH + i) & 0x0F0F0F0Fu) << 4;
    const int s0 = sl[i];
    if (s0 >= 0 && sl[i + 1] == s0 + 1 && sl[i + 2] == s0 + 2 && sl[i + 3] == s0 + 3 && (s0 & pm) + 3 <= pm) {
      __builtin_memcpy(c.vc + ((kv_block(c, s0, h) * c.rb + r) << c.pshift) + (s0 & pm), &w, 4);
    } else {
      for (int e = 0; e < 4; ++e) {
        const int s = sl[i + e];
        if (s >= 0) c.vc[((kv_block(c, s, h) * c.rb + r) << c.pshift) + (s & pm)] = (uint8_t)(w >> (8 * e));
      }
    }
  }
}

// ------------------------------------------------------------ cache read --
// The inverse, laid out the same: fl32(s (q - z)), rounded once to the output
// type; a slot outside the pool reads as zeros.
template <class T, int BITS, int NCH, int TW>
__global__ __launch_bounds__(256) void k_kv_read(const KvReadProb p) {
  constexpr int PITCH = TW + 4;
  __shared__ __attribute__((aligned(16))) uint8_t vt[64 * NCH * BITS / 8 * PITCH];
  __shared__ int sl[TW];
  const KvPool& c = p.c;
  const int tid = threadIdx.x, lane = tid & 15, sub = tid >> 4;
  const int h = blockIdx.y;
  const long long t0 = (long long)blockIdx.x * TW;
  const int nt = (int)min((long long)TW, p.tokens - t0);
  const int pm = (1 << c.pshift) - 1, D = c.dim;
  const long long nslot = (long long)c.pages << c.pshift;
  if (tid < TW) {
    const int s = tid < nt ? p.slots[t0 + tid] : -1;
    sl[tid] = s >= 0 && s < nslot ? s : -1;
  }
  __syncthreads();
  constexpr int GW = TW / 4;
  for (int job = tid; job < c.rb * GW; job += 256) {
    const int r = job / GW, i = 4 * (job % GW);
    uint32_t w = 0;
    const int s0 = sl[i];
    if (s0 >= 0 && sl[i + 1] == s0 + 1 && sl[i + 2] == s0 + 2 && sl[i + 3] == s0 + 3 && (s0 & pm) + 3 <= pm) {
      __builtin_memcpy(&w, c.vc + ((kv_block(c, s0, h) * c.rb + r) << c.pshift) + (s0 & pm), 4);
    } else {
      for (int e = 0; e < 4; ++e) {
        const int s = sl[i + e];
        if (s >= 0) w |= (uint32_t)c.vc[((kv_block(c, s, h) * c.rb + r) << c.pshift) + (s & pm)] << (8 * e);
      }
    }
    *(uint32_t*)(vt + r * PITCH + i) = w;
  }
  __syncthreads();
  for (int job = sub; job < 2 * TW; job += 16) {
    const int kv = job >= TW, i = kv ? job - TW : job;
    if (i >= nt) continue;
    const int slot = sl[i];
    T* dst = kv ? (T*)p.v + (t0 + i) * p.vt + h * p.vh : (T*)p.k + (t0 + i) * p.kt + h * p.kh;
    float s = 0.f, z = 0.f;
    const size_t at = slot < 0 ? 0 : (kv_block(c, slot, h) << c.pshift) + (slot & pm);
    if (slot >= 0) {
      s = (kv ? c.vs : c.ks)[at];
      z = (float)(kv ? c.vz : c.kz)[at];
    }
    const uint8_t* krow = c.kc + at * c.rb;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int d = 64 * j + 4 * lane;
      if (d >= D) continue;
      uint32_t q = 0;
      if (slot >= 0) {
        if (kv) {
          const int rows = BITS == 8 ? D : D >> 1;
          const int r = d < rows ? d : d - rows, sh = d < rows ? 0 : 4;  // 4 bits: the upper half's nibbles
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t b = vt[(r + e) * PITCH + i];
            q |= (BITS == 8 ? b : (b >> sh) & 15u) << (8 * e);
          }
        } else if (BITS == 8) {
          q = *(const uint32_t*)(krow + d);
        } else {
          const uint32_t w = *(const uint16_t*)(krow + (d >> 1));
          q = (w & 15u) | (w & 0xF0u) << 4 | (w & 0xF00u) << 8 | (w & 0xF000u) << 12;
        }
      }
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = slot < 0 ? 0.f : __fmul_rn(s, (float)((q >> (8 * e)) & 255u) - z);
      store_vals<4>(dst + d, v);
    }
  }
}

// ------------------------------------------------------------- launchers --
hipError_t launch_rope_table(const RopeFreq& f, int length, int half, double mag, float* table, hipStream_t st) {
  const long long n = (long long)length * half;
  hipLaunchKernelGGL(k_rope_table, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, f, length, half, mag, table);
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
  const int v = fits(4) ? 4 : 1;
  const int nth = p.dim / (2 * v);
  const long long n = p.tokens * p.heads * nth;
  const dim3 grid((unsigned)((n + 255) / 256));
  if (v == 4)
    hipLaunchKernelGGL((k_rope<TX, TY, 4, INTER>), grid, dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((k_rope<TX, TY, 1, INTER>), grid, dim3(256), 0, st, p);
  return hipGetLastError();
}
template <class TX, class TY>
hipError_t rope_l(const RopeProb& p, int layout, hipStream_t st) {
  return layout ? rope_v<TX, TY, true>(p, st) : rope_v<TX, TY, false>(p, st);
}

template <class T, int BITS, int NCH>
void kv_write_n(const KvWriteProb& p, hipStream_t st) {
  const dim3 grid((unsigned)((p.tokens + 63) / 64), p.c.heads);
  hipLaunchKernelGGL((k_kv_write<T, BITS, NCH, 64>), grid, dim3(256), 0, st, p);
}
template <class T, int BITS>
hipError_t kv_write_b(const KvWriteProb& p, hipStream_t st) {
  switch ((p.c.dim + 63) / 64) {
    case 1: kv_write_n<T, BITS, 1>(p, st); break;
    case 2: kv_write_n<T, BITS, 2>(p, st); break;
    case 3: kv_write_n<T, BITS, 3>(p, st); break;
    default: kv_write_n<T, BITS, 4>(p, st); break;
  }
  return hipGetLastError();
}
template <class T, int BITS, int NCH>
void kv_read_n(const KvReadProb& p, hipStream_t st) {
  const dim3 grid((unsigned)((p.tokens + 63) / 64), p.c.heads);
  hipLaunchKernelGGL((k_kv_read<T, BITS, NCH, 64>), grid, dim3(256), 0, st, p);
}
template <class T, int BITS>
hipError_t kv_read_b(const KvReadProb& p, hipStream_t st) {
  switch ((p.c.dim + 63) / 64) {
    case 1: kv_read_n<T, BITS, 1>(p, st); break;
    case 2: kv_read_n<T, BITS, 2>(p, st); break;
    case 3: kv_read_n<T, BITS, 3>(p, st); break;
    default: kv_read_n<T, BITS, 4>(p, st); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeProb& p, int xtype, int ytype, int layout, hipStream_t st) {
  if (xtype)
    return ytype ? rope_l<float, float>(p, layout, st) : rope_l<float, uint16_t>(p, layout, st);
  return ytype ? rope_l<uint16_t, float>(p, layout, st) : rope_l<uint16_t, uint16_t>(p, layout, st);
}

hipError_t launch_kv_write(const KvWriteProb& p, int type, int bits, hipStream_t st) {
  if (type) return bits == 8 ? kv_write_b<float, 8>(p, st) : kv_write_b<float, 4>(p, st);
  return bits == 8 ? kv_write_b<uint16_t, 8>(p, st) : kv_write_b<uint16_t, 4>(p, st);
}

hipError_t launch_kv_read(const KvReadProb& p, int type, int bits, hipStream_t st) {
  if (type) return bits == 8 ? kv_read_b<float, 8>(p, st) : kv_read_b<float, 4>(p, st);
  return bits == 8 ? kv_read_b<uint16_t, 8>(p, st) : kv_read_b<uint16_t, 4>(p, st);
}
