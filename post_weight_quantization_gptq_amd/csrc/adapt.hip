// The quantised product with a low-rank adapter for every row (gfx950):
//   Y = X What^T + alpha_a (X down_a^T) up_a^T,  a = ids[row]
// in two launches: T = X down_a^T into workspace (and, for many rows, the weights as
// bf16), then the product with alpha_a T up_a^T added to its sums before they are
// stored.
#include "common.h"
#include "adapt.h"


namespace {

typedef const __attribute__((address_space(1))) uint32_t gu32;
typedef const __attribute__((address_space(1))) u32x4 gu32x4;
typedef const __attribute__((address_space(1))) uint8_t gu8;
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack2(float a, float b) {  // nearest, ties to even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ float bf_low(uint32_t v) { return __builtin_bit_cast(float, v << 16); }
__device__ __forceinline__ float bf_high(uint32_t v) { return __builtin_bit_cast(float, v & 0xFFFF0000u); }

// The 32 codes of a k-step: BITS words of a row's bitstream; codes 8 u .. 8 u + 7
// as bf16(fl32(s (q - z))), the weights' definition.
template <int BITS>
struct Words {
  uint32_t w[BITS];
};
template <int BITS>
__device__ __forceinline__ u32x4 weights8(const Words<BITS>& c, int u, float s, float z) {
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float v[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int bit = BITS * (8 * u + 2 * j + e), at = bit >> 5, off = bit & 31;
      uint32_t q = c.w[at] >> off;
      if (off + BITS > 32) q |= c.w[at + 1] << (32 - off);
      v[e] = __fmul_rn((float)(q & ((1u << BITS) - 1u)) - z, s);
    }
    o[j] = pack2(v[0], v[1]);
  }
  return u32x4{o[0], o[1], o[2], o[3]};
}

// Calls f(adapter, rows) for each adapter of the rows whose ids the first n
// lanes of the wave hold (id < 0: none); rows: a bit for each.  Uniform.
template <class F>
__device__ __forceinline__ void each_adapter(int id, int n, F&& f) {
  uint64_t left = __ballot((int)(threadIdx.x & 63) < n && id >= 0);
  while (left) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    const uint64_t rows = __ballot((int)(threadIdx.x & 63) < n && id == a);
    left &= ~rows;
    f(a, (uint32_t)rows);
  }
}

__device__ __forceinline__ int id_of(const AdaptProb& p, int row) {
  if (row >= p.M) return -1;
  const int a = p.ids[row];
  return (unsigned)a < (unsigned)p.count ? a : -1;
}

// Eight of a row's alpha T, its shares of k added in order, and as three bf16 numbers, the
// nearest and twice the nearest to what is left: 24 bits, which is all of it (two would be off
// by 2^-17 of the adapter's part, more than the fp32 sums of the second product).  The
// first two are finite: past the largest, and for an infinity or a NaN, the last says the
// rest.
struct Parts {
  u32x4 part[3];
};
__device__ __forceinline__ Parts parts_of(const AdaptProb& p, int row, int at, float alpha) {
  const f32x4* t = (const f32x4*)(p.T + (size_t)row * p.rank + at);
  f32x4 a = t[0], b = t[1];
  for (int s = 1; s < p.splits; ++s) {
    t = (const f32x4*)((const float*)t + (size_t)p.M * p.rank);
    a += t[0];
    b += t[1];
  }
  a *= alpha;
  b *= alpha;
  Parts v;
  constexpr float most = 0x1.FEp127f;  // of bf16
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = i < 2 ? a[2 * i] : b[2 * i - 4], y = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
    v.part[0][i] = pack2(__builtin_amdgcn_fmed3f(x, -most, most), __builtin_amdgcn_fmed3f(y, -most, most));
    const float x1 = x - bf_low(v.part[0][i]), y1 = y - bf_high(v.part[0][i]);
    v.part[1][i] = pack2(__builtin_amdgcn_fmed3f(x1, -most, most), __builtin_amdgcn_fmed3f(y1, -most, most));
    v.part[2][i] = pack2(x1 - bf_low(v.part[1][i]), y1 - bf_high(v.part[1][i]));
  }
  return v;
}

__device__ __forceinline__ f32x4 mma16(const u32x4& a, const u32x4& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

}  // namespace

// ------------------------------------------------------------ first launch --
// A load of a matrix operand straight into its registers gives neighbouring lanes
// neighbouring rows: 64 requests of 16 bytes, 16 bytes a cycle and CU.  Loads whose
// neighbouring lanes have neighbouring bytes reach five times that.  So operands come
// through LDS, or were laid out in the order of the lanes before.
// Workgroups of three kinds.
// The first p.wdown: parts of X down_a^T for 32 rows and one share of k, which the
// waves divide.  Each has a ring of its own in LDS, filled two k-steps of 32 ahead: 64
// bytes of a row side by side, their four 16-byte chunks at chunk ^ (row / 2 % 4), so that
// 16 rows of an operand's read have no bank twice (at chunk ^ (row / 4 % 4) each read took
// twice as long).  The waves' sums are added in LDS in order.  slots workgroups have the same rows and share and take the rows' adapters in
// turn.  A row takes the sums of its own adapter only; in place of another adapter's rows
// the first of its own is read.  T[share][row][rank], fp32, is added up (in order) and
// scaled where it is used.
// The next p.wrows, for the product of few rows: X in blocks of 16 rows x 128 k, in the
// order in which that product's lanes take them (k past K: zero).
// The rest, for the product of many rows: the weights as bf16 in blocks of 16 rows x 32
// k, laid out as the ring is; block b of row group n is the 1 KB at (n K / 32 + b) KB.
// Bound by memory for the weights (4096 x 4096 from 4 bits: 42 MB) and by the rows' loads
// beside them: with 4096 rows of five adapters of rank 32 17 us; 999 rows of 16 adapters of
// rank 64 (6144 x 2048, 8 bits) 18 us; 64 rows of 48 adapters of rank 16 6 us.
#define AD_W 4
template <int RT>
struct Down {  // rank <= 16 RT
  static constexpr int STAGE = (2 + RT) * 1024, NS = 3, RED = AD_W * 2 * RT * 1024, RING = AD_W * NS * STAGE;
  static constexpr int LDS = RED > RING ? RED : RING;
};
template <int BITS, int RT>
__global__ __launch_bounds__(64 * AD_W) void k_adapt_down(const AdaptProb p) {
  typedef Down<RT> D;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[D::LDS];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int steps = p.K >> 5;
  if ((int)blockIdx.x >= p.wdown) {
    int i = blockIdx.x - p.wdown;
    u32x4* const mine = (u32x4*)lds + 256 * w;
    if (i < p.wrows) {  // a wave: a block
      const int blocks = (steps + 3) / 4, per = (blocks + AD_W - 1) / AD_W;
      const int n16 = i / per, t = (i % per) * AD_W + w;
      if (t >= blocks) return;
      const int k = 128 * t + 8 * (lane & 15), r4 = lane >> 4;  // four rows a load
      u32x4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[q] = u32x4{0u, 0u, 0u, 0u};
        if (k < p.K) v[q] = *(const u32x4*)(p.X + (size_t)min(16 * n16 + 4 * q + r4, p.M - 1) * p.ldx + k);
      }
      // the lane's 16-byte chunk 4 c + u of row j is lane 16 c + j's in product u
#pragma unroll
      for (int q = 0; q < 4; ++q) mine[64 * (lane & 3) + 16 * (lane >> 2 & 3) + 4 * q + r4] = v[q];
      u32x4* out = (u32x4*)p.XB + ((size_t)n16 * blocks + t) * 256 + lane;
#pragma unroll
      for (int u = 0; u < 4; ++u) out[64 * u] = mine[64 * u + lane];
      return;
    }
    i -= p.wrows;  // a wave: four blocks; a lane unpacks 32 codes
    const int per = (steps + 4 * AD_W - 1) / (4 * AD_W), n16 = i / per, s0 = (i % per) * 4 * AD_W + 4 * w;
    if (s0 >= steps) return;
    const int r = lane >> 2, c = lane & 3, n = min(16 * n16 + r, p.N - 1), st = min(s0 + c, steps - 1);
    gu32* codes = (gu32*)(p.P + ((size_t)n * steps + st) * BITS);
    gfloat* gs = (gfloat*)(p.S + (size_t)n * p.G);
    gu8* gz = (gu8*)(p.Z + (size_t)n * p.G);
    Words<BITS> cw;
#pragma unroll
    for (int e = 0; e < BITS; ++e) cw.w[e] = codes[e];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int g = (32 * st + 8 * u) >> p.gshift;
      mine[64 * c + 4 * r + (u ^ (r >> 1 & 3))] = weights8<BITS>(cw, u, gs[g], (float)gz[g]);
    }
    u32x4* out = (u32x4*)(p.W + ((size_t)n16 * steps + s0) * 512) + lane;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (s0 + u < steps) out[64 * u] = mine[64 * u + lane];
    return;
  }
  const int slot = blockIdx.x % (unsigned)p.slots, i0 = blockIdx.x / (unsigned)p.slots;
  const int split = i0 % p.splits, m0 = i0 / p.splits * 32;
  const int parts = p.splits * AD_W, part = split * AD_W + w;
  const int b0 = (int)((long long)steps * part / parts), b1 = (int)((long long)steps * (part + 1) / parts);
  float* T = p.T + ((size_t)split * p.M + m0) * p.rank;
  uint8_t* const ring = lds + w * D::NS * D::STAGE;
  const int lr = lane >> 2, lc = 8 * ((lane & 3) ^ (lane >> 3 & 3));  // a copy's row and k
  const int j = lane & 15, c = lane >> 4, at = j * 64 + ((c ^ (j >> 1 & 3)) << 4);
  int count = 0;
  each_adapter(id_of(p, m0 + (lane & 31)), 32, [&](int a, uint32_t rows) {
    if (count++ % p.slots != slot) return;
    const int first = __builtin_ctz(rows);
    const uint16_t *x[2], *d[RT];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int r = 16 * m + lr;
      x[m] = p.X + (size_t)(m0 + (rows >> r & 1 ? r : first)) * p.ldx + lc;
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) d[t] = p.down + ((size_t)a * p.rank + min(16 * t + lr, p.rank - 1)) * p.K + lc;
    auto issue = [&](int s, int stage) {
      uint8_t* to = ring + stage * D::STAGE;
#pragma unroll
      for (int m = 0; m < 2; ++m)
        __builtin_amdgcn_global_load_lds((const void*)(x[m] + 32 * s), (lds_void*)(to + 1024 * m), 16, 0, 0);
#pragma unroll
      for (int t = 0; t < RT; ++t)
        __builtin_amdgcn_global_load_lds((const void*)(d[t] + 32 * s), (lds_void*)(to + 1024 * (2 + t)), 16, 0, 0);
    };
    f32x4 acc[2][RT];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int t = 0; t < RT; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (b0 < b1) {
      issue(b0, 0);
      issue(min(b0 + 1, b1 - 1), 1);
      int stage = 0;
#pragma unroll 1
      for (int s = b0; s < b1; ++s) {
        // past the last step the copies repeat it, into stages that no one reads again
        issue(min(s + 2, b1 - 1), stage >= 1 ? stage - 1 : 2);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(VmWait<2 * (2 + RT)>::value);  // step s has landed
        __builtin_amdgcn_sched_barrier(0);
        const uint8_t* from = ring + stage * D::STAGE + at;
        const u32x4 x0 = *(const u32x4*)from, x1 = *(const u32x4*)(from + 1024);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const u32x4 b = *(const u32x4*)(from + 1024 * (2 + t));
          acc[0][t] = mma16(x0, b, acc[0][t]);
          acc[1][t] = mma16(x1, b, acc[1][t]);
        }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0x3F | 3 << 14 | 7 << 4);  // its reads are back: lgkmcnt 0
        __builtin_amdgcn_sched_barrier(0);
        stage = stage == 2 ? 0 : stage + 1;
      }
      __builtin_amdgcn_s_waitcnt(VmWait<0>::value);
    }
    __syncthreads();
    f32x4(*red)[2 * RT][64] = (f32x4(*)[2 * RT][64])lds;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int t = 0; t < RT; ++t) red[w][m * RT + t][lane] = acc[m][t];
    __syncthreads();
    for (int t = w; t < 2 * RT; t += AD_W) {
      f32x4 z = red[0][t][lane];
#pragma unroll
      for (int q = 1; q < AD_W; ++q) z += red[q][t][lane];
      const int col = 16 * (t % RT) + j;
      // rows 4 c + r, column j of the 16 ranks
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * (t / RT) + 4 * c + r;
        if ((rows >> row & 1) && col < p.rank) T[row * p.rank + col] = z[r];
      }
    }
    __syncthreads();
  });
}

// ------------------------------------------------------- product, few rows --
// 16 RB rows by 16 CB outputs a workgroup, k split among its waves; each code is
// unpacked once for all the rows.  A lane takes 32 neighbouring codes of a row at a time,
// which are its k in four products; X lies in that order.  The (16 rows, adapter) pairs are
// shared out among the waves, too; all sums are added in LDS in order.  Bound by waits on
// X, which every workgroup reads (64 rows of 4096 x 4096: 134 MB from the L2s): 64 rows at
// 4 bits with 48 adapters of rank 16 15.7 us; one row of 2048 x 6144 at 3 bits 8.5 us.
template <int BITS, int RB, int CB, int NW>
__global__ __launch_bounds__(64 * NW) void k_adapt_rows(const AdaptProb p) {
  constexpr int PAIRS = 16 * RB, MINE = (PAIRS + NW - 1) / NW, AT = MINE < 8 ? MINE : 8;
  constexpr int SUMS = NW * RB * CB * 1024, ROWS = 16 * RB * (6 * 128 + 16);
  static_assert(NW % RB == 0, "a wave's pairs are of one group of rows");
  __shared__ __attribute__((aligned(16))) uint8_t lds[SUMS > ROWS ? SUMS : ROWS];  // the rows' T, then the waves' sums
  __shared__ int pa[PAIRS];
  __shared__ uint32_t pm[PAIRS];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int j = lane & 15, c = lane >> 4;
  const int n0 = blockIdx.x * 16 * CB, m0 = blockIdx.y * 16 * RB;
  const int steps = p.K >> 5, blocks = (steps + 3) / 4;
  gu32* codes[CB];
  gfloat* gs[CB];
  gu8* gz[CB];
  int nrow[CB];
#pragma unroll
  for (int n = 0; n < CB; ++n) {
    nrow[n] = min(n0 + 16 * n + j, p.N - 1);
    codes[n] = (gu32*)(p.P + (size_t)nrow[n] * (steps * BITS));
    gs[n] = (gfloat*)(p.S + (size_t)nrow[n] * p.G);
    gz[n] = (gu8*)(p.Z + (size_t)nrow[n] * p.G);
  }
  const u32x4* x[RB];
#pragma unroll
  for (int m = 0; m < RB; ++m)
    x[m] = (const u32x4*)p.XB + (size_t)min((m0 >> 4) + m, (p.M - 1) >> 4) * blocks * 256 + lane;
  f32x4 acc[RB][CB];
#pragma unroll
  for (int m = 0; m < RB; ++m)
#pragma unroll
    for (int n = 0; n < CB; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  // blocks of 128 k, the next one's loads in flight beside the products of one
  const int b0 = blocks * w / NW, b1 = blocks * (w + 1) / NW;
  struct Block {
    u32x4 x[4][RB];
    Words<BITS> q[CB];
    float s[CB];
    uint32_t z[CB];
  };
  auto load = [&](Block& k, int i) {
    const int s = min(4 * i + c, steps - 1);
#pragma unroll
    for (int n = 0; n < CB; ++n) {
#pragma unroll
      for (int e = 0; e < BITS; ++e) k.q[n].w[e] = codes[n][(size_t)s * BITS + e];
      k.s[n] = gs[n][(32 * s) >> p.gshift];
      k.z[n] = gz[n][(32 * s) >> p.gshift];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int m = 0; m < RB; ++m) k.x[u][m] = x[m][(size_t)i * 256 + 64 * u];
  };
  auto add = [&](const Block& k, int i) {
    const bool whole = 4 * i + 4 <= steps, on = 4 * i + c < steps;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int n = 0; n < CB; ++n) {
        float s = k.s[n];
        uint32_t z = k.z[n];
        if (p.gshift < 5) {  // uniform: grids of 8 or 16 codes
          const int g = (32 * min(4 * i + c, steps - 1) + 8 * u) >> p.gshift;
          s = gs[n][g];
          z = gz[n][g];
        }
        u32x4 b = weights8<BITS>(k.q[n], u, s, (float)z);
        if (!whole && !on) b = u32x4{0u, 0u, 0u, 0u};  // past the last k, where X is zero, too
#pragma unroll
        for (int m = 0; m < RB; ++m) acc[m][n] = mma16(k.x[u][m], b, acc[m][n]);
      }
  };
  Block even, odd;
  const int per = p.rank >> 3, pitch = 6 * p.rank + 16;  // chunks of eight: of T's first numbers, of the next, of the last
  for (int i = tid; i < PAIRS; i += 64 * NW) pa[i] = -1;
  for (int i = tid; i < 16 * RB * per; i += 64 * NW) {
    const int row = i / per, q = i % per, a = id_of(p, m0 + row);
    if (a < 0) continue;
    const Parts v = parts_of(p, m0 + row, 8 * q, p.alpha ? p.alpha[a] : 1.f);
#pragma unroll
    for (int e = 0; e < 3; ++e) *(u32x4*)(lds + row * pitch + 16 * (e * per + q)) = v.part[e];
  }
  if (b0 < b1) load(even, b0);  // on its way beside the adapters' loads
  __syncthreads();
  if (p.rank > 0)
    for (int rb = w; rb < RB; rb += NW) {
      int k = 0;
      each_adapter(id_of(p, m0 + 16 * rb + j), 16, [&](int a, uint32_t rows) {
        if (lane == 0) {
          pa[k * RB + rb] = a;
          pm[k * RB + rb] = rows;
        }
        ++k;
      });
    }
  __syncthreads();
  for (int i0 = w; i0 < PAIRS; i0 += NW * AT) {
    int pair[AT], some = -1;
#pragma unroll
    for (int k = 0; k < AT; ++k) {
      pair[k] = i0 + NW * k < PAIRS ? __builtin_amdgcn_readfirstlane(pa[i0 + NW * k]) : -1;
      some = max(some, pair[k]);
    }
    if (some < 0) break;  // a group's pairs come first
    f32x4 z[AT][CB];
#pragma unroll
    for (int k = 0; k < AT; ++k)
#pragma unroll
      for (int n = 0; n < CB; ++n) z[k][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int q0 = 0; q0 < per; q0 += 4) {
      const int q = min(q0 + c, per - 1);
      const bool there = q0 + c < per;
      const u32x4 none = {0u, 0u, 0u, 0u};
      // all loads without a branch between them: a pair that is not there reads adapter 0's
      u32x4 b[AT][CB];
#pragma unroll
      for (int k = 0; k < AT; ++k)
#pragma unroll
        for (int n = 0; n < CB; ++n)
          b[k][n] = *(const gu32x4*)(p.up + ((size_t)max(pair[k], 0) * p.N + nrow[n]) * p.rank + 8 * q);
#pragma unroll
      for (int k = 0; k < AT; ++k)
#pragma unroll
        for (int n = 0; n < CB; ++n) b[k][n] = there ? b[k][n] : none;
#pragma unroll
      for (int e = 0; e < 3; ++e) {
        u32x4 t = *(const u32x4*)(lds + (16 * (w % RB) + j) * pitch + 16 * (e * per + q));
        t = there ? t : none;
#pragma unroll
        for (int k = 0; k < AT; ++k)
#pragma unroll
          for (int n = 0; n < CB; ++n) z[k][n] = mma16(t, b[k][n], z[k][n]);
      }
    }
#pragma unroll
    for (int k = 0; k < AT; ++k) {
      const int i = i0 + NW * k;
      if (pair[k] < 0) continue;
      const uint32_t rows = pm[i];
#pragma unroll
      for (int m = 0; m < RB; ++m)
        if (i % RB == m) {
#pragma unroll
          for (int n = 0; n < CB; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (rows >> (4 * c + r) & 1) acc[m][n][r] += z[k][n][r];
        }
    }
  }
  if (b0 < b1) {
    int i = b0;
#pragma unroll 1
    for (;; i += 2) {
      load(odd, min(i + 1, b1 - 1));
      add(even, i);
      if (i + 2 >= b1) break;  // no load that the barrier below would wait for
      load(even, i + 2);
      add(odd, i + 1);
    }
    if (i + 1 < b1) add(odd, i + 1);
  }
  __syncthreads();  // no wave reads T any more
  f32x4(*red)[RB * CB][64] = (f32x4(*)[RB * CB][64])lds;
#pragma unroll
  for (int m = 0; m < RB; ++m)
#pragma unroll
    for (int n = 0; n < CB; ++n) red[w][m * CB + n][lane] = acc[m][n];
  __syncthreads();
  for (int t = w; t < RB * CB; t += NW) {
    f32x4 y = red[0][t][lane];
#pragma unroll
    for (int q = 1; q < NW; ++q) y += red[q][t][lane];
    const int col = n0 + 16 * (t % CB) + j;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = m0 + 16 * (t / CB) + 4 * c + r;
      if (row < p.M && col < p.N) p.Y[(size_t)row * p.ldy + col] = y[r];
    }
  }
}

// ------------------------------------------------------ product, many rows --
// BM x BN of Y a workgroup, WM x WN a wave, on 16x16x32 MFMA (4096 x 4096 x 4096, the
// product alone: 110 us, on 32x32x16 117; the power limit bounds both, 92 us on zeros); KH
// k-steps of 32 a stage of LDS, in a ring of NS stages filled NS - 1 ahead.  One barrier
// a stage.  The fragments of a step are read beside the products of the one before.
// With 4096 rows of five adapters of rank 32 114 to 122 us by card, 1.2 PFLOP/s; 999 rows of
// 16 adapters of rank 64, 6144 x 2048, 40 us.
// SPLIT: parts workgroups have a tile, a share of k and of the adapters' part each; the one
// that is done last adds all sums in order and stores them.
template <int BM, int BN, int WM, int WN, int KH, int NS, bool SPLIT>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, 1) void k_adapt_tile(const AdaptProb p) {
  constexpr int NW = (BM / WM) * (BN / WN), AI = WM / 16, BJ = WN / 16;
  constexpr int NA = BM / 16 / NW, NB = BN / 16 / NW;  // 1 KB copies of a wave and k-step
  constexpr int HALF = (BM + BN) * 64, STAGE = KH * HALF, PER = KH * (NA + NB);
  // rows of products before a stage's barrier; those behind it cover the next stage's reads
  constexpr int BEFORE = AI >= 4 ? AI / 2 : 0;
  constexpr int PITCH = 3 * 8 * 16 + 16, RING = NS * STAGE, ROWS = BM * PITCH;
  static_assert(NA * NW * 16 == BM && NB * NW * 16 == BN, "whole copies");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[RING > ROWS ? RING : ROWS];  // the ring, then the rows' T
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tm = (p.M + BM - 1) / BM, tn = (p.N + BN - 1) / BN, nt = tm * tn;
  // Consecutive workgroups go to the eight XCDs in turn: each gets a run of tiles,
  // four rows of tiles by as many columns as it takes, so that its L2 holds few of either
  const int parts = SPLIT ? p.parts : 1, share = SPLIT ? blockIdx.x / (unsigned)nt : 0, bid = blockIdx.x - share * nt;
  const int xcd = bid & 7;
  const int t = xcd * (nt >> 3) + min(xcd, nt & 7) + (bid >> 3);
  const int band = t / (4 * tn), rows = min(4, tm - 4 * band), in = t - 4 * band * tn;
  const int m0 = (4 * band + in % rows) * BM, n0 = (in / rows) * BN;
  // stages[first] .. stages - 1 are this workgroup's
  const int steps = p.K >> 5, all = (steps + KH - 1) / KH;
  const int first = all * share / parts, stages = all * (share + 1) / parts;

  const uint16_t* ga[NA];
  const uint16_t* gb[NB];
#pragma unroll
  for (int q = 0; q < NA; ++q) {
    const int row = min(m0 + 16 * (NW * q + w) + (lane >> 2), p.M - 1);
    ga[q] = p.X + (size_t)row * p.ldx + 8 * ((lane & 3) ^ (lane >> 3 & 3));
  }
#pragma unroll
  for (int q = 0; q < NB; ++q) {
    const int g16 = min((n0 >> 4) + NW * q + w, (p.N - 1) >> 4);
    gb[q] = p.W + (size_t)g16 * steps * 512 + 8 * lane;
  }
  auto issue = [&](int stage, int slot) {
#pragma unroll
    for (int h = 0; h < KH; ++h) {
      const int step = min(stage * KH + h, steps - 1);
      uint8_t* base = lds + slot * STAGE + h * HALF;
#pragma unroll
      for (int q = 0; q < NA; ++q)
        __builtin_amdgcn_global_load_lds((const void*)(ga[q] + step * 32), (lds_void*)(base + (NW * q + w) * 1024), 16, 0, 0);
#pragma unroll
      for (int q = 0; q < NB; ++q)
        __builtin_amdgcn_global_load_lds((const void*)(gb[q] + (size_t)step * 512),
                                         (lds_void*)(base + BM * 64 + (NW * q + w) * 1024), 16, 0, 0);
    }
  };
  const int j16 = lane & 15, c4 = lane >> 4;  // an operand's row and its part of k
  const int wm0 = WM * (w / (BN / WN)), wn0 = WN * (w % (BN / WN));
  const int at = j16 * 64 + ((c4 ^ (j16 >> 1 & 3)) << 4);
  auto rd = [&](int slot, int h, bf16x8* fa, bf16x8* fb) {
    const uint8_t* from = lds + slot * STAGE + h * HALF + at;
#pragma unroll
    for (int i = 0; i < AI; ++i) fa[i] = *(const bf16x8*)(from + wm0 * 64 + 1024 * i);
#pragma unroll
    for (int j = 0; j < BJ; ++j) fb[j] = *(const bf16x8*)(from + (BM + wn0) * 64 + 1024 * j);
  };
  f32x4 acc[AI][BJ];
#pragma unroll
  for (int i = 0; i < AI; ++i)
#pragma unroll
    for (int j = 0; j < BJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto mma = [&](const bf16x8* fa, const bf16x8* fb, int i0, int i1) {
#pragma unroll
    for (int i = 0; i < AI; ++i)
      if (i >= i0 && i < i1) {
#pragma unroll
        for (int j = 0; j < BJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
      }
  };

  if (first < stages) {
#pragma unroll
    for (int q = 0; q < NS - 1; ++q) issue(min(first + q, stages - 1), q);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(VmWait<(NS - 2) * PER>::value);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    bf16x8 fa[2][AI], fb[2][BJ];
    rd(0, 0, fa[0], fb[0]);
    int slot = 0;
    // stage s, whose first fragments are in buffer f; ahead: stages that may still be on
    // their way behind its barrier
    auto stage = [&](int s, int f, auto more, auto ahead) __attribute__((always_inline)) {
      const int before = slot == 0 ? NS - 1 : slot - 1, next = slot == NS - 1 ? 0 : slot + 1;
      // into the stage of s - 1, which all waves have read; past the last stage the
      // copies repeat it, into stages that no one reads again
      if (decltype(more)::value) issue(min(s + NS - 1, stages - 1), before);
      __builtin_amdgcn_sched_barrier(0);
      const bool whole = KH == 1 || KH * s + KH <= steps;  // uniform; else the second k-step is past K
#pragma unroll
      for (int h = 0; h < KH - 1; ++h) {
        rd(slot, h + 1, fa[(f + h + 1) & 1], fb[(f + h + 1) & 1]);
        mma(fa[(f + h) & 1], fb[(f + h) & 1], 0, AI);
      }
      const int e = (f + KH - 1) & 1;
      if (whole) mma(fa[e], fb[e], 0, BEFORE);
      __builtin_amdgcn_sched_barrier(0);
      // stage s + 1 has landed; this wave's reads are back
      __builtin_amdgcn_s_waitcnt(VmWait<decltype(ahead)::value * PER>::value & ~(15 << 8));
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      // (behind the last stage: read, not used)
      rd(next, 0, fa[e ^ 1], fb[e ^ 1]);
      if (whole) mma(fa[e], fb[e], BEFORE, AI);
      slot = next;
    };
    std::integral_constant<int, NS - 2> most;
    std::integral_constant<int, 1> one;
    std::integral_constant<int, 0> none;
    std::true_type yes;
    std::false_type no;
    if constexpr (KH == 1) {
      for (int s = first; s < stages; s += 2) {
        stage(s, 0, yes, most);
        if (s + 1 < stages) stage(s + 1, 1, yes, most);
      }
    } else {
      static_assert(KH == 2 && NS == 4, "two steps a stage");
      // the last three without copies behind them (a branch in the stage instead: 44.9 us
      // for 999 rows, 41.5 with none)
      int s = first;
      for (; s + 3 < stages; ++s) stage(s, 0, yes, most);
      if (s + 2 < stages) stage(s++, 0, no, one);
      if (s + 1 < stages) stage(s++, 0, no, none);
      stage(s, 0, no, none);
    }
    __builtin_amdgcn_s_waitcnt(VmWait<0>::value);  // no copy into LDS outlives the group
  }

  // The adapters' part, eight chunks of eight ranks at a time.  The rows' T goes to LDS as bf16
  // (the ring is free), 16 bytes more than a row so that the rows of a read fall on different
  // banks.  For one adapter of the wave's rows after the other its half is read once
  // for all of them; the products are from zero on and added to its own rows only: what it
  // holds reaches no other's.  Of several workgroups each takes some of the chunks.
  if (p.rank > 0) {
    const int per = p.rank >> 3;
    const int qa = per * share / parts, qb = per * (share + 1) / parts;  // this workgroup's chunks
    constexpr int IH = (WM + 63) / 64;
    int ids[IH];
#pragma unroll
    for (int h = 0; h < IH; ++h) ids[h] = 64 * h + lane < WM ? id_of(p, m0 + wm0 + 64 * h + lane) : -1;
#pragma unroll 1
    for (int q1 = qa; q1 < qb; q1 += 8) {
      const int nq = min(8, qb - q1);
      __syncthreads();
      for (int i = threadIdx.x; i < BM * nq; i += 64 * NW) {
        const int row = i / nq, q = i % nq, a = id_of(p, m0 + row);
        if (a < 0) continue;
        const Parts v = parts_of(p, m0 + row, 8 * (q1 + q), p.alpha ? p.alpha[a] : 1.f);
#pragma unroll
        for (int e = 0; e < 3; ++e) *(u32x4*)(lds + row * PITCH + 16 * (8 * e + q)) = v.part[e];
      }
      __syncthreads();
      uint64_t open[IH];
#pragma unroll
      for (int h = 0; h < IH; ++h) open[h] = __ballot(ids[h] >= 0);
#pragma unroll 1
      for (;;) {
        int a = -1;
#pragma unroll
        for (int h = 0; h < IH; ++h)
          if (a < 0 && open[h]) a = __builtin_amdgcn_readlane(ids[h], __builtin_ctzll(open[h]));
        if (a < 0) break;
        uint64_t mine[IH];
#pragma unroll
        for (int h = 0; h < IH; ++h) {
          mine[h] = __ballot(ids[h] == a);
          open[h] &= ~mine[h];
        }
        const u32x4 none = {0u, 0u, 0u, 0u};
        // the loads for all columns are in flight together
        u32x4 b[BJ][2];
#pragma unroll
        for (int j = 0; j < BJ; ++j) {
          const int col = min(n0 + wn0 + 16 * j + j16, p.N - 1);
          const uint16_t* up = p.up + ((size_t)a * p.N + col) * p.rank + 8 * q1;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            b[j][g] = none;
            if (4 * g + c4 < nq) b[j][g] = *(const u32x4*)(up + 8 * (4 * g + c4));
          }
        }
#pragma unroll
        for (int i = 0; i < AI; ++i) {
          const uint32_t rows = (uint32_t)(mine[i / 4] >> (16 * (i % 4))) & 0xFFFFu;
          if (!rows) continue;  // uniform
          const uint8_t* t = lds + (wm0 + 16 * i + j16) * PITCH + 16 * c4;
          f32x4 z[BJ];
#pragma unroll
          for (int j = 0; j < BJ; ++j) z[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int g = 0; g < 2; ++g)
            if (4 * g < nq) {  // uniform
#pragma unroll
              for (int e = 0; e < 3; ++e) {
                u32x4 v = *(const u32x4*)(t + 16 * (8 * e + 4 * g));
                v = 4 * g + c4 < nq ? v : none;
#pragma unroll
                for (int j = 0; j < BJ; ++j) z[j] = mma16(v, b[j][g], z[j]);
              }
            }
#pragma unroll
          for (int j = 0; j < BJ; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (rows >> (4 * c4 + r) & 1) acc[i][j][r] += z[j][r];
        }
      }
    }
  }

  if (SPLIT && parts > 1) {
    // past the L2, which other XCDs do not share
    constexpr size_t NEXT = 64 * NW, SIZE = (size_t)AI * BJ * 2 * NEXT;  // the threads' first 8 bytes, their second ones, ..
    uint64_t* const sums = (uint64_t*)p.part + t * SIZE + threadIdx.x;
    uint64_t* const to = sums + (size_t)share * nt * SIZE;
#pragma unroll
    for (int i = 0; i < AI; ++i)
#pragma unroll
      for (int j = 0; j < BJ; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          __hip_atomic_store(to + ((i * BJ + j) * 2 + e) * NEXT,
                             __builtin_bit_cast(uint64_t, f32x2{acc[i][j][2 * e], acc[i][j][2 * e + 1]}),
                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // they are in memory before the count says so
    __syncthreads();
    if (threadIdx.x == 0) {
      const int last = __hip_atomic_fetch_add(p.done + t, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
      if (last) __hip_atomic_store(p.done + t, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      *(int*)lds = last;
    }
    __syncthreads();
    if (!*(const int*)lds) return;
    constexpr int G = AI * BJ <= 4 ? 4 : 2;  // shares whose loads are in flight together
    f32x4 z[AI][BJ];
#pragma unroll
    for (int i = 0; i < AI; ++i)
#pragma unroll
      for (int j = 0; j < BJ; ++j) z[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int s0 = 0; s0 < parts; s0 += G) {
      uint64_t v[G][AI][BJ][2];
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (s0 + g < parts && s0 + g != share) {
          const uint64_t* const get = sums + (size_t)(s0 + g) * nt * SIZE;
#pragma unroll
          for (int i = 0; i < AI; ++i)
#pragma unroll
            for (int j = 0; j < BJ; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                v[g][i][j][e] = __hip_atomic_load(get + ((i * BJ + j) * 2 + e) * NEXT, __ATOMIC_RELAXED,
                                                  __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (s0 + g < parts) {
          const bool own = s0 + g == share;
#pragma unroll
          for (int i = 0; i < AI; ++i)
#pragma unroll
            for (int j = 0; j < BJ; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const f32x2 x = __builtin_bit_cast(f32x2, v[g][i][j][e]);
                z[i][j][2 * e] += own ? acc[i][j][2 * e] : x.x;
                z[i][j][2 * e + 1] += own ? acc[i][j][2 * e + 1] : x.y;
              }
        }
    }
#pragma unroll
    for (int i = 0; i < AI; ++i)
#pragma unroll
      for (int j = 0; j < BJ; ++j) acc[i][j] = z[i][j];
  }
#pragma unroll
  for (int i = 0; i < AI; ++i)
#pragma unroll
    for (int j = 0; j < BJ; ++j) {
      const int col = n0 + wn0 + 16 * j + j16;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = m0 + wm0 + 16 * i + 4 * c4 + r;
        if (row < p.M && col < p.N) p.Y[(size_t)row * p.ldy + col] = acc[i][j][r];
      }
    }
}

// ------------------------------------------------------------- launchers --
namespace {
template <int BITS, int RT>
void down_rank(const AdaptProb& p, hipStream_t st) {
  AdaptProb q = p;
  const int per = ((p.K >> 5) + 4 * AD_W - 1) / (4 * AD_W);  // workgroups of 16 rows of X or of the weights
  q.wdown = p.rank ? (p.M + 31) / 32 * p.splits * p.slots : 0;
  q.wrows = p.shape ? 0 : (p.M + 15) / 16 * per;
  const int n = q.wdown + q.wrows + (p.shape ? (p.N + 15) / 16 * per : 0);
  if (n) hipLaunchKernelGGL((k_adapt_down<BITS, RT>), dim3((unsigned)n), dim3(64 * AD_W), 0, st, q);
}
template <int BITS>
void down_bits(const AdaptProb& p, hipStream_t st) {
  if (p.rank <= 16)
    down_rank<BITS, 1>(p, st);
  else if (p.rank <= 32)
    down_rank<BITS, 2>(p, st);
  else if (p.rank <= 64)
    down_rank<BITS, 4>(p, st);
  else
    down_rank<BITS, 8>(p, st);
}
template <int BM, int BN, int WM, int WN, int KH, int NS, bool SPLIT = false>
hipError_t tile_shape(const AdaptProb& p, hipStream_t st) {
  const unsigned tiles = ((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
  hipLaunchKernelGGL((k_adapt_tile<BM, BN, WM, WN, KH, NS, SPLIT>), dim3(SPLIT ? p.parts * tiles : tiles),
                     dim3((BM / WM) * (BN / WN) * 64), 0, st, p);
  return hipGetLastError();
}
template <int BITS, int RB, int CB, int NW>
void rows_shape(const AdaptProb& p, hipStream_t st) {
  const dim3 grid((unsigned)((p.N + 16 * CB - 1) / (16 * CB)), (unsigned)((p.M + 16 * RB - 1) / (16 * RB)));
  hipLaunchKernelGGL((k_adapt_rows<BITS, RB, CB, NW>), grid, dim3(64 * NW), 0, st, p);
}
template <int BITS>
hipError_t product_bits(const AdaptProb& p, hipStream_t st) {
  if (!p.shape) {
    // 64 rows of 4096 outputs (256 workgroups) 21 us, by 32 outputs 25; 128 rows 38 and 26; 89
    // rows of 715 16 and 24.  (Up to 64 rows of more outputs: by 16 as well, 32 not measured.)
    if (p.M <= 16)
      rows_shape<BITS, 1, 1, 8>(p, st);
    else if (p.M <= 32)
      rows_shape<BITS, 2, 1, 8>(p, st);
    else if (p.M <= 64)
      rows_shape<BITS, 4, 1, 8>(p, st);
    else if (p.N <= 2048)
      rows_shape<BITS, 4, 1, 8>(p, st);
    else
      rows_shape<BITS, 4, 2, 8>(p, st);
    return hipGetLastError();
  }
  switch (p.shape) {
    case 1: return tile_shape<64, 64, 32, 32, 2, 4, true>(p, st);
    case 2: return tile_shape<128, 128, 64, 32, 2, 4, true>(p, st);
    case 3: return tile_shape<128, 128, 64, 32, 2, 4>(p, st);
    case 4: return tile_shape<128, 256, 64, 64, 1, 6>(p, st);
    default: return tile_shape<256, 256, 128, 64, 1, 4>(p, st);
  }
}
}  // namespace

hipError_t launch_adapt_down(const AdaptProb& p, int bits, hipStream_t st) {
  switch (bits) {
    case 2: down_bits<2>(p, st); break;
    case 3: down_bits<3>(p, st); break;
    case 4: down_bits<4>(p, st); break;
    default: down_bits<8>(p, st); break;
  }
  return hipGetLastError();
}

hipError_t launch_adapt_product(const AdaptProb& p, int bits, hipStream_t st) {
  switch (bits) {
    case 2: return product_bits<2>(p, st);
    case 3: return product_bits<3>(p, st);
    case 4: return product_bits<4>(p, st);
    default: return product_bits<8>(p, st);
  }
}
