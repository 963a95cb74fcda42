// Attention of drafted tokens over the quantised cache (gfx950).
#include "common.h"
#include "serve.h"

// One wave per (sequence, token, query head): 64 positions at a time, one per
// lane for the scores, then the lanes take dimensions for the weighted sum.
template <int BITS>
__global__ __launch_bounds__(64) void k_tree_attn(const AttnProb p) {
  __shared__ float qs[256], pr[64];
  __shared__ size_t row[64];
  const KvPool& c = p.c;
  const int lane = threadIdx.x, D = c.dim;
  const int hq = blockIdx.x % p.heads, h = hq / p.group;
  const int bt = blockIdx.x / p.heads, b = bt / p.tokens, t = bt % p.tokens;
  const uint16_t* q = p.q + b * p.qb + t * p.qt + hq * p.qh;
  for (int d = lane; d < D; d += 64) qs[d] = __builtin_bit_cast(float, (uint32_t)q[d] << 16);
  const int len = p.lengths[b];
  const long long cap = (long long)p.width << c.pshift;
  const int n = len < 0 ? 0 : (int)min((long long)len + p.tokens, cap);
  const int pm = (1 << c.pshift) - 1;
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < n; j0 += 64) {
    const int j = j0 + lane;
    bool see = j < n;
    if (see && j >= len)
      see = p.mask ? (p.mask[(size_t)bt * p.words + ((j - len) >> 5)] >> ((j - len) & 31)) & 1u : j - len <= t;
    float x = -INFINITY;
    size_t at = 0;
    if (see) {
      const int page = p.tables[(size_t)b * p.width + (j >> c.pshift)];
      see = (unsigned)page < (unsigned)c.pages;
      if (see) {
        at = (((size_t)page * c.heads + h) << c.pshift) + (j & pm);
        const uint8_t* k = c.kc + at * c.rb;
        const float z = (float)c.kz[at];
        float a = 0.f;
        for (int d = 0; d < D; ++d) {
          const int code = BITS == 8 ? k[d] : (k[d >> 1] >> (4 * (d & 1))) & 15;
          a += qs[d] * ((float)code - z);
        }
        x = a * c.ks[at] * p.scale;
      }
    }
    float mt = x;
    for (int o = 32; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor(mt, o));
    const float mn = fmaxf(m, mt);
    const float al = mn == -INFINITY ? 1.f : exp2f(m - mn);
    const float e = see ? exp2f(x - mn) : 0.f;
    l = l * al + e;
    m = mn;
    __syncthreads();
    pr[lane] = see ? e * c.vs[at] : 0.f;
    row[lane] = see ? at : (size_t)0;
    __syncthreads();
    for (int u = 0; u < 4; ++u) acc[u] *= al;
    for (int i = 0; i < 64; ++i) {
      const float w = pr[i];
      if (w == 0.f) continue;
      const size_t a = row[i];
      const float z = (float)c.vz[a];
      const uint8_t* vb = c.vc + ((a >> c.pshift) * c.rb << c.pshift) + (a & pm);
      for (int u = 0; u < 4; ++u) {
        const int d = lane + 64 * u;
        if (d >= D) continue;
        const int r = BITS == 8 || d < D / 2 ? d : d - D / 2;
        const int by = vb[(size_t)r << c.pshift];
        const int code = BITS == 8 ? by : (d < D / 2 ? by & 15 : by >> 4);
        acc[u] += w * ((float)code - z);
      }
    }
    __syncthreads();
  }
  for (int o = 32; o > 0; o >>= 1) l += __shfl_xor(l, o);
  uint16_t* out = p.o + b * p.ob + t * p.ot + hq * p.oh;
  for (int u = 0; u < 4; ++u) {
    const int d = lane + 64 * u;
    if (d < D) out[d] = __builtin_bit_cast(uint16_t, (__bf16)(l == 0.f ? 0.f : acc[u] / l));
  }
}

hipError_t launch_tree_attn(const AttnProb& p, int bits, hipStream_t st) {
  const dim3 grid((unsigned)((long long)p.seqs * p.tokens * p.heads));
  if (bits == 8)
    hipLaunchKernelGGL(k_tree_attn<8>, grid, dim3(64), 0, st, p);
  else
    hipLaunchKernelGGL(k_tree_attn<4>, grid, dim3(64), 0, st, p);
  return hipGetLastError();
}
