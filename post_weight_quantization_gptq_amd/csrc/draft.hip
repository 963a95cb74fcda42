// From a target model's logits to the next tokens (gfx950): probabilities at a
// temperature, and drafted tokens checked against them.
#include "common.h"
#include "serve.h"

#include <algorithm>

namespace {

// N values from any address of their type.
template <int N>
__device__ __forceinline__ void load_any(const float* p, float* o) {
  __builtin_memcpy(o, p, 4 * N);
}

}  // namespace

// ---------------------------------------------------------- probabilities --
// p_v = exp((l_v - max) / t) / sum, fp32, as powers of two of (l - max) log2(e) / t;
// t = 0: 1 at the first maximum.  A row with a NaN or +infinity (t > 0), or a
// temperature below 0 or not finite, is NaN; a row of -infinity alone is zero.
// A workgroup has a row, which stays in its registers from the load on: 4 C values a
// thread, as they came.  Rows that are longer (fp32 past 65536 values, bf16 past 131072) are
// read in such blocks twice, for the sum and for the result.
// Bound by HBM where there are rows for the CUs: 208 rows of 100003 bf16 values, 125 MB in
// 24.8 us, 5.0 TB/s (31.5 with the sum behind the largest value), of 65536 fp32 values 109 MB
// in 21.7 us; read twice, 208 rows of 100003 fp32 values 36 us, of 131072 46.5, of 200003 bf16
// values 52.  Five rows of 32768 fp32 values, one CU each, 7.4 us.
namespace {

template <class T>
struct Raw {  // four values of a row
  uint32_t w[sizeof(T)];
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(float, w[i]);
    else return __builtin_bit_cast(float, i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ Raw() {}
  // the first n of four, -infinity in place of the others
  __device__ __forceinline__ Raw(const T* v, int n) {
    T o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) o[i] = i < n ? v[i] : -INFINITY;
      else o[i] = i < n ? v[i] : 0xFF80;
    }
    __builtin_memcpy(w, o, sizeof(w));
  }
  // what was made of the values is made again from here on: kept, it would take the
  // registers that the row needs
  __device__ __forceinline__ void anew() {
#pragma unroll
    for (unsigned i = 0; i < sizeof(T); ++i) asm volatile("" : "+v"(w[i]));
  }
};

// The first lane's.
__device__ __forceinline__ float all_lanes(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}

template <int NT, class F>
__device__ __forceinline__ float over_all(float x, float* part, F&& f) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x = f(x, __shfl_xor(x, o));
  __syncthreads();  // part may still be read
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  // (a number a lane: all of them in every lane would take the registers that a row needs)
  x = part[threadIdx.x & (NT / 64 - 1)];
#pragma unroll
  for (int o = NT / 128; o > 0; o >>= 1) x = f(x, __shfl_xor(x, o));
  return x;
}

}  // namespace

// ONE: the row is a block; else it is read block after block, once for each use.
template <class T, int NT, int C, bool ONE>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(NT / 256, 4))) void k_probs(const ProbsProb p) {
  __shared__ float part[16], sums[16];
  const int tid = threadIdx.x, V = p.vocab;
  const int b = __builtin_amdgcn_readfirstlane(blockIdx.x / (unsigned)p.tokens);
  const int t = blockIdx.x - b * p.tokens;
  const T* x = (const T*)p.x + b * p.xs + t * p.xt;
  float* y = p.y + b * p.ys + t * p.yt;
  const float warm = p.warm ? p.warm[b] : 1.f;
  const bool greedy = warm == 0.f, fair = warm >= 0.f && warm <= 3.402823466e38f;
  // Logits are made smaller by a power of two first, half of them or about 1 / t: the
  // difference of two of any size is finite, and the factor below no smaller than log2(e) / 4.
  // It is held finite: where it would not be, all but the maximum vanishes.  The factor is two
  // numbers: one is off by up to 2^-24 of itself, which a value d below the largest has d / t
  // times.  The first is below the factor, so that the second is above 0: times -infinity it
  // must not be NaN.  What the first leaves of log2(e) is exact but for its own last bit.
  const int down = min(max((int)(__builtin_bit_cast(uint32_t, warm) >> 23 & 255) - 127, 1), 126);
  const float half = __builtin_bit_cast(float, (127 - down) << 23);
  constexpr float log2e = 1.44269502162933f, log2e_rest = 1.92596299112661e-8f, ln2 = 0.693147180559945f;
  const float nearest = fminf(log2e / (warm * half), 3.402823466e38f);
  const float c = all_lanes(__builtin_bit_cast(float, __builtin_bit_cast(int, nearest) - 1));
  const float rest = all_lanes(fmaxf((fmaf(-c, warm * half, log2e) + log2e_rest) * (c * ln2), 0x1p-100f));
  constexpr int ROW = 4 * NT, BLOCK = C * ROW;
  auto store = [&](const float* a, int v0, bool whole) {
    const int v = v0 + 4 * tid;
    if (whole) {
      __builtin_memcpy((y + v0) + 4u * threadIdx.x, a, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (v + i < V) y[v + i] = a[i];
    }
  };
  // whole chunks of a block, and the one that the row ends in
  Raw<T> r[C];
  T rag[4];
  // All loads of a block one after the other with no branch between them, so that the
  // first ones can be waited for alone; those past the row's end read its first chunk.
  auto load = [&](int v0) {
    const int whole = (V - v0) / ROW;
    if (whole > 0)
#pragma unroll
      for (int k = 0; k < C; ++k) {
        // (a base for all lanes and a 32-bit offset: an address a chunk would take two registers)
        __builtin_memcpy(&r[k], (x + (v0 + (k < whole ? k : 0) * ROW)) + 4u * threadIdx.x, sizeof(r[k]));
        if (k % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // in this order
      }
  };
  // before load(), and put together where it is used, so that no one waits for it
  auto load_rag = [&](int v0) {
    const int at = v0 + (V - v0) / ROW * ROW + 4 * tid;
#pragma unroll
    for (int i = 0; i < 4; ++i) rag[i] = x[min(at + i, V - 1)];
  };
  auto ragged = [&](int v0) { return Raw<T>(rag, V - (v0 + (V - v0) / ROW * ROW + 4 * tid)); };
  // f(chunk, its first value's index, whether it is whole) for the row
  auto each = [&](auto&& f) {
    for (int v0 = 0; v0 < (ONE ? 1 : V); v0 += BLOCK) {
      if (!ONE) {
        load_rag(v0);
        load(v0);
      }
      const int whole = (V - v0) / ROW;
#pragma unroll
      for (int k = 0; k < C; ++k) {
        if (ONE) r[k].anew();
        if (k < whole) f(r[k], v0 + k * ROW, true);  // uniform
      }
      if (whole < C) f(ragged(v0), v0 + whole * ROW, false);
    }
  };
  if (greedy || !fair) {
    float m = -INFINITY, first = V, odd = fair ? 0.f : 1.f;  // (below 2^24 an index is exact in fp32)
    auto look = [&](const Raw<T>& a, int v0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = a.get(i);
        first = v > m ? (float)(v0 + 4 * tid + i) : first;
        m = fmaxf(m, v);
        odd = v != v ? 1.f : odd;
      }
    };
    for (int v0 = 0; v0 < (ONE ? 1 : V); v0 += BLOCK) {
      load_rag(v0);
      load(v0);
      const int whole = (V - v0) / ROW;
#pragma unroll
      for (int k = 0; k < C; ++k)
        if (k < whole) look(r[k], v0 + k * ROW);  // uniform
      if (whole < C) look(ragged(v0), v0 + whole * ROW);
    }
    auto larger = [](float u, float v) { return fmaxf(u, v); };
    const float top = over_all<NT>(m, part, larger);
    const bool bad = over_all<NT>(odd, part, larger) > 0.f;
    first = over_all<NT>(m == top ? first : (float)V, part, [](float u, float v) { return fminf(u, v); });
    for (int v0 = 0; v0 < V; v0 += ROW) {
      float a[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = bad ? NAN : v0 + 4 * tid + i == (int)first ? 1.f : 0.f;
      store(a, v0, v0 + ROW <= V);
    }
    return;
  }
  // The sum beside the loads: of the powers over the largest value so far, made smaller
  // where that grows.  A NaN, or infinity less infinity, makes it NaN.
  float m = -INFINITY, l = 0.f;
  auto base = [](float m) { return m == -INFINITY ? 0.f : m; };
  auto power = [&](float v, float from) {
    const float d = fmaf(v, half, -from);
    return __builtin_amdgcn_exp2f(fmaf(d, c, d * rest));
  };
  auto take = [&](const Raw<T>* a, auto n) {
    float top = m;
#pragma unroll
    for (int k = 0; k < decltype(n)::value; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, a[k].get(i));
    const float from = base(top) * half;
    // (four sums of a chunk, then those: 4 roundings of few values, not 16 of all so far)
    float of[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < decltype(n)::value; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) of[i] += power(a[k].get(i), from);
    l = fmaf(l, power(m, from), (of[0] + of[1]) + (of[2] + of[3]));
    m = top;
  };
  std::integral_constant<int, 1> one;
  std::integral_constant<int, 4> four;
  for (int v0 = 0; v0 < (ONE ? 1 : V); v0 += BLOCK) {
    load_rag(v0);
    load(v0);
    const int whole = (V - v0) / ROW;
#pragma unroll
    for (int k = 0; k < C; k += 4) {
      if (k + 4 <= whole) {  // uniform
        take(r + k, four);
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (k + j < whole) take(r + k + j, one);
      }
    }
    if (whole < C) {
      const Raw<T> last = ragged(v0);
      take(&last, one);
    }
  }
  // all loads are back by now; said here, or the stores below would wait for one another
  __builtin_amdgcn_s_waitcnt(VmWait<0>::value);
  auto join = [&](float m2, float l2) {
    const float top = fmaxf(m, m2), from = base(top) * half;
    l = l * power(m, from) + l2 * power(m2, from);
    m = top;
  };
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) join(__shfl_xor(m, o), __shfl_xor(l, o));
  if ((tid & 63) == 0) {
    part[tid >> 6] = m;
    sums[tid >> 6] = l;
  }
  __syncthreads();
  m = part[tid & (NT / 64 - 1)];
  l = sums[tid & (NT / 64 - 1)];
#pragma unroll
  for (int o = NT / 128; o > 0; o >>= 1) join(__shfl_xor(m, o), __shfl_xor(l, o));
  // One lane's sum for all (that of each wave's first lane is the same): one product of a join is
  // rounded and the other is not, so that two lanes that joined each other differ by a last
  // bit, and equal logits would not have equal probabilities.
  l = all_lanes(l);
  m = base(m) * half;
  const float scale = l > 0.f ? 1.f / l : l;  // of -infinity alone 0
  each([&](const Raw<T>& a, int v0, bool whole) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = power(a.get(i), m) * scale;
    store(q, v0, whole);
  });
}

// ----------------------------------------------------------- verification --
// The walk of a sequence: at node c, r_0 = p_c and R_0 = 1; its children are
// tried in the order of their indexes, x accepted if u q_c(x) R_j < r_j(x), else
//   r_{j+1} = max(r_j - R_j q_c, 0) = max(p_c - (R_0 + .. + R_j) q_c, 0), R_{j+1} = sum of r_{j+1}
// (without q: r(x) = 0, R_{j+1} = R_j - r_j(x)).  The next token is the first v
// where the sum of r up to v passes u_0 times the whole.  All of it in 64 bits:
// a sum over 1e5 values in 32 is off by as much as the values are wide, and the
// token would be a neighbour's.
// Tiles of 4096 values: a tile's sum is a thread's, a wave's and the workgroup's, the sum
// over tiles is one tree, so that it does not show which workgroup took which.
// split workgroups have a sequence.  Every one walks, from the few values that the nodes'
// tests need, to where a sum over the vocabulary is wanted (a rejected child has a
// sibling, or the walk is over), adds up its tiles there and counts itself; the last one
// goes on with all of them, alone.  A chain ends there; a tree wants a sum more for
// every rejected child that has siblings: each in a launch of its own, as far as the
// launches go (131072 values: 11 us, 18 us where a workgroup has all of them, which 64-bit
// arithmetic bounds).  Where the vocabulary is small the launches cost more than they save:
// 16 trees of 27 nodes over 8192 values 57 to 70 us by seed, 28 to 39 in one launch; 32768: 46
// to 91 and 28 to 69; 65536: 63 to 83 and 59 to 79; 131072: 50 to 80 and 65 to 113.
// Bound by latency: a chain over 32768 values takes 11.4 us, of which the nodes' values
// are 2.4, the walk 1.6, the sums 2.3, their hand-over 2.1 and the draw 3.1; 16 trees of 27
// nodes over 131072 values 53 to 119 us, by how many sums they want.
#define VF_TILE 4096
#define VF_NODES 1024

namespace {

__device__ __forceinline__ double clean(float v) { return v > 0.f ? (double)v : 0.0; }  // NaN: 0

struct VerifyLds {
  int par[VF_NODES], x[VF_NODES], path[VF_NODES];
  float u[VF_NODES], pv[VF_NODES], qv[VF_NODES];
  int gone[VF_NODES];     // without q: tokens taken out of r
  double part[16];
  int lo[16], hi[16], last;
};

}  // namespace

// What a launch leaves to the next one, of a sequence.
struct VerifyState {
  double mass, times;
  int cur, rounds, taken, i, done, pad;
};

template <bool DRAWN>
__global__ __launch_bounds__(1024) __attribute__((amdgpu_waves_per_eu(4, 4))) void k_verify(const VerifyProb a) {
  extern __shared__ double tiles[];  // [tiles], then [tiles][16] of the waves
  __shared__ VerifyLds s;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int T = a.tokens, ntile = (a.vocab + VF_TILE - 1) / VF_TILE;
  double* const waves = tiles + ntile;
  const long long b = blockIdx.x / (unsigned)a.split;
  const int share = blockIdx.x % (unsigned)a.split;
  const float* P = a.p + b * a.ps;
  const float* Q = DRAWN ? a.q + b * a.qs : nullptr;
  VerifyState* const state = (VerifyState*)a.state + b;
  VerifyState from{1.0, 0.0, 0, 0, 1, 1, 0, 0};
  if (a.launch > 0) from = *state;
  // a node a thread; in LDS only before it is used: a launch that begins with a sum has its
  // values' loads beside the sum's
  int nx = 0, npar = -1, npath = tid ? -1 : 0;
  float nu = 0.f, np = 0.f, nq = 0.f;
  if (tid < T) {
    nx = a.draft[b * T + tid];
    npar = a.parents ? a.parents[b * T + tid] : tid - 1;
    nu = a.u[b * T + tid];
    if (a.launch > 0) npath = a.path[b * T + tid];
    // (a node whose parent does not come before it is reached by no walk)
    if (!(tid > 0 && npar >= 0 && npar < tid && nx >= 0 && nx < a.vocab)) npar = -1;
    if (npar >= 0) {
      np = P[npar * a.pt + nx];
      if (DRAWN) nq = Q[npar * a.qt + nx];
    }
  }
  auto nodes = [&]() {
    if (tid < T) {
      s.par[tid] = npar;
      s.x[tid] = nx;
      s.u[tid] = nu;
      s.pv[tid] = np;
      if (DRAWN) s.qv[tid] = nq;
      s.path[tid] = npath;
    }
    __syncthreads();
  };
  if (from.done) return;
  int cur = from.cur, rounds = from.rounds, taken = from.taken, i = from.i;
  double mass = from.mass;      // R of the current round,
  bool known = a.launch == 0;   // if it has been added up,
  double times = from.times;    // and of those before it

  // r of the current round from the node's values of token v
  auto rest = [&](float pv, float qv, int v) {
    double r = clean(pv);
    if (DRAWN) {
      if (rounds) r = fmax(r - times * clean(qv), 0.0);
    } else {
      for (int j = 0; j < rounds; ++j) r = s.gone[j] == v ? 0.0 : r;
    }
    return r;
  };
  // the first child of the current node from i on, or T
  auto child = [&](int i) {
    for (int k = i & ~63; k < T; k += 64) {
      const uint64_t m = __ballot(k + lane >= i && k + lane < T && s.par[k + lane] == cur);
      if (m) return k + (int)__builtin_ctzll(m);
    }
    return T;
  };
  // on to where a sum is wanted
  auto walk = [&]() {
    for (i = child(i); i < T; i = child(i + 1)) {
      if (!known) return;
      const double r = rest(s.pv[i], DRAWN ? s.qv[i] : 0.f, s.x[i]);
      if ((double)s.u[i] * (DRAWN ? clean(s.qv[i]) : 1.0) * mass < r) {
        if (tid == 0) s.path[taken] = i;
        ++taken;
        cur = i;
        rounds = 0;
        mass = 1.0;
        times = 0.0;
      } else if (DRAWN) {
        times += mass;
        known = false;
        ++rounds;
      } else {
        __syncthreads();  // all have read gone[]
        if (tid == 0) s.gone[rounds] = s.x[i];
        __syncthreads();
        mass -= r;
        ++rounds;
      }
    }
  };
  // the node's four values from v on
  auto load = [&](int v, float* pv, float* qv) {
    const float* pr = P + cur * a.pt + v;
    const float* qr = DRAWN ? Q + cur * a.qt + v : nullptr;
    if (v + 4 <= a.vocab) {
      load_any<4>(pr, pv);
      if (DRAWN && rounds) load_any<4>(qr, qv);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        pv[e] = v + e < a.vocab ? pr[e] : 0.f;
        if (DRAWN && rounds) qv[e] = v + e < a.vocab ? qr[e] : 0.f;
      }
    }
  };
  // tiles[] of every step-th tile from t0 on, eight at a time: their loads are in flight
  // together, and halving the lanes' tiles as the lanes are added takes 10 exchanges, not 48
  auto sums = [&](int t0, int step) {
    __syncthreads();  // tiles[] have been read
    for (int base = t0; base < ntile; base += 8 * step) {
      float pv[8][4] = {}, qv[8][4] = {};
      double z[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int t = base + k * step;
        if ((t + 1) * VF_TILE <= a.vocab) {  // uniform: a whole tile
          load_any<4>(P + cur * a.pt + t * VF_TILE + 4 * tid, pv[k]);
          if (DRAWN && rounds) load_any<4>(Q + cur * a.qt + t * VF_TILE + 4 * tid, qv[k]);
        }
      }
      const int rag = (ntile - 1 - base) / step;  // the tile that may be ragged, the last one, of these eight
      if (a.vocab % VF_TILE && base + rag * step == ntile - 1 && rag < 8) {
        float pe[4], qe[4] = {0.f, 0.f, 0.f, 0.f};
        load((ntile - 1) * VF_TILE + 4 * tid, pe, qe);
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            pv[k][e] = k == rag ? pe[e] : pv[k][e];
            qv[k][e] = k == rag ? qe[e] : qv[k][e];
          }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        z[k] = 0.0;
        const int t = base + k * step, v = t * VF_TILE + 4 * tid;
        if (t < ntile)
          z[k] = (rest(pv[k][0], qv[k][0], v) + rest(pv[k][1], qv[k][1], v + 1)) +
                 (rest(pv[k][2], qv[k][2], v + 2) + rest(pv[k][3], qv[k][3], v + 3));
      }
#pragma unroll
      for (int h = 4; h > 0; h /= 2) {
        const bool upper = lane & (8 * h);
#pragma unroll
        for (int k = 0; k < h; ++k) {
          const double give = upper ? z[k] : z[k + h];
          z[k] = (upper ? z[k + h] : z[k]) + __shfl_xor(give, 8 * h);
        }
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) z[0] += __shfl_xor(z[0], o);
      const int t = base + step * (lane >> 3);  // lane bits 5, 4, 3: which of 4, 2, 1 was kept
      if ((lane & 7) == 0 && t < ntile) waves[16 * t + w] = z[0];
    }
    __syncthreads();
    for (int t = t0 + step * (tid >> 4); t < ntile; t += step * 64) {
      double z = waves[16 * t + (tid & 15)];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) z += __shfl_xor(z, o);
      if ((tid & 15) == 0) tiles[t] = z;
    }
    __syncthreads();
  };
  auto total = [&]() {
    double z = 0.0;
    for (int t = lane; t < ntile; t += 64) z += tiles[t];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) z += __shfl_xor(z, o);
    return z;
  };

  if (a.launch == 0) {
    nodes();
    walk();
  }
  sums(share, a.split);
  if (a.split > 1) {
    uint64_t* const all = (uint64_t*)a.sums + b * ntile;
    for (int t = share + a.split * tid; t < ntile; t += a.split * 1024)
      __hip_atomic_store(all + t, __builtin_bit_cast(uint64_t, tiles[t]), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // they are in memory before the count says so
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0) {
      int* const ct = a.count + b;
      s.last = __hip_atomic_fetch_add(ct, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.split - 1;
      if (s.last) __hip_atomic_store(ct, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!s.last) return;
    for (int t = tid; t < ntile; t += 1024)
      tiles[t] = __builtin_bit_cast(double, __hip_atomic_load(all + t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    if (a.launch > 0) nodes();
    __syncthreads();
  }
  double whole = total();
  while (i < T) {
    const int c0 = cur, r0 = rounds;
    mass = whole;
    known = true;
    walk();
    if (cur == c0 && rounds == r0) break;  // the walk is over where the sum was
    if (a.launch < a.launches - 1) {
      __syncthreads();  // the walk's nodes are one thread's: other waves may be here before it
      if (tid < T) a.path[b * T + tid] = s.path[tid];
      if (tid == 0) *state = VerifyState{mass, times, cur, rounds, taken, i, 0, 0};
      return;
    }
    sums(0, 1);
    whole = total();
  }
  if (!(whole > 0.0)) {  // nothing is left of r: the target's own
    rounds = 0;
    times = 0.0;
    sums(0, 1);
    whole = total();
  }
  // From 1 on no sum passes, said here since the sums below are added in another order than
  // the whole: one may be a last bit larger.
  const double pass = s.u[0] >= 1.f ? (double)INFINITY : (double)s.u[0] * whole;
  // the first tile that holds anything and whose sum passes, then within it; none: the
  // last value there is
  int t = -1, end = -1;
  double before = 0.0;
  for (int t0 = 0; t0 < ntile && t < 0; t0 += 64) {
    const double v = t0 + lane < ntile ? tiles[t0 + lane] : 0.0;
    double x = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double y = __shfl_up(x, o);
      if (lane >= o) x += y;
    }
    const uint64_t past = __ballot(v > 0.0 && before + x > pass), some = __ballot(v > 0.0);
    if (some) end = t0 + 63 - __builtin_clzll(some);
    if (past) t = t0 + __builtin_ctzll(past);
    before += __shfl(past ? x - v : x, past ? __builtin_ctzll(past) : 63);
  }
  const bool inside = t >= 0;
  if (!inside) t = end;
  int found = -1;
  if (t >= 0) {
    const int v0 = t * VF_TILE + 4 * tid;
    float pv[4], qv[4];
    double r[4];
    load(v0, pv, qv);
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = rest(pv[e], qv[e], v0 + e);
    const double z = (r[0] + r[1]) + (r[2] + r[3]);
    double x = z;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double y = __shfl_up(x, o);
      if (lane >= o) x += y;
    }
    if (lane == 63) s.part[w] = x;
    __syncthreads();
    x = x - z + before;
    for (int k = 0; k < w; ++k) x += s.part[k];
    int lo = INT32_MAX, hi = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int v = v0 + e;
      x += r[e];
      if (r[e] > 0.0) {
        hi = v;
        if (x > pass) lo = min(lo, v);
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      lo = min(lo, __shfl_xor(lo, o));
      hi = max(hi, __shfl_xor(hi, o));
    }
    if (lane == 0) {
      s.lo[w] = lo;
      s.hi[w] = hi;
    }
    __syncthreads();
    for (int k = 0; k < 16; ++k) {
      lo = min(lo, s.lo[k]);
      hi = max(hi, s.hi[k]);
    }
    found = inside && lo != INT32_MAX ? lo : hi;
  }
  if (tid < T) a.path[b * T + tid] = s.path[tid];
  if (tid == 0) {
    a.counts[b] = taken;
    a.next[b] = found;
    if (a.launch < a.launches - 1) state->done = 1;
  }
}

// ------------------------------------------------------------- launchers --
namespace {
// the fewest threads and values that hold a row; C: as many as 64 registers hold
template <class T, int C>
void probs_row(const ProbsProb& p, dim3 grid, hipStream_t st) {
  if (p.vocab <= 4096)
    hipLaunchKernelGGL((k_probs<T, 256, 4, true>), grid, dim3(256), 0, st, p);
  else if (p.vocab <= 16384)
    hipLaunchKernelGGL((k_probs<T, 1024, 4, true>), grid, dim3(1024), 0, st, p);
  else if (p.vocab <= 32768)
    hipLaunchKernelGGL((k_probs<T, 1024, 8, true>), grid, dim3(1024), 0, st, p);
  else if (p.vocab <= 4096 * C)
    hipLaunchKernelGGL((k_probs<T, 1024, C, true>), grid, dim3(1024), 0, st, p);
  else
    hipLaunchKernelGGL((k_probs<T, 1024, 8, false>), grid, dim3(1024), 0, st, p);
}
}  // namespace

hipError_t launch_probabilities(const ProbsProb& p, int type, hipStream_t st) {
  const long long most = std::max(((1LL << 22) - 1) / p.tokens, 1LL);  // 2^32 threads a launch
  for (long long b = 0; b < p.seqs; b += most) {
    ProbsProb q = p;
    q.seqs = std::min(most, p.seqs - b);
    q.x = (const uint8_t*)p.x + b * p.xs * (type ? 4 : 2);
    q.y = p.y + b * p.ys;
    if (p.warm) q.warm = p.warm + b;
    const dim3 grid((unsigned)(q.seqs * p.tokens));
    if (type)
      probs_row<float, 16>(q, grid, st);
    else
      probs_row<uint16_t, 32>(q, grid, st);
  }
  return hipGetLastError();
}

int verify_tiles(int vocab) { return (vocab + VF_TILE - 1) / VF_TILE; }

size_t verify_state() { return sizeof(VerifyState); }

hipError_t launch_verify(VerifyProb p, hipStream_t st) {
  const dim3 grid((unsigned)(p.seqs * p.split));
  const size_t lds = (size_t)verify_tiles(p.vocab) * 17 * sizeof(double);
  for (p.launch = 0; p.launch < p.launches; ++p.launch) {
    if (p.q)
      hipLaunchKernelGGL(k_verify<true>, grid, dim3(1024), lds, st, p);
    else
      hipLaunchKernelGGL(k_verify<false>, grid, dim3(1024), lds, st, p);
  }
  return hipGetLastError();
}
