// Shapes of the attention's launches, from the call's sizes alone (no HIP: the
// tests build this for the host).
#pragma once
#include <algorithm>

struct AttnPlan {
  // Row blocks of 16 nb rows (64 nb in the kernel for many rows), shares of a key
  // head and row block that run at once, the most units (shares of a key head)
  // there can be, the most of them in the workspace, and the most shares and the
  // expected number of a sequence.
  int nb, nrb, wide, fit, units, kept, most, shares;
};

// Rows of a call (R of a sequence and key head), and shares of its positions (`hold`
// runs of 256 in a sequence's table).  k_tree_attn takes as few blocks
// of up to 48 rows (32 for head sizes above 128, whose sums need the registers)
// as hold the rows of a (sequence, key head), of equal size; where that is more
// than one, k_tree_attn_wide takes 64 or 128 rows a block if it pads them to no
// more.  24 sequences of 8 heads, 2048 to 4096 positions of 128, 8 bits, narrow
// and wide: 64 rows 84.0 and 76.5 us, 96 rows 101.5 and 105.1, 128 rows 136.4
// and 115.2, 192 rows 181.4 and 207.6, 256 rows 229.9 and 218.3.
inline AttnPlan plan_attention(long long R, int seqs, int kv_heads, int dim, long long hold, int ncu) {
  AttnPlan p{};
  const long long r16 = (R + 15) / 16, most = dim <= 128 ? 3 : 2;
  p.nrb = (int)((r16 + most - 1) / most);
  p.nb = (int)((r16 + p.nrb - 1) / p.nrb);
  const long long wide = R > 64 && dim <= 128 ? 8 : 4, wrb = (r16 + wide - 1) / wide;
  p.wide = p.nrb > 1 && wrb * wide <= (long long)p.nrb * p.nb;
  if (p.wide) {
    p.nrb = (int)wrb;
    p.nb = (int)wide / 4;
  }
  // shares of one head and row block: what runs at once, and one more for each
  // sequence by rounding up; those of sequences with more than one are at most
  // twice what runs at once, or, at 256 positions or more each, what the tables hold
  // Workgroups of four waves, two to a CU; from 17 rows on of eight (head sizes
  // up to 128), or of four that need a SIMD's registers each, one to a CU: their
  // shares are half as many to join (40 rows of 131071 positions 41 us, 46 with
  // four waves; 4 rows of 4096 to 8192 positions 89 us with eight, 85 with four).
  const long long slots = (p.wide || p.nb == 1 ? 2 : 1) * ncu;
  const long long fit = std::max(slots / ((long long)kv_heads * p.nrb), 1LL);
  p.fit = (int)fit;
  p.units = (int)((std::min(fit, hold * seqs) + seqs) * kv_heads);
  p.kept = (int)(std::min(2 * fit, hold * seqs) * kv_heads);
  p.most = (int)std::min(fit, hold);
  p.shares = (int)std::min(hold, std::max(fit / seqs, 1LL));
  return p;
}

// The launch that joins shares: G threads for every four values of a row, as
// many rows as 256 threads hold, and no thread beyond them (head sizes of 96 and
// 192 leave room for none or a part of a row: a thread there would look for its
// partners' sums past the end of the array).
// Eight threads for a value where there are many shares: 160 rows of 128
// shares 8 us, 15 with one; 13824 rows of three shares 5 us, 11 with eight.
struct JoinPlan {
  int G, rows, threads;
};
inline JoinPlan plan_join(int dim, int shares) {
  const int G = shares >= 16 ? (dim <= 128 ? 8 : 4) : 1, q4 = dim / 4;
  const int rows = std::max(256 / (q4 * G), 1);
  return JoinPlan{G, rows, rows * q4 * G};
}
// Thread tid of it: the k-th of dimensions d .. d + 3 of row i; its j-th partner
// is tid + j dim / 4.
struct JoinThread {
  int i, k, d;
};
constexpr JoinThread join_thread(int tid, int dim, int G) {
  return JoinThread{tid / (dim / 4 * G), tid / (dim / 4) % G, 4 * (tid % (dim / 4))};
}

// Workgroups of the attention's launch (rounded up for the XCDs) and their threads.
inline long long attention_blocks(const AttnPlan& p) { return ((long long)p.units + 7) / 8 * 8 * p.nrb; }
inline int attention_threads(const AttnPlan& p, int dim) { return !p.wide && p.nb > 1 && dim <= 128 ? 512 : 256; }
// Whether the threads of both launches can be counted in 32 bits (rows: of all
// sequences and query heads).
inline bool attention_fits(const AttnPlan& p, long long rows, int dim) {
  const JoinPlan j = plan_join(dim, p.shares);
  const long long join = p.most > 1 ? (rows + j.rows - 1) / j.rows * j.threads : 0;
  return attention_blocks(p) * attention_threads(p, dim) < 1LL << 32 && join < 1LL << 32;
}
