// tree_part.cuh -- how the attention of drafted rows is cut into work, for the kernels that do it
// (dense_tc.cu, tree_rows.cu) and the one that joins their partial results (tree_combine.cu).
//
// An item is a row tile of a sequence (up to RPT of its drafted rows, GH heads of one KV head) with
// all of the sequence's keys, T key tiles of 128. Items lie one after another on a line, each
// T + 1 long: a step for what a unit takes beside its tiles, then its tiles. The line is cut into
// as many equal pieces as there are slots (CTAs, or halves of one); a slot walks its piece, a unit
// for each item that it meets. So all slots have the same work whatever the lengths are, an item
// has as many units as pieces touch its tiles, and neither a list of units nor a launch to make
// one is needed: a CTA sums up the lengths for itself (1 to 2 us; the planner of the shared
// prefixes, a launch of its own, takes 8). From one unit to the next in a walk the item or the
// slot moves on by one, so item + slot numbers the units without a gap that matters, and the place
// of a unit's partial result follows from it.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace gqa {

// A sequence in shared memory; entry B closes the line.
struct alignas(16) TreeSeq {
  int cost0, item0, row0, hist;
};
static_assert(sizeof(TreeSeq) * (kTreeSeqs + 1) + 12 * 8 <= 16384, "the sequences' table and the scan's sums");

// Row tiles, key tiles and the first key (on a block's boundary) of a sequence of n > 0 rows behind hist.
struct TreeShape {
  int tiles, T, key0;
};
__device__ __forceinline__ TreeShape tree_shape(const TreeWork& w, int n, int hist) {
  TreeShape s;
  s.key0 = first_visible_key(hist, w.window) / w.bs * w.bs;
  s.tiles = (n + w.RPT - 1) / w.RPT;
  s.T = (hist + n - s.key0 + 127) / 128;
  return s;
}

// The line, by all THREADS of a CTA; `seq` (and the sums behind it) in shared memory. Ends with a barrier. CTA
// `cta` of `ctas` also writes its share of what the join reads, and CTA 0 reports lengths out of range.
template <int THREADS>
__device__ void tree_line(const TreeWork& w, TreeSeq* seq, int cta, int ctas) {
  constexpr int kWarps = THREADS / 32, kEach = (kTreeSeqs + THREADS - 1) / THREADS;
  int2* sums = reinterpret_cast<int2*>(seq + kTreeSeqs + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  TreeSeq mine[kEach];
  int n_of[kEach];
  int cost = 0, items = 0;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int b = tid * kEach + k;
    mine[k] = TreeSeq{0, 0, 0, 0};
    n_of[k] = 0;
    if (b < w.B) {
      const int s0 = __ldg(w.row_starts + b), s1 = __ldg(w.row_starts + b + 1), hist = w.offsets ? __ldg(w.offsets + b) : 0;
      const long long n = (long long)s1 - s0;
      const bool ok = s0 >= 0 && n >= 0 && s1 <= w.N && n <= w.max_rows && hist >= 0 && hist + n <= w.capacity;
      bad |= !ok;
      mine[k].row0 = s0;
      mine[k].hist = hist;
      n_of[k] = ok ? (int)n : 0;
    }
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    mine[k].cost0 = cost;
    mine[k].item0 = items;
    if (n_of[k] > 0) {
      const TreeShape s = tree_shape(w, n_of[k], mine[k].hist);
      items += w.heads * s.tiles;
      cost += w.heads * s.tiles * (s.T + 1);
    }
  }
  int2 x = make_int2(cost, items);
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, x.x, off), b = __shfl_up_sync(0xffffffffu, x.y, off);
    if (lane >= off) {
      x.x += a;
      x.y += b;
    }
  }
  if (lane == 31) sums[warp] = x;
  bad = __syncthreads_or(bad);
  int2 before = make_int2(0, 0), all = make_int2(0, 0);
#pragma unroll
  for (int v = 0; v < kWarps; ++v) {
    const int2 s = sums[v];
    if (v < warp) {
      before.x += s.x;
      before.y += s.y;
    }
    all.x += s.x;
    all.y += s.y;
  }
  before.x += x.x - cost;
  before.y += x.y - items;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int b = tid * kEach + k;
    mine[k].cost0 += before.x;
    mine[k].item0 += before.y;
    if (b < w.B) seq[b] = mine[k];
    if (b % ctas == cta && b < w.B) {
      int4* rec = reinterpret_cast<int4*>(w.rec + b);
      rec[0] = make_int4(mine[k].row0, n_of[k], mine[k].cost0, mine[k].item0);
      rec[1] = make_int4(mine[k].hist, 0, 0, 0);
    }
  }
  if (tid == 0) {
    seq[w.B] = TreeSeq{all.x, all.y, 0, 0};
    if (cta == 0) {
      w.line[0] = all.x;
      w.line[1] = min(w.slots, all.x);
      if (bad) raise_error(w.err, kErrBounds);
    }
  }
  __syncthreads();
  // which sequence a row is of: a hint that the join checks, since nothing is written for rows outside
  for (int b = cta; b < w.B; b += ctas) {
    if ((b + 1 < w.B ? seq[b + 1].item0 : all.y) == seq[b].item0) continue;
    const int s0 = seq[b].row0, n = __ldg(w.row_starts + b + 1) - s0;
    for (int i = tid; i < n; i += THREADS) w.row_seq[s0 + i] = b;
  }
}

// A slot's walk along its piece of the line.
struct TreeWalk {
  int at, end, slot;
};
__device__ __forceinline__ TreeWalk tree_walk(const TreeWork& w, const TreeSeq* seq, int slot) {
  const int C = seq[w.B].cost0, S = min(w.slots, C);
  TreeWalk k;
  k.slot = slot;
  k.at = slot < S ? (int)((long long)C * slot / S) : 0;
  k.end = slot < S ? (int)((long long)C * (slot + 1) / S) : 0;
  return k;
}

// The next unit of a walk; false at its end.
struct TreeUnit {
  int b, hc, tile, row0, n, hist;  // hc: KV head and head chunk; the sequence's rows row0 .. row0 + n - 1
  int key0, key1, index;
};
__device__ __forceinline__ bool tree_next(const TreeWork& w, const TreeSeq* seq, TreeWalk& k, TreeUnit& u) {
  while (k.at < k.end) {
    int lo = 0, hi = w.B;  // the last sequence that starts at or before `at`
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (seq[mid].cost0 <= k.at) lo = mid;
      else hi = mid;
    }
    const TreeSeq q = seq[lo];
    u.b = lo;
    u.row0 = q.row0;
    u.hist = q.hist;
    u.n = __ldg(w.row_starts + lo + 1) - q.row0;
    const TreeShape s = tree_shape(w, u.n, q.hist);
    const int r = k.at - q.cost0, item = r / (s.T + 1), off = r - item * (s.T + 1);
    const int to = min(s.T + 1, off + k.end - k.at);
    k.at += to - off;
    if (to <= 1) continue;  // (the item's first step alone)
    u.hc = item / s.tiles;
    u.tile = item - u.hc * s.tiles;
    u.key0 = s.key0 + max(off - 1, 0) * 128;
    u.key1 = min(s.key0 + (to - 1) * 128, q.hist + u.n);
    u.index = q.item0 + item + k.slot;
    return true;
  }
  return false;
}

// The slot whose piece holds place x of the line.
__device__ __forceinline__ int tree_slot_of(int C, int S, int x) {
  return (int)((((long long)x + 1) * S - 1) / C);
}

// Drafted rows that row i (of n, packed row `row`) sees: bits o .. o + 31 of its mask. Bits below 0 stand
// for the history and are set, those from n on are not.
__device__ __forceinline__ uint32_t tree_bits(const TreeWork& w, int row, int i, int n, int o) {
  uint32_t x;
  if (!w.mask) {  // a chain: rows up to its own
    const int upto = i + 1 - o;
    x = upto >= 32 ? 0xffffffffu : upto <= 0 ? 0u : (1u << upto) - 1u;
  } else {
    const unsigned long long* m = w.mask + (size_t)row * w.words;
    const int first = max(o, 0), word = first >> 6, shift = first & 63;
    unsigned long long v = word < w.words ? __ldg(m + word) >> shift : 0ull;
    if (shift > 32 && word + 1 < w.words) v |= __ldg(m + word + 1) << (64 - shift);
    x = (uint32_t)v;
    if (o < 0) x = o <= -32 ? 0xffffffffu : x << -o | ((1u << -o) - 1u);
  }
  const int left = n - o;
  return left >= 32 ? x : left <= 0 ? 0u : x & ((1u << left) - 1u);
}

// Drafted rows that row i sees, itself among them where its mask says so; at least 1: the row stands at
// position hist + this - 1.
__device__ __forceinline__ int tree_depth(const TreeWork& w, int row, int i, int n) {
  if (!w.mask) return i + 1;
  const unsigned long long* m = w.mask + (size_t)row * w.words;
  int c = 0;
  for (int x = 0; x < w.words; ++x) {
    const int left = n - 64 * x;
    unsigned long long v = left > 0 ? __ldg(m + x) : 0ull;
    if (left > 0 && left < 64) v &= (1ull << left) - 1;
    c += __popcll(v);
  }
  return max(c, 1);
}

// Of the 32 drafted rows from o on that `bits` names, those within the window of a row at depth `depth`
// (bits of the history stay).
__device__ __forceinline__ uint32_t tree_window(const TreeWork& w, uint32_t bits, int row0, int n, int o, int depth) {
  if (depth <= w.window) return bits;  // (the first drafted row is in it)
  uint32_t out = bits;
  for (uint32_t x = bits; x; x &= x - 1) {
    const int j = o + __ffs(x) - 1;
    if (j >= 0 && tree_depth(w, row0 + j, j, n) <= depth - w.window) out &= ~(x & -x);
  }
  return out;
}

}  // namespace gqa
