// tree_part.cuh -- how the attention of drafted rows is cut into work, for the kernels that do it
// (dense_tc.cu, tree_rows.cu) and the one that joins their partial results (tree_combine.cu).
//
// An item is a row tile of a sequence (up to RPT of its drafted rows, GH heads of one KV head) with
// all of the sequence's keys, T key tiles of 128 (SIMT: 64). Items lie one after another on a line, each
// T + 1 long: a step for what a unit takes beside its tiles, then its tiles. The line is cut into
// as many equal pieces as there are slots (CTAs, or halves of one); a slot walks its piece, a unit
// for each item that it meets. So all slots have the same work whatever the lengths are, an item
// has as many units as pieces touch its tiles, and neither a list of units nor a launch to make
// one is needed: a CTA sums up the lengths for itself (the planner of the shared prefixes, a
// launch of its own, takes 8 us). From one unit to the next in a walk the item or the slot moves
// on by one, so item + slot numbers the units without a gap that matters, and the place of a
// unit's partial result follows from it. A unit that has all of an item's tiles writes the rows' outputs.
//
// There are two lines. Where a sequence has two row tiles or more (of the same heads), pairs of them lie on the
// first, cut for the CTAs: the halves of a CTA take a tile each of the same keys at the same time, so
// that the second finds them in L2. (As items of their own, 8 sequences of two row tiles behind 24,600 keys
// read every key twice from HBM: 257 us.) Single row tiles lie on the second, cut for all the
// halves. Every slot has its piece of both.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace gqa {

// A sequence in shared memory; entry B closes the lines. [0] the line of pairs, [1] that of single tiles.
// (The kernels go by what is here: row_starts is read once, whatever happens to it meanwhile.)
struct alignas(16) TreeSeq {
  int cost0[2], item0[2], row0, n, hist, pad;
};
static_assert(sizeof(TreeSeq) * (kTreeSeqs + 1) + 12 * 16 <= 16384, "the sequences' table and the scan's sums");

// Row tiles, key tiles and the first key (on a block's boundary) of a sequence of n > 0 rows behind hist.
struct TreeShape {
  int tiles, T, key0;
};
__device__ __forceinline__ TreeShape tree_shape(const TreeWork& w, int n, int hist) {
  TreeShape s;
  s.key0 = first_visible_key(hist, w.window) / w.bs * w.bs;
  s.tiles = (n + w.RPT - 1) / w.RPT;
  s.T = (hist + n - s.key0 + (1 << w.step_log2) - 1) >> w.step_log2;
  return s;
}
// Items of each of its head chunks on line x.
__device__ __forceinline__ int tree_items(const TreeWork& w, int tiles, int x) {
  return x == 0 ? (w.pair_slots ? tiles >> 1 : 0) : w.pair_slots ? tiles & 1 : tiles;
}
__device__ __forceinline__ int tree_slots(const TreeWork& w, int x) { return x == 0 ? w.pair_slots : w.slots; }

// The slot whose piece holds place x of a line of length C cut for S.
__device__ __forceinline__ int tree_slot_of(int C, int S, int x) {
  return (int)((((long long)x + 1) * S - 1) / C);
}

// The lines, by all THREADS of a CTA; `seq` (and the sums behind it) in shared memory. Ends with a barrier. CTA 0
// reports lengths out of range.
template <int THREADS>
__device__ void tree_line(const TreeWork& w, TreeSeq* seq, int cta) {
  constexpr int kWarps = THREADS / 32, kEach = (kTreeSeqs + THREADS - 1) / THREADS;
  int4* sums = reinterpret_cast<int4*>(seq + kTreeSeqs + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  TreeSeq mine[kEach];
  int4 sum = make_int4(0, 0, 0, 0);  // costs, items
  bool bad = false, back = false;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int b = tid * kEach + k;
    mine[k] = TreeSeq{};
    if (b < w.B) {
      const int s0 = __ldg(w.row_starts + b), s1 = __ldg(w.row_starts + b + 1), hist = w.offsets ? __ldg(w.offsets + b) : 0;
      const long long n = (long long)s1 - s0;
      const bool ok = s0 >= 0 && n >= 0 && s1 <= w.N && n <= w.max_rows && hist >= 0 && hist + n <= w.capacity;
      bad |= !ok;
      back |= n < 0;
      mine[k].row0 = s0;
      mine[k].hist = hist;
      mine[k].n = ok ? (int)n : 0;
    }
  }
  // starts that go back: sequences overlap, and their tiles may be more than there is room for; none is taken
  back = __syncthreads_or(back);
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    if (back) mine[k].n = 0;
    mine[k].cost0[0] = sum.x;
    mine[k].cost0[1] = sum.y;
    mine[k].item0[0] = sum.z;
    mine[k].item0[1] = sum.w;
    if (mine[k].n > 0) {
      const TreeShape s = tree_shape(w, mine[k].n, mine[k].hist);
      const int pairs = w.heads * tree_items(w, s.tiles, 0), singles = w.heads * tree_items(w, s.tiles, 1);
      sum.x += pairs * (s.T + 1);
      sum.y += singles * (s.T + 1);
      sum.z += pairs;
      sum.w += singles;
    }
  }
  int4 x = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, x.x, off), b = __shfl_up_sync(0xffffffffu, x.y, off);
    const int c = __shfl_up_sync(0xffffffffu, x.z, off), d = __shfl_up_sync(0xffffffffu, x.w, off);
    if (lane >= off) x = make_int4(x.x + a, x.y + b, x.z + c, x.w + d);
  }
  if (lane == 31) sums[warp] = x;
  bad = __syncthreads_or(bad);
  int4 before = make_int4(x.x - sum.x, x.y - sum.y, x.z - sum.z, x.w - sum.w), all = make_int4(0, 0, 0, 0);
#pragma unroll
  for (int v = 0; v < kWarps; ++v) {
    const int4 s = sums[v];
    if (v < warp) before = make_int4(before.x + s.x, before.y + s.y, before.z + s.z, before.w + s.w);
    all = make_int4(all.x + s.x, all.y + s.y, all.z + s.z, all.w + s.w);
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int b = tid * kEach + k;
    mine[k].cost0[0] += before.x;
    mine[k].cost0[1] += before.y;
    mine[k].item0[0] += before.z;
    mine[k].item0[1] += before.w;
    if (b < w.B) seq[b] = mine[k];
  }
  if (tid == 0) {
    seq[w.B] = TreeSeq{{all.x, all.y}, {all.z, all.w}, 0, 0, 0, 0};
    if (cta == 0) {
      w.line[0] = 2 * all.z + all.w;  // row tiles
      if (bad) raise_error(w.err, kErrBounds);
    }
  }
  __syncthreads();
}

// What the join reads: for each row tile of this CTA's share of the sequences its rows and its parts. By `threads`
// threads of the CTA that have nothing else to do yet (before the first load it took 1 us of the call).
__device__ __forceinline__ void tree_publish(const TreeWork& w, const TreeSeq* seq, int cta, int ctas, int tid, int threads) {
  for (int b = cta; b < w.B; b += ctas) {
    const TreeSeq q = seq[b];
    if (q.n == 0) continue;
    const int first = 2 * q.item0[0] + q.item0[1], n = q.n;
    const TreeShape s = tree_shape(w, n, q.hist);
    for (int e = tid; e < w.heads * s.tiles; e += threads) {
      const int hc = e / s.tiles, tile = e - hc * s.tiles, paired = 2 * tree_items(w, s.tiles, 0);
      const int x = tile >= paired, each = tree_items(w, s.tiles, x);
      const int in = hc * each + (x ? tile - paired : tile >> 1);  // of the sequence's items on line x
      const int C = seq[w.B].cost0[x], S = min(tree_slots(w, x), C), at = q.cost0[x] + in * (s.T + 1);
      const int s0 = tree_slot_of(C, S, at + 1), s1 = tree_slot_of(C, S, at + s.T);
      TreeRec r;
      r.row = q.row0 + tile * w.RPT;
      r.n = min(w.RPT, n - tile * w.RPT);
      r.hc = hc;
      r.b = b;
      r.parts = w.whole && s0 == s1 ? 0 : s1 - s0 + 1;
      r.stride = x ? 1 : 2;
      r.part = x ? 2 * (seq[w.B].item0[0] + w.pair_slots) + q.item0[1] + in + s0 : 2 * (q.item0[0] + in + s0) + (tile & 1);
      r.hist = q.hist;
      r.row0 = q.row0;
      r.rows = n;
      int4* to = reinterpret_cast<int4*>(w.rec + first + e);
      to[0] = make_int4(r.row, r.n, r.hc, r.b);
      to[1] = make_int4(r.part, r.parts, r.stride, r.hist);
      to[2] = make_int4(r.row0, r.rows, 0, 0);
    }
  }
}

// A slot's walk along its piece of line x.
struct TreeWalk {
  int at, end, slot;
};
__device__ __forceinline__ TreeWalk tree_walk(const TreeWork& w, const TreeSeq* seq, int x, int slot) {
  const int C = seq[w.B].cost0[x], S = min(tree_slots(w, x), C);
  TreeWalk k;
  k.slot = slot;
  // C * slot / S in 32 bits (by 64-bit divisions a walk began 0.5 us later)
  const int each = S > 0 ? C / S : 0, rest = C - each * S;
  k.at = slot < S ? each * slot + rest * slot / S : 0;
  k.end = slot < S ? each * (slot + 1) + rest * (slot + 1) / S : 0;
  return k;
}

// The next unit of a walk along line x; false at its end. half: the tile of a pair that is wanted.
struct TreeUnit {
  int b, hc, tile, row0, n, hist;  // hc: KV head and head chunk; the sequence's rows row0 .. row0 + n - 1
  int key0, key1, index;  // index: of its partial result; below 0: it has all of the item's keys and is ~ the row tile
};
__device__ __forceinline__ bool tree_next(const TreeWork& w, const TreeSeq* seq, int x, int half, TreeWalk& k, TreeUnit& u) {
  while (k.at < k.end) {
    int lo = 0, hi = w.B;  // the last sequence that starts at or before `at`
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (seq[mid].cost0[x] <= k.at) lo = mid;
      else hi = mid;
    }
    const TreeSeq q = seq[lo];
    u.b = lo;
    u.row0 = q.row0;
    u.hist = q.hist;
    u.n = q.n;
    const TreeShape s = tree_shape(w, u.n, q.hist);
    const int r = k.at - q.cost0[x], item = r / (s.T + 1), off = r - item * (s.T + 1);
    const int to = min(s.T + 1, off + k.end - k.at);
    k.at += to - off;
    if (to <= 1) continue;  // (the item's first step alone)
    const int each = tree_items(w, s.tiles, x);
    u.hc = item / each;
    u.tile = x ? 2 * tree_items(w, s.tiles, 0) + item - u.hc * each : 2 * (item - u.hc * each) + half;
    u.key0 = s.key0 + (max(off - 1, 0) << w.step_log2);
    u.key1 = min(s.key0 + ((to - 1) << w.step_log2), q.hist + u.n);
    const int at = q.item0[x] + item + k.slot;
    u.index = x ? 2 * (seq[w.B].item0[0] + w.pair_slots) + at : 2 * at + half;
    if (w.whole && off <= 1 && to == s.T + 1) u.index = ~(2 * q.item0[0] + q.item0[1] + u.hc * s.tiles + u.tile);
    return true;
  }
  return false;
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
