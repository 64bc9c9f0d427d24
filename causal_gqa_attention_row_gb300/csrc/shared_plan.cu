// shared_plan.cu -- the plan of a shared-prefix decode step, by one CTA: which sequences
// have a prefix to share, and the list of units that dense_tc_kernel works off, the
// prefixes' first, then those of the sequences' own keys.
//
// A product with V mixes the keys of a tile before any mask can hold a key back whose V is
// not finite (0 * NaN). So a group shares just the keys that every one of its sharers sees:
// [key_lo, prefix), key_lo the highest that a sharer's window leaves. A member that ends
// in the prefix, or whose window does not reach it, does not share; what a sharer sees
// below key_lo and behind the prefix are its own keys, two ranges.
//
// The prefix of group g is tiles_g row tiles per KV head (and head chunk) times n_g key
// tiles; the own keys of a sequence are one row tile per KV head (and head chunk). Units
// take c key tiles each, c the same for all and chosen to minimise
//   max(ceil(prefix units / slots) * (c + kDenseUnitTiles), (all tiles + units * kDenseUnitTiles) / slots) + c / 8,
// in key tiles: the rounds that the prefixes' equal units take on the slots (units worked on
// at a time), in whose last round own units fill the rest, or all work spread evenly; and
// something for the longest unit, which the rest may have to wait for.
// Every candidate c is tried, a thread each. Own units are listed longest first.
//
// The other kernels wait for this one. It runs on an SM that has run other code since the
// last step, so most of its time is the fetch of its own: it is kept short (one copy of
// each step, no unrolled loops, no 64-bit divisions), and up to kPlanGroups groups stay in
// shared memory.
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace gqa {
namespace {

constexpr int kPlanGroups = 128;
constexpr int kBuckets = 64;
// Candidates for c: all lengths up to the longest range's, so that the last one, a single key
// range for each row tile, is among them however long the tables are.
constexpr int kMostTiles = 1 << 23;
static_assert((long long)kMostTiles * 128 >= INT_MAX / 2, "a table row names up to INT_MAX / 2 keys");

// Exclusive prefix sums of three values over the CTA; `total` receives the sums. Ends with
// a barrier.
template <int kWarps>
__device__ __forceinline__ void exclusive_scans(int (&v)[3], int (&total)[3], int (*warp_sums)[kWarps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x[3] = {v[0], v[1], v[2]};
#pragma unroll 1
  for (int off = 1; off < 32; off <<= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int y = __shfl_up_sync(0xffffffffu, x[k], off);
      if (lane >= off) x[k] += y;
    }
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < 3; ++k) warp_sums[k][warp] = x[k];
  __syncthreads();
  int w[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) w[k] = lane < kWarps ? warp_sums[k][lane] : 0;
#pragma unroll 1
  for (int off = 1; off < 32; off <<= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int y = __shfl_up_sync(0xffffffffu, w[k], off);
      if (lane >= off) w[k] += y;
    }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    total[k] = __shfl_sync(0xffffffffu, w[k], 31);
    const int before = __shfl_sync(0xffffffffu, w[k], max(warp - 1, 0));
    v[k] = (warp == 0 ? 0 : before) + x[k] - v[k];
  }
  __syncthreads();
}

// CTA-wide sum of 32-bit values and minimum of 64-bit ones (shuffles, then one value a
// warp: 64-bit atomics on one shared word by every thread took the kernel 10 us). End with a
// barrier.
template <int kWarps>
__device__ __noinline__ int block_sum(int v, int* warps) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  v = __reduce_add_sync(0xffffffffu, (threadIdx.x & 31) < kWarps ? warps[threadIdx.x & 31] : 0);
  __syncthreads();
  return v;
}
__device__ __forceinline__ unsigned long long warp_min(unsigned long long v) {
#pragma unroll 1
  for (int off = 16; off >= 1; off >>= 1) {
    const unsigned long long o = __shfl_xor_sync(0xffffffffu, v, off);
    v = o < v ? o : v;
  }
  return v;
}

// What sequence b, of length n, brings to the plan.
struct Seq {
  int g;             // the group that it shares the prefix of, or -1
  int len;           // 0: out of range
  int first;         // the first key it sees
  int key0[2], nt[2];  // own keys, below the shared ones and behind them: tiles from a block's boundary on
  int end[2];
};
// (not inlined: the kernel's time is mostly that of fetching its code)
__device__ __noinline__ Seq sequence(const SharedPlan& s, const DenseGroup* groups, int n_groups, int b, int n) {
  Seq q = {-1, 0, 0, {0, 0}, {0, 0}, {0, 0}};
  if (n < 1 || n > s.capacity) return q;
  q.len = n;
  q.first = first_visible_key(n - 1, s.window);
  if (n_groups > 0 && b >= groups[0].first) {
    int lo = 0, hi = n_groups;  // first[lo] <= b < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (groups[mid].first <= b) lo = mid;
      else hi = mid;
    }
    const DenseGroup& d = groups[lo];
    if (b < d.first + d.members && n >= d.prefix && q.first < d.prefix) q.g = lo;
  }
  q.key0[0] = q.first / s.bs * s.bs;
  q.end[0] = q.g < 0 ? n : groups[q.g].key_lo;
  if (q.end[0] > q.first) q.nt[0] = (q.end[0] - q.key0[0] + 127) / 128;
  if (q.g >= 0) {
    q.key0[1] = groups[q.g].prefix;
    q.end[1] = n;
    q.nt[1] = (n - q.key0[1] + 127) / 128;
  }
  return q;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) shared_plan_kernel(const __grid_constant__ SharedPlan s) {
  constexpr int kWarps = kThreads / 32;
  __shared__ int warp_sums[3][kWarps];
  __shared__ int bucket_at[kBuckets];
  __shared__ int bad, bad_len, max_tiles;
  __shared__ unsigned long long warp_best[kWarps];
  __shared__ DenseGroup group_s[kPlanGroups];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x;
  DenseGroup* groups = s.n_groups <= kPlanGroups ? group_s : s.groups;
  if (tid == 0) {
    bad = bad_len = 0;
    max_tiles = 1;
  }
  if (tid < kBuckets) bucket_at[tid] = 0;
  // (the thread's own length is on its way while the groups are read)
  const int len_tid = tid < s.B ? __ldg(s.seq_lens + tid) : 0;
  const auto seq_of = [&](int b) {
    return sequence(s, groups, bad ? 0 : s.n_groups, b, b == tid ? len_tid : __ldg(s.seq_lens + b));
  };
  __syncthreads();
  // ---- groups: ascending starts within the batch, prefixes within the tables; with
  // anything else no prefix is shared (every sequence reads its own rows) and the
  // error word says so
  for (int g = tid; g < s.n_groups; g += kThreads) {
    const int a = s.group_starts[g], z = s.group_starts[g + 1], nb = s.shared_blocks[g];
    if (a < 0 || z < a || z > s.B || nb < 0 || nb > s.mbps) bad = 1;
    DenseGroup d = {};
    d.first = a;
    d.members = z - a;
    d.prefix = z - a >= 2 ? nb * s.bs : 0;
    d.source = s.B;
    groups[g] = d;
  }
  __syncthreads();
  const int n_groups = bad ? 0 : s.n_groups;
#pragma unroll 1
  for (int b0 = 0; b0 < s.B; b0 += kThreads) {
    const int b = b0 + tid;
    int g = -1, first = 0;
    if (b < s.B) {
      const Seq q = seq_of(b);
      if (q.len == 0) bad_len = 1;
      g = q.g;
      first = q.first;
    }
    // (most warps hold members of one group: one atomic a warp then)
    const int g0 = __shfl_sync(0xffffffffu, g, 0);
    const bool one = __all_sync(0xffffffffu, g == g0);
    const int most = __reduce_max_sync(0xffffffffu, one ? first : 0);
    if (g >= 0 && (!one || (tid & 31) == 0)) {
      atomicMax(&groups[g].key_lo, one ? most : first);
      atomicAdd(&groups[g].sharers, one ? 32 : 1);
      atomicMin(&groups[g].source, b);
    }
  }
  __syncthreads();
  if ((bad || bad_len) && tid == 0) raise_error(s.err, kErrBounds);
  for (int g = tid; g < n_groups; g += kThreads) {
    DenseGroup d = groups[g];
    d.key_lo = (d.key_lo + s.bs - 1) / s.bs * s.bs;
    const int nt = d.sharers >= 2 ? max(d.prefix - d.key_lo + 127, 0) / 128 : 0;
    if (nt == 0) d.prefix = 0;
    d.n_splits = nt;
    d.tiles = nt > 0 ? (d.members + s.RPT - 1) / s.RPT : 0;
    groups[g] = d;
    if (nt > 0) atomicMax(&max_tiles, nt);
  }
  __syncthreads();
  // ---- c (costs in floats: any c is right, the same one for the same batch)
  const int heads = s.Hkv * s.n_hchunks;
  int mine = 0, longest = 0;
#pragma unroll 1
  for (int b = tid; b < s.B; b += kThreads) {
    const Seq q = seq_of(b);
    mine += q.nt[0] + q.nt[1];
    longest = max(longest, max(q.nt[0], q.nt[1]));
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if ((tid & 31) == 0) atomicMax(&max_tiles, longest);
  const int own_tiles = block_sum<kWarps>(mine, warp_sums[0]);  // of each head chunk
  const float own_all = (float)own_tiles * (float)heads, own_items = (float)s.B * (float)heads;
  const int c_own_least = (int)ceilf(own_all / (float)kOwnExtra);  // own parts <= 2 items + kOwnExtra
  const int c_most = max_tiles;
  unsigned long long best = ~0ull;
#pragma unroll 1
  for (int c = 1 + tid; c <= c_most; c += kThreads) {
    float units = 0.f, tiles = 0.f;
#pragma unroll 1
    for (int g = 0; g < n_groups; ++g) {
      const float t = (float)(heads * groups[g].tiles);
      units += t * (float)((groups[g].n_splits + c - 1) / c);
      tiles += t * (float)groups[g].n_splits;
    }
    if (units > (float)s.max_prefix_units) continue;
    const float rounds = ceilf(units / (float)s.slots) * (float)(c + kDenseUnitTiles);
    const float even =
        (tiles + own_all + (units + own_all / (float)max(c, c_own_least) + own_items * 0.5f) * (float)kDenseUnitTiles) /
        (float)s.slots;
    // an eighth of a unit for the tail that one leaves behind (the geometric mean of a step's time
    // over twelve batches, 8 to 300 sequences behind 1,000 to 60,000 keys: with a quarter 62.1 us,
    // an eighth 59.8; with a quarter and units that cost 2, 3 or 4 tiles 59.9, 60.4, 60.7); ties go
    // to the longer units
    const float cost = fmaxf(rounds, even) + 0.125f * (float)c;
    const unsigned long long key = (unsigned long long)__float_as_uint(cost) << 32 | (unsigned)(kMostTiles - c);
    best = key < best ? key : best;
  }
  best = warp_min(best);
  if ((tid & 31) == 0) warp_best[tid >> 5] = best;
  __syncthreads();
  best = warp_min(warp_best[tid & (kWarps - 1)]);
  // (the largest c always fits: the caller sized max_prefix_units for it)
  const int c = best == ~0ull ? c_most : kMostTiles - (int)(best & 0xffffffffu);
  const int c_own = min(max(c, c_own_least), max_tiles);  // (the longest range in one part)
  // ---- key ranges per group; own parts: of c_own tiles, the last of a range shorter (rest tiles)
  const int per = (s.n_groups + kThreads - 1) / kThreads;
  const int lo = min(n_groups, tid * per), hi = min(n_groups, lo + per);
  int at[3] = {0, 0, 0};  // prefix units, own parts, those of them that are full
  for (int g = lo; g < hi; ++g) {
    DenseGroup& d = groups[g];
    d.n_splits = (d.n_splits + c - 1) / c;
    at[0] += heads * d.tiles * d.n_splits;
  }
  const auto bucket = [&](int rest) { return (c_own - rest) * (kBuckets - 1) / c_own; };
  const int per_b = (s.B + kThreads - 1) / kThreads;
  const int b_lo = min(s.B, tid * per_b), b_hi = min(s.B, b_lo + per_b);
#pragma unroll 1
  for (int b = b_lo; b < b_hi; ++b) {
    const Seq q = seq_of(b);
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
      const int nt = e ? q.nt[1] : q.nt[0], full = nt / c_own, rest = nt - full * c_own;
      at[1] += (full + (rest != 0)) * heads;
      at[2] += full * heads;
      if (rest) atomicAdd(&bucket_at[bucket(rest)], heads);
    }
  }
  int sum[3];
  exclusive_scans(at, sum, warp_sums);  // (its barriers: the buckets are in place)
  const int n_prefix = sum[0], n_full = sum[2];
  for (int g = lo; g < hi; ++g) {
    DenseGroup& d = groups[g];
    d.unit0 = at[0];
    at[0] += heads * d.tiles * d.n_splits;
  }
  if (tid < 32) {  // where the buckets start, two a lane
    const int x = bucket_at[2 * tid], y = bucket_at[2 * tid + 1];
    int before = x + y;
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, before, off);
      if (tid >= off) before += up;
    }
    bucket_at[2 * tid] = n_prefix + n_full + before - x - y;
    bucket_at[2 * tid + 1] = n_prefix + n_full + before - y;
    if (tid == 31) {
      s.units_listed[0] = n_prefix + n_full + before;
      s.units_listed[1] = 0;  // the ticket counter
    }
  }
  __syncthreads();
  // ---- the sequences' records, the first of their full units left in the last field ...
#pragma unroll 1
  for (int b = b_lo; b < b_hi; ++b) {
    const Seq q = seq_of(b);
    SeqPlan r = {};
    r.n_own = (q.nt[0] + c_own - 1) / c_own + (q.nt[1] + c_own - 1) / c_own;
    r.own_part0 = at[1];
    r.full0 = n_prefix + at[2];
    if (q.g >= 0) {
      const DenseGroup& d = groups[q.g];
      const int i = b - d.first, tile = i / s.RPT;
      r.n_pre = d.n_splits;
      r.pre_unit0 = d.unit0 + tile * d.n_splits;
      r.pre_stride = d.tiles * d.n_splits;
      r.row0 = (i - tile * s.RPT) * s.GH;
    }
    s.seq[b] = r;
    at[1] += heads * r.n_own;
    at[2] += heads * (q.nt[0] / c_own + q.nt[1] / c_own);
  }
  __syncthreads();
  // ---- ... and the units, a thread per sequence and head chunk
  const int part_step = (int)(dense_part_floats(s.own_rows, s.dv) / 4);
#pragma unroll 1
  for (int w = tid; w < s.B * heads; w += kThreads) {
    const int b = w / heads, x = w - b * heads;
    const Seq q = seq_of(b);
    const int full0 = q.nt[0] / c_own, full1 = q.nt[1] / c_own;
    int part = s.seq[b].own_part0 + x * s.seq[b].n_own;
    int full_at = s.seq[b].full0 + x * (full0 + full1);
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
      const int full = e ? full1 : full0, rest = (e ? q.nt[1] : q.nt[0]) - full * c_own;
      const int key0 = e ? q.key0[1] : q.key0[0], end = e ? q.end[1] : q.end[0];
#pragma unroll 1
      for (int y = 0; y < full + (rest != 0); ++y) {
        DenseUnit u;
        u.i0 = u.seq = b;
        u.n_i = 1;
        u.head0 = x * s.GH;  // (KV head x / n_hchunks, head chunk x % n_hchunks)
        u.key0 = key0 + y * c_own * 128;
        u.key1 = min(u.key0 + c_own * 128, end);
        u.part = s.own_part_at + part++ * part_step;
        u.batch_or_own = 1;
        s.units[y == full ? atomicAdd(&bucket_at[bucket(rest)], 1) : full_at++] = u;
      }
    }
  }
  const int unit_step = (int)(dense_part_floats(128, s.dv) / 4);
#pragma unroll 1
  for (int x = tid; x < n_prefix; x += kThreads) {
    int a = 0, z = n_groups;  // the last group that starts at or below x
    while (z - a > 1) {
      const int mid = (a + z) / 2;
      if (groups[mid].unit0 <= x) a = mid;
      else z = mid;
    }
    const DenseGroup& d = groups[a];
    const int y = (x - d.unit0) / d.n_splits, split = x - d.unit0 - y * d.n_splits;
    const int hc = y / d.tiles, tile = y - hc * d.tiles;
    DenseUnit u;
    u.i0 = d.first + tile * s.RPT;
    u.n_i = min(s.RPT, d.members - tile * s.RPT);
    u.head0 = hc * s.GH;
    u.seq = d.source;
    u.key0 = d.key_lo + split * c * 128;
    u.key1 = min(u.key0 + c * 128, d.prefix);
    u.part = x * unit_step;
    u.batch_or_own = 0;
    s.units[x] = u;
  }
}

}  // namespace

cudaError_t launch_shared_plan(const SharedPlan& s, cudaStream_t st) {
  // Barriers cost less with fewer warps, the units' records with more threads: at 8 items
  // (sequences times head chunks) 17.3 us a call with 256 threads and 18.4 with 1024, at 512
  // items 45.4 and 45.7, at 2048 items 197.5 and 193.5.
  const bool few = (long long)s.B * s.Hkv * s.n_hchunks <= 1024;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(few ? 256 : 1024);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return few ? cudaLaunchKernelEx(&cfg, shared_plan_kernel<256>, s) : cudaLaunchKernelEx(&cfg, shared_plan_kernel<1024>, s);
}

}  // namespace gqa
