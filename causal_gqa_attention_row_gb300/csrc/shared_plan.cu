// shared_plan.cu -- the plan of a shared-prefix decode step, by one CTA: which sequences
// have a prefix to share (groups of two members or more), and the list of units that
// dense_tc_kernel works off, the prefixes' first, then those of the sequences' own keys.
//
// The prefix of group g is tiles_g row tiles per KV head (and head chunk) times n_g key
// tiles; the own keys of a sequence are one row tile per KV head (and head chunk). Units
// take c key tiles each, c the same for all and chosen to minimise
//   max(ceil(prefix units / slots) * (c + kDenseUnitTiles), (all tiles + units * kDenseUnitTiles) / slots) + c / 4,
// in key tiles: the rounds that the prefixes' equal units take on the slots (units worked on
// at a time), in whose last round own units fill the rest, or all work spread evenly; and
// something for the longest unit, which the rest may have to wait for.
// Every candidate c is tried, a thread each. Own units are listed longest first.
//
// The other kernels wait for this one, so its round trips to memory count: groups, their
// bounds and the lengths are read at once, and up to kPlanGroups groups stay in shared memory.
#include "common.cuh"
#include "internal.h"

namespace gqa {
namespace {

constexpr int kThreads = 1024;
constexpr int kPlanGroups = 128;
constexpr int kBuckets = 64;
constexpr int kMostTiles = 1 << 20;  // candidates for c

// Exclusive prefix sum over the CTA; `total` receives the sum. Ends with a barrier.
__device__ __forceinline__ int exclusive_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int w = warp_sums[lane];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, off);
    if (lane >= off) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = warp == 0 ? 0 : __shfl_sync(0xffffffffu, w, warp - 1);
  __syncthreads();
  return before + x - v;
}

// CTA-wide minimum and sum of 64-bit values (shuffles, then one value a warp: 64-bit
// atomics on one shared word by every thread took the kernel 10 us). Ends with a barrier.
__device__ __forceinline__ unsigned long long block_min(unsigned long long v, unsigned long long* warps) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    const unsigned long long o = __shfl_xor_sync(0xffffffffu, v, off);
    v = o < v ? o : v;
  }
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  v = warps[threadIdx.x & 31];
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    const unsigned long long o = __shfl_xor_sync(0xffffffffu, v, off);
    v = o < v ? o : v;
  }
  __syncthreads();
  return v;
}
__device__ __forceinline__ unsigned long long block_sum(unsigned long long v, unsigned long long* warps) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  v = warps[threadIdx.x & 31];
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(kThreads) shared_plan_kernel(const SharedPlan s) {
  __shared__ int warp_sums[32];
  __shared__ int bucket_at[kBuckets];
  __shared__ int bad, bad_len, max_tiles;
  __shared__ unsigned long long warp_values[32];
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
    d.prefix = nb;
    d.kv_hi = 0;            // largest length of a member ...
    d.key_lo = s.capacity;  // ... and the smallest
    groups[g] = d;
  }
  const int len0 = tid < s.B ? s.seq_lens[tid] : 0;
  // the length of sequence b, 0 if it is out of range
  const auto length = [&](int b) {
    const int n = b == tid ? len0 : s.seq_lens[b];
    return n >= 1 && n <= s.capacity ? n : 0;
  };
  for (int b = tid; b < s.B; b += kThreads)
    if (length(b) == 0) bad_len = 1;
  __syncthreads();
  const bool ok = !bad;
  if ((bad || bad_len) && tid == 0) raise_error(s.err, kErrBounds);
  const auto find = [&](int b) {  // the group of sequence b, -1 without one
    if (!ok || s.n_groups == 0 || b < groups[0].first) return -1;
    int lo = 0, hi = s.n_groups;  // first[lo] <= b < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (groups[mid].first <= b) lo = mid;
      else hi = mid;
    }
    return b < groups[lo].first + groups[lo].members ? lo : -1;
  };
  for (int b0 = 0; b0 < s.B; b0 += kThreads) {
    const int b = b0 + tid, len = b < s.B ? length(b) : 0, g = len ? find(b) : -1;
    // (most warps hold members of one group: one atomic a warp then)
    if (__all_sync(0xffffffffu, g == __shfl_sync(0xffffffffu, g, 0))) {
      const int most = __reduce_max_sync(0xffffffffu, len), least = __reduce_min_sync(0xffffffffu, len);
      if (g >= 0 && (tid & 31) == 0) {
        atomicMax(&groups[g].kv_hi, most);
        atomicMin(&groups[g].key_lo, least);
      }
    } else if (g >= 0) {
      atomicMax(&groups[g].kv_hi, len);
      atomicMin(&groups[g].key_lo, len);
    }
  }
  __syncthreads();
  for (int g = tid; g < s.n_groups; g += kThreads) {
    DenseGroup d = groups[g];
    d.prefix = ok && d.members >= 2 ? d.prefix * s.bs : 0;
    d.kv_hi = min(d.prefix, d.kv_hi);
    // tiles that every member's window hides are left out
    d.key_lo = first_visible_key(d.key_lo - 1, s.window) / 128 * 128;
    const int nt = (d.kv_hi - d.key_lo + 127) / 128;
    if (nt <= 0) d.kv_hi = d.prefix = 0;
    d.n_splits = max(nt, 0);
    d.tiles = nt > 0 ? (d.members + s.RPT - 1) / s.RPT : 0;
    groups[g] = d;
    if (nt > 0) atomicMax(&max_tiles, nt);
  }
  __syncthreads();
  // ---- own keys [key0, key0 + n) of sequence b, key0 on a block's boundary
  const auto own_keys = [&](int b, int& key0) {
    const int g = find(b), len = length(b);
    key0 = max(g < 0 ? 0 : groups[g].prefix, first_visible_key(len - 1, s.window) / s.bs * s.bs);
    return max(len - key0, 0);
  };
  const int heads = s.Hkv * s.n_hchunks;
  unsigned long long mine_own = 0;
  int longest = 0;
  for (int b = tid; b < s.B; b += kThreads) {
    int key0;
    const int nt = (own_keys(b, key0) + 127) / 128;
    mine_own += (unsigned long long)nt * heads;
    longest = max(longest, nt);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (longest > 1 && (tid & 31) == 0) atomicMax(&max_tiles, longest);
  // ---- c
  const long long own_tiles = (long long)block_sum(mine_own, warp_values), own_items = (long long)s.B * heads;
  const long long c_own_least = (own_tiles + kOwnExtra - 1) / kOwnExtra;  // own parts <= items + kOwnExtra
  const int c_most = min(max_tiles, kMostTiles);
  unsigned long long mine_best = ~0ull;
  for (int c = 1 + tid; c <= c_most; c += kThreads) {
    long long units = 0, tiles = 0;
    for (int g = 0; g < s.n_groups; ++g) {
      const long long t = (long long)heads * groups[g].tiles;
      units += t * ((groups[g].n_splits + c - 1) / c);
      tiles += t * groups[g].n_splits;
    }
    if (units > s.max_prefix_units) continue;
    const long long rounds = (units + s.slots - 1) / s.slots * (c + kDenseUnitTiles);
    const long long even =
        (tiles + own_tiles + (units + own_tiles / max((long long)c, c_own_least) + own_items / 2) * kDenseUnitTiles) /
        s.slots;
    // a quarter of a unit for the tail that one leaves behind; ties go to the longer units
    const long long cost = 4 * max(rounds, even) + c;
    const unsigned long long key = (unsigned long long)cost << 24 | (unsigned)(kMostTiles - c);
    mine_best = key < mine_best ? key : mine_best;
  }
  const unsigned long long best = block_min(mine_best, warp_values);
  // (the largest c always fits: the caller sized max_prefix_units for it)
  const int c = best == ~0ull ? c_most : kMostTiles - (int)(best & 0xffffff);
  const int c_own = (int)max((long long)c, max(c_own_least, 1ll));
  // ---- key ranges per group and where its units start
  const int per = (s.n_groups + kThreads - 1) / kThreads;
  const int lo = min(s.n_groups, tid * per), hi = min(s.n_groups, lo + per);
  int mine = 0;
  for (int g = lo; g < hi; ++g) {
    DenseGroup& d = groups[g];
    d.n_splits = (d.n_splits + c - 1) / c;
    mine += heads * d.tiles * d.n_splits;
  }
  int n_prefix;
  int at = exclusive_scan(mine, warp_sums, n_prefix);
  for (int g = lo; g < hi; ++g) {
    DenseGroup& d = groups[g];
    d.unit0 = at;
    at += heads * d.tiles * d.n_splits;
  }
  // ---- own parts: of c_own tiles, the last of a sequence shorter
  const auto own_parts = [&](int b, int& key0, int& rest) {  // rest: tiles of the last one if not c_own
    const int nt = (own_keys(b, key0) + 127) / 128;
    rest = nt % c_own;
    return (nt + c_own - 1) / c_own;
  };
  const auto bucket = [&](int rest) {
    return min((int)((long long)(c_own - rest) * kBuckets / c_own), kBuckets - 1);
  };
  const int per_b = (s.B + kThreads - 1) / kThreads;
  const int b_lo = min(s.B, tid * per_b), b_hi = min(s.B, b_lo + per_b);
  int mine_parts = 0, mine_full = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    int key0, rest;
    const int n = own_parts(b, key0, rest);
    mine_parts += n * heads;
    mine_full += (n - (rest != 0)) * heads;
    if (rest) atomicAdd(&bucket_at[bucket(rest)], heads);
  }
  int n_parts, n_full;
  int part_at = exclusive_scan(mine_parts, warp_sums, n_parts);  // (its barriers: unit0 and the buckets are in place)
  int full_at = n_prefix + exclusive_scan(mine_full, warp_sums, n_full);
  if (tid < 32) {  // where the buckets start, two a lane
    const int x = bucket_at[2 * tid], y = bucket_at[2 * tid + 1];
    int sum = x + y;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, off);
      if (tid >= off) sum += up;
    }
    bucket_at[2 * tid] = n_prefix + n_full + sum - x - y;
    bucket_at[2 * tid + 1] = n_prefix + n_full + sum - y;
    if (tid == 31) {
      s.units_listed[0] = n_prefix + n_full + sum;
      s.units_listed[1] = 0;  // the ticket counter
    }
  }
  __syncthreads();
  const int part_step = (int)(dense_part_floats(s.own_rows, s.dv) / 4);
  for (int b = b_lo; b < b_hi; ++b) {
    int key0, rest;
    const int n = own_parts(b, key0, rest), len = length(b);
    SeqPlan q = {};
    q.n_own = n;
    q.own_part0 = part_at;
    const int g = len ? find(b) : -1;
    if (g >= 0 && groups[g].prefix > 0) {
      const DenseGroup d = groups[g];
      const int i = b - d.first;
      q.n_pre = d.n_splits;
      q.pre_unit0 = d.unit0 + i / s.RPT * d.n_splits;
      q.pre_stride = d.tiles * d.n_splits;
      q.row0 = i % s.RPT * s.GH;
    }
    s.seq[b] = q;
    int rest_at = rest ? atomicAdd(&bucket_at[bucket(rest)], heads) : 0;
    for (int x = 0; x < heads; ++x)
      for (int y = 0; y < n; ++y) {
        DenseUnit u;
        u.i0 = u.seq = b;
        u.n_i = 1;
        u.head0 = x * s.GH;  // (KV head x / n_hchunks, head chunk x % n_hchunks)
        u.key0 = key0 + y * c_own * 128;
        u.key1 = min(u.key0 + c_own * 128, len);
        u.part = s.own_part_at + part_at * part_step;
        u.batch_or_own = 1;
        ++part_at;
        s.units[y == n - 1 && rest ? rest_at++ : full_at++] = u;
      }
  }
  const int unit_step = (int)(dense_part_floats(128, s.dv) / 4);
  for (int x = tid; x < n_prefix; x += kThreads) {
    int a = 0, z = s.n_groups;  // the last group that starts at or below x
    while (z - a > 1) {
      const int mid = (a + z) / 2;
      if (groups[mid].unit0 <= x) a = mid;
      else z = mid;
    }
    const DenseGroup d = groups[a];
    int y = x - d.unit0;
    const int split = y % d.n_splits;
    y /= d.n_splits;
    const int tile = y % d.tiles;
    DenseUnit u;
    u.i0 = d.first + tile * s.RPT;
    u.n_i = min(s.RPT, d.members - tile * s.RPT);
    u.head0 = y / d.tiles * s.GH;
    u.seq = d.first;
    u.key0 = d.key_lo + split * c * 128;
    u.key1 = min(u.key0 + c * 128, d.kv_hi);
    u.part = x * unit_step;
    u.batch_or_own = 0;
    s.units[x] = u;
  }
}

}  // namespace

cudaError_t launch_shared_plan(const SharedPlan& s, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_plan_kernel, s);
}

}  // namespace gqa
