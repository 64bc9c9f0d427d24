// plan_rows.cu -- the index arrays of a step, from the requests' lengths: block tables that grow
// from a list of free blocks and give back what they no longer need, the packed rows' starts,
// positions and slots, and the masks of drafted trees.
//
//   need_b = max(ceil((len_b + new_b) / bs), keep_b),  give_b = max(0, held_b - need_b),
//   take_b = max(0, need_b - held_b),  R = sum give
//   b is served where take_b = 0 or take_0 + .. + take_b <= free + R
//   the list is a stack: the R blocks given back go onto it, sequence by sequence, entries
//   ascending; the t-th block taken is the one at free + R - 1 - t
//
// Measured in replayed graphs: 256 sequences of one row 4.9 us, 128 trees of up to 64 rows 6.1, 48 prompts of up to
// 2,048 rows with too few blocks 6.1, 794 trees of seven rows 7.4; 4,096 sequences of one row 27. Where the state is
// written in place a second launch of one CTA does it: 6.4, 7.1 and 6.8 for the first three.
//
// What it reads and writes is small (20 bytes a sequence, 12 and more a row), so what bounds it is
// latency: one launch, and in it one chain of loads (the lengths, the block, the store). So no
// CTA waits for another: each scans all lengths for itself (and looks at all entries that are given
// back, below) and then writes what is its sequences' own, a warp or more for each (a CTA for each
// sequence had 794 of them of seven rows scan all lengths 794 times: 11 to 13 us). A block that is
// given back and taken in one call is not read from the list, where another CTA would be
// writing it, but found at its place in the table that gives it back, by a search over the
// prefix sums of give_b, which stay in shared memory. The list below `free` is only read, above
// it only written. Where a sequence has many rows they are cut into slices by grid y. A row's ancestors are indices
// that descend, so a thread that walks up from its row writes the words of the mask from the highest to the lowest
// and holds one at a time.

#include <atomic>
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace gqa {
namespace {

constexpr int kPlanRowsThreads = 256;
constexpr int kMany = 16, kLongs = 1024;            // of entries given back (below)

// What sequence b brings.
struct Req {
  int len, rows, held, need;  // need: held where nothing moves
  bool ok;                    // its numbers are in range
};
// out: a bit each for sequences that are out of range by other numbers (NULL: there are none).
__device__ __forceinline__ Req request(const PlanRows& p, int b, const uint32_t* out) {
  Req r;
  r.len = __ldg(p.lens + b);
  const int n = __ldg(p.new_rows + b);
  r.held = p.held_in[b];  // (may be the array that the state is written to)
  const int keep = p.keep ? __ldg(p.keep + b) : 0;
  const long long want = (long long)r.len + n;
  r.rows = max(n, 0);
  r.ok = r.len >= 0 && n >= 0 && n <= p.N && want <= (long long)p.mbps * p.bs && r.held >= 0 && r.held <= p.mbps &&
         keep >= 0 && keep <= r.held && (!p.parents || n <= 64ll * p.words) && !(out && out[b >> 5] >> (b & 31) & 1u);
  r.need = r.ok ? max((int)((want + p.bs - 1) / p.bs), keep) : r.held;
  return r;
}

// What a scan sums: rows, blocks wanted, blocks given back.
struct Sums {
  long long rows;
  int take, give;
};
// Exclusive prefix sums over the CTA and their totals. Ends with a barrier.
__device__ __forceinline__ void scan(Sums& v, Sums& total, Sums* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long r = __shfl_up_sync(0xffffffffu, x.rows, off);
    const int t = __shfl_up_sync(0xffffffffu, x.take, off), g = __shfl_up_sync(0xffffffffu, x.give, off);
    if (lane >= off) x = Sums{x.rows + r, x.take + t, x.give + g};
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  Sums before = {0, 0, 0};
  total = Sums{0, 0, 0};
#pragma unroll
  for (int w = 0; w < kPlanRowsThreads / 32; ++w) {
    const Sums s = sums[w];
    if (w < warp) before = Sums{before.rows + s.rows, before.take + s.take, before.give + s.give};
    total = Sums{total.rows + s.rows, total.take + s.take, total.give + s.give};
  }
  v = Sums{before.rows + x.rows - v.rows, before.take + x.take - v.take, before.give + x.give - v.give};
  __syncthreads();
}

// The mask of row i and its depth: up from the row, an ancestor at a time.
__device__ __forceinline__ int walk_up(const PlanRows& p, long long start, int i) {
  unsigned long long* out = p.mask + (start + i) * p.words;
  int at = i, word = p.words - 1, depth = 0;
  unsigned long long bits = 0;
  while (true) {
    while (word > at / 64) {  // (nothing further in this word)
      out[word--] = bits;
      bits = 0;
    }
    if (at < 64 * p.words) bits |= 1ull << (at & 63);
    const int up = __ldg(p.parents + start + at);
    if (up < 0 || up >= at) {
      if (up != -1) raise_error(p.err, kErrBounds);
      break;
    }
    at = up;
    ++depth;
  }
  for (; word >= 0; --word) {
    out[word] = bits;
    bits = 0;
  }
  return depth;
}

// A bit each for the sequences that give back an entry that is no block, and for those with rows from `cut` on.
__device__ __noinline__ void look_for_them(const PlanRows& p, int cut, uint32_t* out) {
  for (int i = threadIdx.x; i < (p.B + 31) / 32; i += kPlanRowsThreads) out[i] = 0;
  __syncthreads();
  for (int b = threadIdx.x / 16; b < p.B; b += kPlanRowsThreads / 16) {
    const Req r = request(p, b, nullptr);
    bool none = b >= cut && r.rows > 0;
    for (int k = r.need + (int)threadIdx.x % 16; k < r.held; k += 16)
      none |= (unsigned)__ldg(p.tables + (size_t)b * p.mbps + k) >= (unsigned)p.num_blocks;
    if (none) atomicOr(out + b / 32, 1u << (b & 31));
  }
}

// PER: sequences of a thread in a round of the scans. One where that takes a round or two (256 sequences of one row
// 4.9 us, with four 6.0), four where it would take more (1,024 of them 7.3 us, with one 8.9).
template <int PER>
__global__ void __launch_bounds__(kPlanRowsThreads) plan_rows_kernel(const PlanRows p) {
  constexpr int kPer = PER, kRound = kPlanRowsThreads * kPer, kFew = PER == 1 ? 8 : 4;
  __shared__ Sums sums[kPlanRowsThreads / 32];
  __shared__ int taken_s, n_longs, cut_s;
  __shared__ int2 longs[kLongs];  // sequences that give back more than kFew: where in the tables, how many
  extern __shared__ __align__(16) unsigned char dyn[];
  Sums* first = reinterpret_cast<Sums*>(dyn);       // before each of this CTA's sequences
  int* give0 = reinterpret_cast<int*>(first + p.per);  // [B + 1]
  uint32_t* out_s = reinterpret_cast<uint32_t*>(give0 + p.B + 1);
  if (threadIdx.x == 0) {
    n_longs = 0;
    cut_s = INT_MAX;
  }
  __syncthreads();
  // launched as a programmatic dependent: the lengths may come from the kernel before this one
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x;
  const int b_lo = (int)min((long long)blockIdx.x * p.per, (long long)p.B), b_hi = min(p.B, b_lo + p.per);
  const int free_raw = __ldg(p.free_in), free = min(max(free_raw, 0), p.num_blocks);
  // ---- all lengths, and all entries that are given back: one that is no block must not come onto the list, so its
  // sequence keeps all, and where the others' blocks lie on the list hangs on that. The thread that has the length of
  // a sequence that gives back a few reads them behind the scan; of those that give back more a half warp each does. If one
  // turns out to be no block, or the rows are more than N, such sequences are looked for and everything is summed up
  // without them. (128 requests of 256 that are over and give back 16,000 entries: 7.5 us, 5.0 without a look at them.)
  const uint32_t* out = nullptr;
  Sums total;  // (blocks wanted, whether served or not)
  bool bad = free_raw != free;
  const auto block_entry = [&](int e) { return (unsigned)e < (unsigned)p.num_blocks; };
#pragma unroll 1
  while (true) {
    total = Sums{0, 0, 0};
    bool found = false;
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += kRound) {
      const int b = b0 + tid * kPer;
      Sums of[kPer], v = {0, 0, 0}, sum;
      unsigned back[kPer][kFew];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        of[k] = Sums{0, 0, 0};
#pragma unroll
        for (int x = 0; x < kFew; ++x) back[k][x] = 0;
        if (b + k < p.B) {
          const Req r = request(p, b + k, out);
          bad |= !r.ok;
          of[k] = Sums{r.rows, max(0, r.need - r.held), max(0, r.held - r.need)};
          const int at = (b + k) * p.mbps + r.need, give = of[k].give;
#pragma unroll
          for (int x = 0; x < kFew; ++x)
            if (x < give) back[k][x] = (unsigned)__ldg(p.tables + at + x);
          if (give > kFew && !out) {
            const int to = atomicAdd(&n_longs, 1);
            if (to < kLongs) longs[to] = make_int2(at + kFew, give - kFew);
            else
              for (int x = kFew; x < give; ++x) found |= !block_entry(__ldg(p.tables + at + x));
          }
        }
        v = Sums{v.rows + of[k].rows, v.take + of[k].take, v.give + of[k].give};
      }
      scan(v, sum, sums);
      v = Sums{v.rows + total.rows, v.take + total.take, v.give + total.give};
      unsigned most = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (b + k < p.B) give0[b + k] = v.give;
        if (b + k >= b_lo && b + k < b_hi) first[b + k - b_lo] = v;
        if (of[k].rows > 0 && v.rows + of[k].rows > p.N) atomicMin(&cut_s, b + k);
        v = Sums{v.rows + of[k].rows, v.take + of[k].take, v.give + of[k].give};
#pragma unroll
        for (int x = 0; x < kFew; ++x) most = max(most, back[k][x]);
      }
      found |= most >= (unsigned)p.num_blocks;
      total = Sums{total.rows + sum.rows, total.take + sum.take, total.give + sum.give};
    }
    if (tid == 0) {
      give0[p.B] = total.give;
      taken_s = 0;
    }
    if (!out) {  // (the scan ends with a barrier: they are all noted)
#pragma unroll 1
      for (int i = tid / 16; i < min(n_longs, kLongs); i += kPlanRowsThreads / 16) {
        const int2 l = longs[i];
#pragma unroll 1
        for (int k = tid % 16; k < l.y; k += 16 * kMany) {
          unsigned e[kMany], most = 0;
#pragma unroll
          for (int x = 0; x < kMany; ++x) e[x] = k + 16 * x < l.y ? (unsigned)__ldg(p.tables + l.x + k + 16 * x) : 0;
#pragma unroll
          for (int x = 0; x < kMany; ++x) most = max(most, e[x]);
          found |= most >= (unsigned)p.num_blocks;
        }
      }
    }
    if (!__syncthreads_or(found || total.rows > p.N) || out) break;
    look_for_them(p, cut_s, out_s);
    out = out_s;
    __syncthreads();
  }
  const long long room = (long long)free + total.give;  // blocks that can be taken
  bad |= room > p.num_blocks || total.rows > p.N;
  // ---- blocks that are taken: all that are wanted, or as many as the sequences served take
  int taken = (int)min((long long)total.take, room);
  const bool state_only = !p.write_rows;  // (one CTA)
  if (total.take > room || state_only) {
    int before = 0, most = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += kRound) {
      const int b = b0 + tid * kPer;
      int take[kPer], need[kPer], held[kPer];
      Sums v = {0, 0, 0}, sum;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        take[k] = need[k] = held[k] = 0;
        if (b + k < p.B) {
          const Req r = request(p, b + k, out);
          need[k] = r.need;
          held[k] = r.held;
          take[k] = max(0, r.need - r.held);
        }
        v.take += take[k];
      }
      scan(v, sum, sums);  // (its barriers: everyone has read before anyone writes)
      v.take += before;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        v.take += take[k];
        const bool served = take[k] == 0 || v.take <= room;
        if (served && take[k]) most = v.take;
        if (state_only && b + k < p.B) p.held_out[b + k] = served ? need[k] : held[k];
      }
      before += sum.take;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if ((tid & 31) == 0) atomicMax(&taken_s, most);
    __syncthreads();
    taken = taken_s;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    if (__syncthreads_or(bad) && tid == 0 && p.report) raise_error(p.err, kErrBounds);
    if (p.write_state && tid == 0) {  // (every thread has read the count)
      p.free_out[0] = (int)min(room - taken, (long long)p.num_blocks);
      p.free_out[1] = total.take - taken;
    }
  }
  if (!p.write_rows) return;
  // ---- this CTA's sequences, `lanes` threads each
  const int lanes = p.lanes, part = (int)blockIdx.y, parts = (int)gridDim.y;
  const int step = parts * lanes, at0 = part * lanes + tid % lanes;
  // the block at place `at` of the list with what is given back
  const auto listed = [&](long long at) -> int {
    if (at < free) return __ldg(p.free_list + at);
    const int g = (int)(at - free);
    int lo = 0, hi = p.B;  // give0[lo] <= g < give0[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (give0[mid] <= g) lo = mid;
      else hi = mid;
    }
    const Req r = request(p, lo, out);
    return __ldg(p.tables + (size_t)lo * p.mbps + r.need + (g - give0[lo]));
  };
#pragma unroll 1
  for (int b = b_lo + tid / lanes; b < b_hi; b += kPlanRowsThreads / lanes) {
    const Req r = request(p, b, out);
    const long long start = first[b - b_lo].rows;
    const int took = first[b - b_lo].take;
    const int take = max(0, r.need - r.held), give = max(0, r.held - r.need);
    const bool served = r.ok && (take == 0 || (long long)took + take <= room);
    int* table = p.tables + (size_t)b * p.mbps;
    if (at0 == 0) {
      if (p.write_state) p.held_out[b] = served ? r.need : r.held;
      p.row_starts[b] = (int)min(start, (long long)INT_MAX);
      if (b == p.B - 1) p.row_starts[p.B] = (int)min(start + r.rows, (long long)INT_MAX);
    }
    const auto block = [&](int k) {  // of the sequence's k-th block; -1: none
      const int e = k < r.held ? __ldg(table + k) : listed(room - 1 - ((long long)took + (k - r.held)));
      if (e >= 0 && e < p.num_blocks) return e;
      raise_error(p.err, kErrBounds);
      return -1;
    };
    // blocks given back, those of them that stay on the list
    for (int k = at0; k < give; k += step) {
      const int g = give0[b] + k, e = __ldg(table + r.need + k);
      if (free + (long long)g < room - taken && free + (long long)g < p.num_blocks) p.free_list[free + g] = e;
    }
    // (what a sequence that is not served wanted: -1, not a block of before that another has by now)
    for (int k = at0; k < take; k += step) table[r.held + k] = served ? block(r.held + k) : -1;
    // rows
    const int rows = (int)min((long long)r.rows, max(0ll, p.N - start));
    for (int i = at0; i < rows; i += step) {
      long long slot = -1;
      if (served) {
        const int k = (r.len + i) / p.bs, e = block(k);
        if (e >= 0) slot = (long long)e * p.bs + (r.len + i - k * p.bs);
      }
      p.slots[start + i] = slot;
      int at = i;
      if (p.parents) at = walk_up(p, start, i);
      p.positions[start + i] = r.len + at;
    }
  }
  // ---- rows behind the last sequence
  const long long threads = (long long)gridDim.x * parts * kPlanRowsThreads;
  for (long long n = total.rows + ((long long)blockIdx.x * parts + part) * kPlanRowsThreads + tid; n < p.N; n += threads) {
    p.slots[n] = -1;
    p.positions[n] = 0;
    if (p.parents)
      for (int w = 0; w < p.words; ++w) p.mask[n * p.words + w] = 0;
  }
}

}  // namespace

cudaError_t launch_plan_rows(PlanRows p, cudaStream_t st) {
  int dev = 0;
  cudaGetDevice(&dev);
  static std::atomic<unsigned long long> attr_done{0};  // per device
  const auto kernel = p.B <= 2 * kPlanRowsThreads ? plan_rows_kernel<1> : plan_rows_kernel<4>;
  if (dev >= 64 || !(attr_done.load(std::memory_order_acquire) >> dev & 1ull)) {
    for (const auto k : {plan_rows_kernel<1>, plan_rows_kernel<4>}) {
      const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kPlanRowsMaxB * 5 + 64 * 1024);
      if (e != cudaSuccess) return e;
    }
    if (dev < 64) attr_done.fetch_or(1ull << dev, std::memory_order_release);
  }
  // a warp for a sequence, up to a CTA where sequences have that many rows (slices of them beyond that); up
  // to two CTAs an SM, since each scans all lengths
  const long long rows = (long long)p.N / p.B;
  p.lanes = 32;
  while (p.lanes < kPlanRowsThreads && p.lanes < rows) p.lanes *= 2;
  const int each = kPlanRowsThreads / p.lanes, most = 2 * kDenseSms;
  const int groups = (p.B + each - 1) / each;
  p.per = each * ((groups + most - 1) / most);
  const int gx = (p.B + p.per - 1) / p.per;
  const long long slices = (rows + kPlanRowsThreads - 1) / kPlanRowsThreads;
  const int gy = slices <= 1 ? 1 : slices < most / gx ? (int)slices : most / gx < 1 ? 1 : most / gx;
  const size_t smem = (size_t)p.per * sizeof(Sums) + (size_t)(p.B + 1) * 4 + (size_t)(p.B + 31) / 32 * 4;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)gx, (unsigned)gy);
  cfg.blockDim = dim3(kPlanRowsThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // every CTA reads the blocks held and the count of free ones: written in the same launch only
  // to other arrays, else by one CTA of a second one
  const bool same = p.held_in == p.held_out || p.free_in == p.free_out;
  p.write_rows = 1;
  p.write_state = !same;
  p.report = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess || !same) return e;
  p.write_rows = 0;
  p.write_state = 1;
  p.report = 0;
  cfg.gridDim = dim3(1);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace gqa
