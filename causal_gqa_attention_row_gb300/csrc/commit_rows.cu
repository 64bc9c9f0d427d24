// commit_rows.cu -- the rows of an accepted path moved together behind a sequence's history, in
// all layers' pools: row len + path[j] to row len + j, path ascending.
//
// The row at place j comes from place path[j] >= j, so what a row overwrites is never wanted by a
// later one: in ascending order nothing is lost, and a thread that owns the same 16 bytes of every
// row needs no other thread. It has eight rows in flight: all loaded, then all stored. A CTA takes
// one sequence in one layer's keys or values; every CTA checks the whole path and its table
// entries before it moves a row. Latency bounds the small calls (path, table entry, row: three
// trips), HBM the large ones. Measured: one sequence, one layer 2.6 us; 64 sequences of up to 8 rows, 28 layers of
// 8 heads of 128 8.4 us (3.5 TB/s of rows read and written).

#include "common.cuh"
#include "internal.h"

namespace gqa {
namespace {

constexpr int kCommitThreads = 128;
constexpr int kCommitStage = 128;  // rows of a path whose places are worked out at a time

__global__ void __launch_bounds__(kCommitThreads) commit_rows_kernel(const __grid_constant__ CommitRows p) {
  __shared__ long long from_s[kCommitStage], to_s[kCommitStage];  // pool rows of KV head 0 (from: -1: stays)
  grid_dep_wait();
  grid_dep_launch();
  const int b = blockIdx.x, tid = threadIdx.x;
  const int len = p.lens_in[b], n = __ldg(p.n_path + b);
  const int s0 = __ldg(p.row_starts + b), s1 = __ldg(p.row_starts + b + 1);
  const long long rows = (long long)s1 - s0, cap = (long long)p.mbps * p.bs;
  bool bad = len < 0 || n < 0 || n > p.max_path || rows < 0 || n > rows || len + rows > cap;
  const int* path = p.path + (size_t)b * p.max_path;
  const int* table = p.tables + (size_t)b * p.mbps;
  const int count = bad ? 0 : n;
  for (int j = tid; j < count; j += kCommitThreads) {
    const int x = __ldg(path + j), before = j > 0 ? __ldg(path + j - 1) : -1;
    const bool in = x > before && x < rows;  // (ascending, so x >= j)
    bad |= !in;
    if (in && x >= j) {
      const int e = __ldg(table + (len + x) / p.bs), f = __ldg(table + (len + j) / p.bs);
      bad |= e < 0 || e >= p.num_blocks || f < 0 || f >= p.num_blocks;
    }
  }
  bad = __syncthreads_or(bad);
  if (p.lens_only || (!p.lens_later && blockIdx.y == 0)) {
    if (tid == 0) {
      if (bad) raise_error(p.err, kErrBounds);
      p.lens_out[b] = bad ? len : len + n;  // (every thread has read the length)
    }
    if (p.lens_only) return;
  }
  if (bad) return;
  const int layer = (int)blockIdx.y >> 1, value = (int)blockIdx.y & 1;
  char* pool = static_cast<char*>(value ? p.v_pools[layer] : p.k_pools[layer]);
  if (!pool) return;
  const int row_bytes = value ? p.v_bytes : p.k_bytes, cpr = row_bytes / 16;
  for (int j0 = 0; j0 < n; j0 += kCommitStage) {
    const int here = min(kCommitStage, n - j0);
    __syncthreads();
    for (int j = tid; j < here; j += kCommitThreads) {
      const int to = len + j0 + j, x = __ldg(path + j0 + j), of = len + x;
      from_s[j] = x == j0 + j ? -1 : (long long)__ldg(table + of / p.bs) * p.Hkv * p.bs + of % p.bs;
      to_s[j] = (long long)__ldg(table + to / p.bs) * p.Hkv * p.bs + to % p.bs;
    }
    __syncthreads();
    for (int c = tid; c < p.Hkv * cpr; c += kCommitThreads) {
      const int h = c / cpr;
      char* at = pool + (long long)h * p.bs * row_bytes + (c - h * cpr) * 16;
      for (int j = 0; j < here; j += 8) {
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (j + u < here && from_s[j + u] >= 0) v[u] = *reinterpret_cast<const uint4*>(at + from_s[j + u] * row_bytes);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (j + u < here && from_s[j + u] >= 0) *reinterpret_cast<uint4*>(at + to_s[j + u] * row_bytes) = v[u];
      }
    }
  }
}

}  // namespace

cudaError_t launch_commit_rows(const CommitRows& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.B, p.lens_only ? 1u : 2u * (unsigned)p.n_layers);
  cfg.blockDim = dim3(kCommitThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, commit_rows_kernel, p);
}

}  // namespace gqa
