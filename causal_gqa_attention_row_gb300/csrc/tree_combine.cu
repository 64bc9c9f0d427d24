// tree_combine.cu -- joins the partial results of drafted rows (tree_part.cuh), in the order of their slots:
//   M = max m_s (and the sink logit),  out = sum 2^(m_s - M) o_s / sum 2^(m_s - M) l_s
//
// A CTA takes rows of one row tile (drafted row, head), next to one another in the parts, rows along the
// lanes: rows by d_v / 4 threads of four columns by `shares` of the parts (several where few rows
// would leave SMs without work), four parts at a time, the shares joined at the end in their order; where a tile
// has one or two parts, two groups of rows at a time instead. Latency bounds it, so a CTA goes on
// through its tile's rows: one trip to memory for the tile's record, which the kernel before has written, then one
// for each two groups. Measured: 2,059 rows of 32 heads, 60% of them in parts, 12 us; four sequences of eight rows 3.7.
// (A CTA for each group of eight rows took 84 us for the former; with a row's place worked out here, by two 64-bit
// divisions a thread, 116.)
//
// Values that a row does not see. A product with V on the tensor cores mixes all keys of a tile, and 0 * NaN is
// NaN: an infinity or NaN in one drafted row's value (or in a history row that the window has left for
// some rows) would reach rows that do not see it. That cannot happen without a result that is not
// finite, so a CTA that has written one looks at the values that its row does not see, and if one of them is not finite
// works the row out again from the keys that it does see, a warp a key. (Looking over
// the values of every tile with drafted rows would have cost all calls.) That is a last resort, a row after the other
// in its tile's CTAs: an infinity in the value of one drafted row that 28 rows behind 5,315 keys do not see (32 heads on 8
// of 128) takes the call from 160 us to 104 ms, one behind 32,000 keys that 15 rows do not see from 32 us to 16 ms; one
// that all rows see 310 us, for the look. Rows whose own scores hold no number are left as they are: a sequence whose
// queries, keys and values are all NaN costs nothing (it took 108 ms while such rows were looked at too).

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "tree_part.cuh"

namespace gqa {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kJoinCtas = 4;  // an SM, about, that a tile's rows are cut for (8, 12: the same, 20: 2 us more)

__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ bool finite4(float4 v) {
  // (an infinity or NaN times zero is NaN)
  const float z = fmaf(v.x, 0.f, fmaf(v.y, 0.f, fmaf(v.z, 0.f, v.w * 0.f)));
  return z == 0.f;
}

// Whether drafted row i of a sequence sees key `key`, which lies at or behind the sequence's first.
struct Row {
  int row, i, n, row0, hist, depth;
};
__device__ __forceinline__ bool sees(const TreeWork& w, const Row& r, int key) {
  const int j = key - r.hist;
  if (j < 0) return w.window <= 0 || key > r.hist + r.depth - 1 - w.window;
  if (!(tree_bits(w, r.row, r.i, r.n, j) & 1u)) return false;
  return w.window <= 0 || tree_depth(w, r.row0 + j, j, r.n) > r.depth - w.window;
}

// The pool row of a key (of KV head kvh), -1 for an entry that is no block.
__device__ __forceinline__ long long pool_row_of(const TreeParams& p, int b, int kvh, int key) {
  const int e = __ldg(p.tables + (size_t)b * p.mbps + key / p.w.bs);
  return e >= 0 && e < p.num_blocks ? ((long long)e * p.Hkv + kvh) * p.w.bs + key % p.w.bs : -1;
}

// Row r of head h worked out from the keys that it sees, by the CTA, if a value that it does not see is not
// finite. (The caller has a barrier before and after.)
__device__ __noinline__ void row_again(const TreeParams& p, int b, const Row& r, int h, float* s_o, float2* s_ml) {
  const TreeWork& w = p.w;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dk = p.dk, dv = p.dv, kvh = h / p.G;
  const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16*>(p.k), *vp = static_cast<const __nv_bfloat16*>(p.v);
  const int first = first_visible_key(r.hist, w.window), end = r.hist + r.n;
  const int own = min(first_visible_key(r.hist + r.depth - 1, w.window), r.hist);
  bool bad = false;
  const auto look = [&](int key) {
    if (sees(w, r, key)) return;
    const long long at = pool_row_of(p, b, kvh, key);
    if (at < 0) return;
    for (int d = lane; d < dv; d += 32) bad |= !(fabsf(__bfloat162float(vp[at * dv + d])) <= 3.4e38f);
  };
  for (int key = first + warp; key < own; key += kJoinThreads / 32) look(key);
  for (int key = r.hist + warp; key < end; key += kJoinThreads / 32) look(key);
  if (!__syncthreads_or(bad)) return;
  constexpr int kMost = 8;  // columns of a lane
  float q[kMost], o[kMost], m = -INFINITY, l = 0.f;
  const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(p.q) + ((size_t)r.row * p.H + h) * dk;
#pragma unroll
  for (int e = 0; e < kMost; ++e) {
    q[e] = lane + 32 * e < dk ? __bfloat162float(qr[lane + 32 * e]) : 0.f;
    o[e] = 0.f;
  }
  for (int key = own + warp; key < end; key += kJoinThreads / 32) {
    if (!sees(w, r, key)) continue;
    const long long at = pool_row_of(p, b, kvh, key);
    if (at < 0) continue;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kMost; ++e)
      if (lane + 32 * e < dk) s = fmaf(q[e], __bfloat162float(kp[at * dk + lane + 32 * e]), s);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= p.qscale;
    if (p.softcap2 > 0.f) s = p.softcap2 * (1.f - 2.f / (exp2_of(s * (2.8853900817779268f / p.softcap2)) + 1.f));
    if (p.alibi) {
      const int j = key - r.hist, at_key = j < 0 ? key : r.hist + tree_depth(w, r.row0 + j, j, r.n) - 1;
      s = fmaf(__ldg(p.alibi + h) * kLog2e, (float)(at_key - (r.hist + r.depth - 1)), s);
    }
    const float mn = fmaxf(m, s), c = mn == -INFINITY ? 0.f : mn;
    const float f = exp2_of(m - c), x = exp2_of(s - c);
    m = mn;
    l = fmaf(l, f, x);
#pragma unroll
    for (int e = 0; e < kMost; ++e)
      if (lane + 32 * e < dv)
        o[e] = x == 0.f ? o[e] * f : fmaf(x, __bfloat162float(vp[at * dv + lane + 32 * e]), o[e] * f);
  }
#pragma unroll
  for (int e = 0; e < kMost; ++e)
    if (lane + 32 * e < dv) s_o[warp * dv + lane + 32 * e] = o[e];
  if (lane == 0) s_ml[warp] = make_float2(m, l);
  __syncthreads();
  for (int d = threadIdx.x; d < dv; d += kJoinThreads) {
    const float z2 = p.sinks ? __ldg(p.sinks + h) * kLog2e : -INFINITY;
    float M = z2;
    for (int x = 0; x < kJoinThreads / 32; ++x) M = fmaxf(M, s_ml[x].x);
    float den = M != -INFINITY && p.sinks ? exp2_of(z2 - M) : 0.f, acc = 0.f;
    for (int x = 0; x < kJoinThreads / 32; ++x) {
      if (s_ml[x].y == 0.f) continue;
      const float f = exp2_of(s_ml[x].x - M);
      den = fmaf(f, s_ml[x].y, den);
      acc = fmaf(f, s_o[x * dv + d], acc);
    }
    static_cast<__nv_bfloat16*>(p.out)[((size_t)r.row * p.H + h) * dv + d] =
        __float2bfloat16_rn(den != 0.f ? acc / den : 0.f);
  }
}

// CHECK: the parts come from the tensor cores (above).
template <typename ET, bool CHECK>
__global__ void __launch_bounds__(kJoinThreads) tree_combine_kernel(const __grid_constant__ TreeParams p, int shares) {
  __shared__ float4 acc_s[CHECK ? 2 * kJoinThreads : kJoinThreads];  // (row_again: eight rows of up to 256 columns)
  __shared__ float2 md_s[kJoinThreads];
  __shared__ uint32_t again_s[4];  // rows of the tile (at most 128) to be worked out again
  if (CHECK) {
    if (threadIdx.x < 4) again_s[threadIdx.x] = 0;
    __syncthreads();
  }
  grid_dep_wait();
  const TreeWork& w = p.w;
  const int dv = p.dv, rows_here = 1024 / dv / shares;  // powers of two, as dv is
  const int tid = threadIdx.x, rr = tid & (rows_here - 1), c = tid / rows_here % (dv / 4);
  const int share = tid / (kJoinThreads / shares);
  const int tiles = __ldcg(w.line);
  const int4 r0 = __ldcg(reinterpret_cast<const int4*>(w.rec + blockIdx.x));
  const int4 r1 = __ldcg(reinterpret_cast<const int4*>(w.rec + blockIdx.x) + 1);
  if ((int)blockIdx.x >= tiles) return;  // as many row tiles as there may be are launched
  const int rows = r0.y * w.GH, total = r1.y;
  if (total == 0) {  // written whole
    const uint32_t odd = CHECK && blockIdx.y == 0 ? __ldcg(reinterpret_cast<const uint32_t*>(w.odd) + blockIdx.x) : 0;
    if (odd == 0) return;
    if (CHECK && tid < 4 && (odd >> 8 * tid & 0xff) && rows > 32 * tid)
      again_s[tid] = rows - 32 * tid >= 32 ? ~0u : (1u << (rows - 32 * tid)) - 1u;
  }
  const size_t part = dense_part_floats(w.R, dv), next = part * r1.z;
  const float* parts = p.partial + part * r1.x;
  // part s of row x: its maximum, sum and this thread's columns
  const auto fetch = [&](int s, int x, float& m, float& l, float4& o) {
    m = -INFINITY;
    l = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (s < total && x < rows) {
      const float* u = parts + s * next;
      m = __ldcg(u + w.R * dv + x);
      l = __ldcg(u + w.R * dv + w.R + x);
      o = __ldcg(reinterpret_cast<const float4*>(u) + c * w.R + x);
    }
  };
  const auto join = [](float m, float l, float4 o, float M, float& den, float4& acc) {
    if (l == 0.f) return;  // no visible key, whatever m and o hold (a NaN in l goes through)
    const float f = exp2_of(m - M);
    den = fmaf(f, l, den);
    acc = make_float4(fmaf(f, o.x, acc.x), fmaf(f, o.y, acc.y), fmaf(f, o.z, acc.z), fmaf(f, o.w, acc.w));
  };
  // x / GH, exact for x and GH up to 128 (a division each took a good third of the kernel's instructions)
  const uint32_t gh_inverse = 65536u / (uint32_t)w.GH + 1u;
  const auto over_gh = [&](int x) { return (int)((uint32_t)x * gh_inverse >> 16); };
  const auto head_of = [&](int x) { return r0.z * w.GH + x - over_gh(x) * w.GH; };
  const auto sink_of = [&](int x) { return p.sinks && x < rows ? __ldg(p.sinks + head_of(x)) * kLog2e : -INFINITY; };
  // row x's output; whether it is not finite
  const auto finish = [&](int x, float den, float4 acc) {
    if (x >= rows) return false;
    const float inv = den != 0.f ? 1.f / den : 0.f;
    const float4 y = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    ET* to = static_cast<ET*>(p.out) + ((size_t)(r0.x + over_gh(x)) * p.H + head_of(x)) * dv + 4 * c;
    if constexpr (sizeof(ET) == 2) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(y.x, y.y), z = __floats2bfloat162_rn(y.z, y.w);
      *reinterpret_cast<uint2*>(to) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&z));
    } else {
      *reinterpret_cast<float4*>(to) = y;
    }
    // (a sum that is not finite comes of the row's own scores: its output holds no number whatever else it does not see)
    return CHECK && den * 0.f == 0.f && !(finite4(y) && finite4(acc));
  };
  const auto mark = [&](int x, bool again) {
    if (CHECK && again) atomicOr(&again_s[x >> 5], 1u << (x & 31));
  };
  const int step = (int)gridDim.y * rows_here;
  if (shares == 1 && total <= 2) {
#pragma unroll 1
    for (int x0 = (int)blockIdx.y * rows_here; x0 < rows && total > 0; x0 += 2 * step) {
      float m[2][2], l[2][2];
      float4 o[2][2];
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int s = 0; s < 2; ++s) fetch(s, x0 + v * step + rr, m[v][s], l[v][s], o[v][s]);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int x = x0 + v * step + rr;
        const float z2 = sink_of(x), M = fmaxf(z2, fmaxf(m[v][0], m[v][1]));
        float den = z2 != -INFINITY ? exp2_of(z2 - M) : 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        join(m[v][0], l[v][0], o[v][0], M, den, acc);
        join(m[v][1], l[v][1], o[v][1], M, den, acc);
        mark(x, finish(x, den, acc));
      }
    }
  }
#pragma unroll 1
  for (int x0 = (int)blockIdx.y * rows_here; x0 < rows && total > 0 && !(shares == 1 && total <= 2); x0 += step) {
    const int x = x0 + rr;
    const float z2 = sink_of(x);
    float M = share == 0 ? z2 : -INFINITY, den = M != -INFINITY ? 1.f : 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int s0 = 4 * share; s0 < total; s0 += 4 * shares) {
      float4 o[4];
      float m[4], l[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) fetch(s0 + t, x, m[t], l[t], o[t]);
      const float Mn = fmaxf(fmaxf(fmaxf(M, m[0]), fmaxf(m[1], m[2])), m[3]);
      const float f = M == -INFINITY ? 0.f : exp2_of(M - Mn);
      den = den == 0.f ? 0.f : den * f;
      acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
      M = Mn;
#pragma unroll
      for (int t = 0; t < 4; ++t) join(m[t], l[t], o[t], M, den, acc);
    }
    if (shares > 1) {
      md_s[tid] = make_float2(M, den);
      acc_s[tid] = acc;
      __syncthreads();
      if (share == 0)
        for (int k = 1; k < shares; ++k) {
          const float2 md = md_s[tid + k * (kJoinThreads / shares)];
          const float4 a = acc_s[tid + k * (kJoinThreads / shares)];
          if (md.y == 0.f) continue;
          const float Mn = fmaxf(M, md.x), f = den == 0.f ? 0.f : exp2_of(M - Mn), f2 = exp2_of(md.x - Mn);
          den = fmaf(f2, md.y, den == 0.f ? 0.f : den * f);
          acc = make_float4(fmaf(f2, a.x, acc.x * f), fmaf(f2, a.y, acc.y * f), fmaf(f2, a.z, acc.z * f),
                            fmaf(f2, a.w, acc.w * f));
          M = Mn;
        }
      __syncthreads();
    }
    if (share == 0) mark(x, finish(x, den, acc));
  }
  if (!CHECK) return;
  __syncthreads();
  for (int k = 0; k < 4; ++k)
    for (uint32_t left = again_s[k]; left; left &= left - 1) {  // (the same for all threads)
      const int x = 32 * k + __ffs(left) - 1;
      Row r;
      r.row = r0.x + over_gh(x);
      const int4 r2 = __ldcg(reinterpret_cast<const int4*>(w.rec + blockIdx.x) + 2);
      r.row0 = r2.x;
      r.i = r.row - r2.x;
      r.n = r2.y;
      r.hist = r1.w;
      r.depth = tree_depth(w, r.row, r.i, r.n);
      row_again(p, r0.w, r, head_of(x), reinterpret_cast<float*>(acc_s), md_s);
      __syncthreads();
    }
}

}  // namespace

cudaError_t launch_tree_combine(const TreeParams& p, int bf16, cudaStream_t st) {
  int dev = 0;
  cudaGetDevice(&dev);
  static std::atomic<unsigned long long> attr_done{0};  // per device
  if (dev >= 64 || !(attr_done.load(std::memory_order_acquire) >> dev & 1ull)) {
    // Shared memory for eight CTAs an SM and the rest for L1: the kernel before leaves 28 KB for that (see
    // dense_combine_kernel), but asking for all of it leaves room for one CTA (2,059 rows of 32 heads: 37 us).
    const auto share = [](const void* k) { return cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, 28); };
    cudaError_t e = share(reinterpret_cast<const void*>(tree_combine_kernel<__nv_bfloat16, true>));
    if (e == cudaSuccess) e = share(reinterpret_cast<const void*>(tree_combine_kernel<__nv_bfloat16, false>));
    if (e == cudaSuccess) e = share(reinterpret_cast<const void*>(tree_combine_kernel<float, false>));
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done.fetch_or(1ull << dev, std::memory_order_release);
  }
  // Few rows: fewer of a CTA, by more shares of their parts, while a share has four parts; many: a CTA goes
  // through more of its tile's. (One sequence of one row, 14 heads on 2 of 64, 32,000 keys: with one share 33 us, with
  // two 24, with eight 19; four sequences of 600 keys, five parts a row: with one share 10.8, with eight 11.4.)
  const int keys = p.w.capacity >> p.w.step_log2, cut = (p.w.slots + p.tiles) / (p.tiles > 0 ? p.tiles : 1);
  const int parts = (keys < cut ? keys : cut) + 1;  // of a row, about, at most
  int rows_here = 1024 / p.dv, shares = 1;
  const auto blocks_of = [&](int rows) { return (long long)p.tiles * ((p.w.R + rows - 1) / rows); };
  while (rows_here > 1 && shares < 8 && 4 * shares < parts && blocks_of(rows_here / 2) <= 2 * kDenseSms) {
    rows_here /= 2;
    shares *= 2;
  }
  const int groups = (p.w.R + rows_here - 1) / rows_here;
  const long long want = (kJoinCtas * (long long)kDenseSms + p.tiles - 1) / (p.tiles > 0 ? p.tiles : 1);
  const int split = want < groups ? (int)want : groups;
  if (p.tiles <= 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.tiles, (unsigned)split);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (!bf16) return cudaLaunchKernelEx(&cfg, tree_combine_kernel<float, false>, p, shares);
  return p.check ? cudaLaunchKernelEx(&cfg, tree_combine_kernel<__nv_bfloat16, true>, p, shares)
                 : cudaLaunchKernelEx(&cfg, tree_combine_kernel<__nv_bfloat16, false>, p, shares);
}

}  // namespace gqa
