// tree_combine.cu -- joins the partial results of drafted rows (tree_part.cuh), in the order of their slots:
//   M = max m_s (and the sink logit),  out = sum 2^(m_s - M) o_s / sum 2^(m_s - M) l_s
//
// A CTA takes rows (drafted row, head) of one head chunk, next to one another in the parts, rows along the
// lanes; rows by d_v / 4 threads of four columns by `shares` of the parts (several where few rows
// would leave SMs without work), four parts at a time, the shares joined at the end in their order. Three
// trips to memory bound it: which sequence the row is of, that sequence's place on the line, the parts.
//
// Values that a row does not see. A product with V on the tensor cores mixes all keys of a tile, and 0 * NaN is
// NaN: an infinity or NaN in one drafted row's value (or in a history row that the window has left for
// some rows) would reach rows that do not see it. That cannot happen without a result that is not
// finite, so a CTA that finds one looks at the values that its row does not see, and if one of them is not finite
// works the row out again from the keys that it does see, a warp a key. (Checked per row here it
// costs a vote; values looked over in every tile by the kernel itself took its MMA warp half a
// tile's time.)

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "tree_part.cuh"

namespace gqa {
namespace {

constexpr int kJoinThreads = 256;

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
  constexpr int kMost = 6;  // columns of a lane: d_k at most 192 on the tensor cores
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
  __shared__ float4 acc_s[kJoinThreads];
  __shared__ float2 md_s[kJoinThreads];
  __shared__ int again_s[kJoinThreads / 4];
  grid_dep_wait();
  const TreeWork& w = p.w;
  const int dv = p.dv, rows_here = 1024 / dv / shares;  // powers of two, as dv is
  const int tid = threadIdx.x, rr = tid & (rows_here - 1), c = tid / rows_here % (dv / 4);
  const int share = tid / (kJoinThreads / shares);
  const long long per_chunk = ((long long)w.N * w.GH + rows_here - 1) / rows_here;
  const int chunk = (int)(blockIdx.x / per_chunk);  // KV head and head chunk
  const long long x = (long long)(blockIdx.x % per_chunk) * rows_here + rr;
  if (CHECK && tid < rows_here) again_s[tid] = 0;
  // ---- the row's place on the line
  bool live = x < (long long)w.N * w.GH;
  const int row = live ? (int)(x / w.GH) : 0, g = live ? (int)(x - (long long)row * w.GH) : 0, h = chunk * w.GH + g;
  const int C = __ldcg(w.line), S = __ldcg(w.line + 1);
  const int b = live ? __ldcg(w.row_seq + row) : -1;
  live = live && b >= 0 && b < w.B;
  int4 rec = make_int4(0, 0, 0, 0);
  int hist = 0;
  if (live) {
    rec = __ldcg(reinterpret_cast<const int4*>(w.rec + b));
    hist = __ldcg(&w.rec[b].hist);
  }
  const int i = row - rec.x, n = rec.y;
  live = live && n > 0 && i >= 0 && i < n && C > 0;
  int first = 0, total = 0, in_tile = 0;
  const float* U = p.partial;
  const size_t part = dense_part_floats(w.R, dv);
  if (live) {
    const TreeShape s = tree_shape(w, n, hist);
    const int tile = i / w.RPT, item = chunk * s.tiles + tile, at = rec.z + item * (s.T + 1);
    first = tree_slot_of(C, S, at + 1);
    total = tree_slot_of(C, S, at + s.T) - first + 1;
    in_tile = (i - tile * w.RPT) * w.GH + g;
    U = p.partial + (size_t)(rec.w + item + first) * part;
  }
  const float z2 = p.sinks && live ? __ldg(p.sinks + h) * kLog2e : -INFINITY;
  float M = share == 0 ? z2 : -INFINITY, den = M != -INFINITY ? 1.f : 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int s0 = 4 * share; s0 < total; s0 += 4 * shares) {
    float4 o[4];
    float m[4], l[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      m[t] = -INFINITY;
      l[t] = 0.f;
      o[t] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s0 + t < total) {
        const float* u = U + (size_t)(s0 + t) * part;
        m[t] = __ldcg(u + (size_t)w.R * dv + in_tile);
        l[t] = __ldcg(u + (size_t)w.R * dv + w.R + in_tile);
        o[t] = __ldcg(reinterpret_cast<const float4*>(u) + (size_t)c * w.R + in_tile);
      }
    }
    const float Mn = fmaxf(fmaxf(fmaxf(M, m[0]), fmaxf(m[1], m[2])), m[3]);
    const float f = M == -INFINITY ? 0.f : exp2_of(M - Mn);
    den = den == 0.f ? 0.f : den * f;
    acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
    M = Mn;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (l[t] == 0.f) continue;  // no visible key, whatever m and o hold (a NaN in l goes through)
      const float f2 = exp2_of(m[t] - M);
      den = fmaf(f2, l[t], den);
      acc.x = fmaf(f2, o[t].x, acc.x);
      acc.y = fmaf(f2, o[t].y, acc.y);
      acc.z = fmaf(f2, o[t].z, acc.z);
      acc.w = fmaf(f2, o[t].w, acc.w);
    }
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
  }
  bool again = false;
  if (live && share == 0) {
    const float inv = den != 0.f ? 1.f / den : 0.f;
    const float4 y = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    ET* to = static_cast<ET*>(p.out) + ((size_t)row * p.H + h) * dv + 4 * c;
    if constexpr (sizeof(ET) == 2) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(y.x, y.y), z = __floats2bfloat162_rn(y.z, y.w);
      *reinterpret_cast<uint2*>(to) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&z));
    } else {
      *reinterpret_cast<float4*>(to) = y;
    }
    again = CHECK && !(finite4(y) && finite4(acc));
  }
  if (CHECK) {
    if (!__syncthreads_or(again)) return;
    if (again) again_s[rr] = 1;
    for (int k = 0; k < rows_here; ++k) {
      __syncthreads();  // (the rows are marked; shared memory is free)
      if (!again_s[k]) continue;
      const long long xk = (long long)(blockIdx.x % per_chunk) * rows_here + k;
      Row r;
      r.row = (int)(xk / w.GH);
      const int bk = __ldcg(w.row_seq + r.row);
      const int4 q = __ldcg(reinterpret_cast<const int4*>(w.rec + bk));
      r.row0 = q.x;
      r.i = r.row - q.x;
      r.n = q.y;
      r.hist = __ldcg(&w.rec[bk].hist);
      r.depth = tree_depth(w, r.row, r.i, r.n);
      row_again(p, bk, r, chunk * w.GH + (int)(xk - (long long)r.row * w.GH), reinterpret_cast<float*>(acc_s), md_s);
    }
  }
}

}  // namespace

cudaError_t launch_tree_combine(const TreeParams& p, int bf16, cudaStream_t st) {
  int dev = 0;
  cudaGetDevice(&dev);
  static std::atomic<unsigned long long> attr_done{0};  // per device
  if (dev >= 64 || !(attr_done.load(std::memory_order_acquire) >> dev & 1ull)) {
    // (the whole L1: see dense_combine_kernel)
    const auto full = [](const void* k) {
      return cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxL1);
    };
    cudaError_t e = full(reinterpret_cast<const void*>(tree_combine_kernel<__nv_bfloat16, true>));
    if (e == cudaSuccess) e = full(reinterpret_cast<const void*>(tree_combine_kernel<__nv_bfloat16, false>));
    if (e == cudaSuccess) e = full(reinterpret_cast<const void*>(tree_combine_kernel<float, false>));
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done.fetch_or(1ull << dev, std::memory_order_release);
  }
  int rows_here = 1024 / p.dv, shares = 1;
  const auto blocks_of = [&](int rows) {
    return (long long)p.w.heads * (((long long)p.w.N * p.w.GH + rows - 1) / rows);
  };
  while (rows_here > 1 && shares < 8 && blocks_of(rows_here / 2) <= 2 * kDenseSms) {
    rows_here /= 2;
    shares *= 2;
  }
  const long long blocks = blocks_of(rows_here);
  if (blocks <= 0) return cudaSuccess;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
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
