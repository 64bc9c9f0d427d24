// qk_rows.cu -- query and key rows on their way into attention: RMS norm per
// head, position rotation in either pair layout, and (for the paged cache) the
// write of keys and values into their pool slots, in one pass over the rows.
//
// For a head row x of d elements with weight w (both optional parts):
//   y_e = x_e / sqrt(mean_e(x_e^2) + eps) * w_e
//   pair (a, b) of y, angle = position * w_t:  a' = m (a cos - b sin), b' = m (a sin + b cos)
// where pair t is (rot_offset + 2t, rot_offset + 2t + 1) or (rot_offset + t,
// rot_offset + t + rot_dim / 2). Everything in fp32, rounded once on the store.
//
// Each row is read once and written once, so memory bounds it; the mapping keeps
// the arithmetic under the memory time. A warp takes an item: one token and a
// share of its rows (heads of q, then of k). L lanes hold a row, two 16-byte
// chunks each, chosen so that for half pairs the second chunk holds the
// partners of the first: the rotation then needs no exchange between lanes (with
// one chunk a lane it took one shuffle per element, as much shared-memory pipe
// time as the loads and stores together). The cosines and sines of the token are
// formed once per item by the whole warp, and stay in registers over its rows.
// The row sums of the norm are fp32, by butterflies over the L lanes.
//
// Few tokens (a decode step): a token's rows are cut into as many items as fill
// the GPU, down to one round of loads each; many tokens: one item per token, so
// that its angles are formed once (qk_parts).
#include "common.cuh"
#include "internal.h"
#include "rope.cuh"

namespace gqa {
namespace {

constexpr int kQkWarps = 4;     // warps (items) per CTA
constexpr int kQkRows = 2;      // rows whose loads are in flight per lane group
constexpr int kMaxPairs = 128;  // rot_dim <= 256

struct RowPtr {
  const void* src;
  void* dst;
};

__device__ __forceinline__ uint4 ld16(const void* p) { return *reinterpret_cast<const uint4*>(p); }

// The first sequence b in [0, B) that holds packed row `tok`, -1 if none does:
// a search over ascending starts, 32 probes a step; the answer is verified, so a
// table that does not ascend gives -1 or a sequence that does hold the row, and
// no index leaves [0, B].
__device__ __forceinline__ int find_sequence(const int32_t* starts, int B, int tok, int lane) {
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const bool in = (long long)lane * step < n;
    const bool le = in && __ldg(starts + lo + lane * step) <= tok;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    if (m == 0) return -1;
    const int at = (31 - __clz(m)) * step;
    lo += at;
    n = min(step, n - at);
  }
  return (__ldg(starts + lo) <= tok && tok < __ldg(starts + lo + 1)) ? lo : -1;
}

// seq_lens_out of sequence b, by one warp: advanced by its rows when they fit
// the capacity and every table entry that they fall on is in range.
__device__ __forceinline__ void advance_length(const QkParams& p, int b, int lane) {
  const int s0 = p.row_starts[b], s1 = p.row_starts[b + 1], len = p.lens_in[b];
  const long long cap = (long long)p.mbps * p.bs;
  bool ok = s0 >= 0 && s0 <= s1 && s1 <= p.N && len >= 0 && (long long)len + (s1 - s0) <= cap;
  if (ok && s1 > s0) {
    const int b0 = len / p.bs, b1 = (len + (s1 - s0) - 1) / p.bs;
    bool bad = false;
    for (int i = b0 + lane; i <= b1; i += 32) {
      const int e = __ldg(p.tables + (size_t)b * p.mbps + i);
      bad |= e < 0 || e >= p.num_blocks;
    }
    ok = !__any_sync(0xffffffffu, bad);
  }
  __syncwarp();  // lens_out may be lens_in: every lane has read it
  if (lane == 0) {
    if (!ok) raise_error(p.err, kErrBounds);
    p.lens_out[b] = ok ? len + (s1 - s0) : len;
  }
}

// L lanes per row: a power of two >= the row's chunk pairs.
template <typename ET, int L, bool PAGED>
__global__ void __launch_bounds__(kQkWarps * 32) qk_rows_kernel(const QkParams p) {
  constexpr int V = Elem<ET>::kPerChunk;  // elements of a 16-byte chunk
  constexpr int kGroups = 32 / L;         // rows a warp works on side by side
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float2 cs_s[kQkWarps][kMaxPairs];
  // rows of a rotation whose pairs do not fall on whole chunks, one per lane group
  __shared__ __align__(16) float row_s[kQkWarps][32 * 2 * V];
  // launched as a programmatic dependent: everything read below may come from
  // the kernel before this one; the next launch may start setting up at once
  grid_dep_wait();
  grid_dep_launch();
  const long long item = (long long)blockIdx.x * kQkWarps + warp;
  const int per_token = p.parts + (PAGED ? 1 : 0);  // PAGED: the last item of a token copies its values
  const long long n_items = p.run_rows ? (long long)p.N * per_token : 0;
  if (item >= n_items) {
    if (PAGED && item - n_items < p.lens_items) advance_length(p, (int)(item - n_items), lane);
    return;
  }
  const int tok = (int)(item / per_token), part = (int)(item % per_token);

  // ---- the token's position and, for the paged append, its slot
  int pos = 0;
  long long slot = 0;  // pool row of KV head 0: (block * Hkv) * bs + row
  const long long tb = PAGED ? 0 : tok / p.T, tt = PAGED ? tok : tok % p.T;
  if (PAGED) {
    const int b = find_sequence(p.row_starts, p.B, tok, lane);
    if (b < 0) return;  // behind the last sequence: left as it is
    const int len = __ldg(p.lens_in + b);
    const long long at = (long long)len + ((long long)tok - __ldg(p.row_starts + b));
    const bool fits = len >= 0 && at < (long long)p.mbps * p.bs;
    const int blk = fits ? __ldg(p.tables + (size_t)b * p.mbps + at / p.bs) : -1;
    if (blk < 0 || blk >= p.num_blocks) {
      if (lane == 0) raise_error(p.err, kErrBounds);
      return;
    }
    pos = (int)at;
    slot = (long long)blk * p.Hkv * p.bs + at % p.bs;
    if (part == p.parts) {  // the values: copied as they are, four chunks in flight per lane
      const int cpv = p.dv / V, n = p.Hkv * cpv;
      for (int i0 = lane; i0 < n; i0 += 4 * 32) {
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i0 + u * 32;
          if (i < n)
            v[u] = ld16(static_cast<const ET*>(p.v.data) + tt * p.v.token_stride + (i / cpv) * p.v.head_stride +
                        (i % cpv) * V);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i0 + u * 32;
          if (i < n)
            *reinterpret_cast<uint4*>(static_cast<ET*>(p.v_pool) + (slot + (long long)(i / cpv) * p.bs) * p.dv +
                                      (i % cpv) * V) = v[u];
        }
      }
      return;
    }
  } else if (p.rot_dim) {
    pos = __ldg(p.positions + tok);
  }

  // ---- this lane's two chunks of every row (-1: none)
  const int li = lane % L, grp = lane / L;
  const int cpr = p.d / V;
  const int half = p.rot_dim / 2;
  const bool by_half = p.layout == 1;
  // whole chunks turn, each with its partner in the same lane
  const bool whole = p.rot_offset % V == 0 && (by_half ? half : p.rot_dim) % V == 0;
  int c0, c1;
  if (by_half && whole && p.rot_dim) {
    const int np = half / V, first = p.rot_offset / V;
    const int o0 = 2 * (li - np), o1 = o0 + 1;  // the others, in order, skipping the rotated ones
    c0 = li < np ? first + li : (o0 < first ? o0 : o0 + 2 * np);
    c1 = li < np ? first + np + li : (o1 < first ? o1 : o1 + 2 * np);
  } else {
    c0 = li;
    c1 = li + (cpr + 1) / 2;
    if (li >= (cpr + 1) / 2) c0 = c1 = cpr;
  }
  if (c0 >= cpr) c0 = -1;
  if (c1 >= cpr) c1 = -1;
  // chunk c turns: whole chunks inside the rotated slice
  auto turns = [&](int c) { return c >= 0 && c * V >= p.rot_offset && c * V < p.rot_offset + p.rot_dim; };
  const bool turn0 = whole && turns(c0), turn1 = whole && turns(c1);

  // ---- rows [r0, r1) of the token's q heads, then k heads
  const int rows = p.H + p.Hk;
  const int r0 = (int)((long long)rows * part / p.parts), r1 = (int)((long long)rows * (part + 1) / p.parts);
  auto row_ptr = [&](int r, bool& is_k) -> RowPtr {
    is_k = r >= p.H;
    if (!is_k)
      return {static_cast<const ET*>(p.q.data) + tb * p.q.batch_stride + tt * p.q.token_stride + r * p.q.head_stride,
              static_cast<ET*>(p.q_out.data) + tb * p.q_out.batch_stride + tt * p.q_out.token_stride +
                  r * p.q_out.head_stride};
    const int h = r - p.H;
    const ET* src = static_cast<const ET*>(p.k.data) + tb * p.k.batch_stride + tt * p.k.token_stride + h * p.k.head_stride;
    if (PAGED) return {src, static_cast<ET*>(p.k_out.data) + (slot + (long long)h * p.bs) * p.d};
    return {src, static_cast<ET*>(p.k_out.data) + tb * p.k_out.batch_stride + tt * p.k_out.token_stride +
                     h * p.k_out.head_stride};
  };
  auto load = [&](int r, uint4 (&v)[2]) {
    v[0] = v[1] = make_uint4(0, 0, 0, 0);
    if (r >= r1) return;
    bool is_k;
    const ET* src = static_cast<const ET*>(row_ptr(r, is_k).src);
    if (c0 >= 0) v[0] = ld16(src + c0 * V);
    if (c1 >= 0) v[1] = ld16(src + c1 * V);
  };

  // the first rows are requested before the angles wait on the position
  uint4 raw[kQkRows][2];
#pragma unroll
  for (int u = 0; u < kQkRows; ++u) load(r0 + u * kGroups + grp, raw[u]);
  uint4 wq[2], wk[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int c = s ? c1 : c0;
    wq[s] = p.q_weight && c >= 0 ? ld16(static_cast<const ET*>(p.q_weight) + c * V) : make_uint4(0, 0, 0, 0);
    wk[s] = p.k_weight && c >= 0 ? ld16(static_cast<const ET*>(p.k_weight) + c * V) : make_uint4(0, 0, 0, 0);
  }
  float2* cs = cs_s[warp];
  for (int t = lane; t < half; t += 32) {
    const float2 w = __ldg(reinterpret_cast<const float2*>(p.freqs) + t);
    float c, s;
    rope_cos_sin_f(pos, w.x, w.y, (double)w.x + (double)w.y, &c, &s);
    cs[t] = make_float2(c * p.magnitude, s * p.magnitude);
  }
  __syncwarp();
  // the V (cos, sin) this lane turns its chunks by: half pairs, one per element
  // of c0 (and its partner in c1); adjacent pairs, V / 2 per chunk
  float2 w[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    int t = by_half ? c0 * V + e - p.rot_offset
                    : ((e < V / 2 ? c0 : c1) * V - p.rot_offset) / 2 + e % (V / 2);
    const bool on = by_half ? turn0 : (e < V / 2 ? turn0 : turn1);
    w[e] = on ? cs[t] : make_float2(1.f, 0.f);
  }

  const float inv_d = 1.f / (float)p.d;
  for (int rb = r0; rb < r1; rb += kQkRows * kGroups) {
    uint4 cur[kQkRows][2];
#pragma unroll
    for (int u = 0; u < kQkRows; ++u) {
      cur[u][0] = raw[u][0];
      cur[u][1] = raw[u][1];
    }
    if (rb + kQkRows * kGroups < r1) {  // the next round's rows, while this one is turned
#pragma unroll
      for (int u = 0; u < kQkRows; ++u) load(rb + kQkRows * kGroups + u * kGroups + grp, raw[u]);
    }
#pragma unroll
    for (int u = 0; u < kQkRows; ++u) {
      const int r = rb + u * kGroups + grp;
      const bool live = r < r1;
      bool is_k = r >= p.H;
      float y[2][V];
      Elem<ET>::chunk_to_f32(cur[u][0], y[0]);
      Elem<ET>::chunk_to_f32(cur[u][1], y[1]);
      if (p.q_weight || p.k_weight) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) ss = fmaf(y[0][e], y[0][e], fmaf(y[1][e], y[1][e], ss));
#pragma unroll
        for (int off = L / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        if (is_k ? p.k_weight != nullptr : p.q_weight != nullptr) {
          const float rs = 1.f / sqrtf(fmaf(ss, inv_d, p.eps));
          float g[2][V];
          Elem<ET>::chunk_to_f32(is_k ? wk[0] : wq[0], g[0]);
          Elem<ET>::chunk_to_f32(is_k ? wk[1] : wq[1], g[1]);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            y[0][e] = y[0][e] * rs * g[0][e];
            y[1][e] = y[1][e] * rs * g[1][e];
          }
        }
      }
      if (whole) {
        if (by_half) {
          if (turn0) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float a = y[0][e], b = y[1][e];
              y[0][e] = fmaf(a, w[e].x, -b * w[e].y);
              y[1][e] = fmaf(a, w[e].y, b * w[e].x);
            }
          }
        } else {
#pragma unroll
          for (int s = 0; s < 2; ++s)
            if (s ? turn1 : turn0) {
#pragma unroll
              for (int e = 0; e < V / 2; ++e) {
                const float2 cw = w[s * (V / 2) + e];
                const float a = y[s][2 * e], b = y[s][2 * e + 1];
                y[s][2 * e] = fmaf(a, cw.x, -b * cw.y);
                y[s][2 * e + 1] = fmaf(a, cw.y, b * cw.x);
              }
            }
        }
      } else {
        // pairs that cross chunks: the row through shared memory, element by element
        float* row = row_s[warp] + grp * (2 * L * V);
        __syncwarp();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int c = s ? c1 : c0;
          if (c >= 0)
#pragma unroll
            for (int e = 0; e < V; ++e) row[c * V + e] = y[s][e];
        }
        __syncwarp();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int c = s ? c1 : c0;
          if (c >= 0)
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const int x = c * V + e - p.rot_offset;  // place in the rotated slice
              if (x < 0 || x >= p.rot_dim) continue;
              const int t = by_half ? (x < half ? x : x - half) : x / 2;
              const bool second = by_half ? x >= half : (x & 1) != 0;
              const int d = by_half ? half : 1;
              const float other = row[c * V + e + (second ? -d : d)];
              const float2 cw = cs[t];
              y[s][e] = second ? fmaf(other, cw.y, y[s][e] * cw.x) : fmaf(y[s][e], cw.x, -other * cw.y);
            }
        }
      }
      if (live) {
        ET* dst = static_cast<ET*>(row_ptr(r, is_k).dst);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int c = s ? c1 : c0;
          if (c < 0) continue;
          uint4 o;
          if constexpr (sizeof(ET) == 2) {
            __nv_bfloat162* o2 = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) o2[e] = __floats2bfloat162_rn(y[s][2 * e], y[s][2 * e + 1]);
          } else {
            o = make_uint4(__float_as_uint(y[s][0]), __float_as_uint(y[s][1]), __float_as_uint(y[s][2]),
                           __float_as_uint(y[s][3]));
          }
          *reinterpret_cast<uint4*>(dst + c * V) = o;
        }
      }
    }
  }
}

template <typename ET, int L, bool PAGED>
cudaError_t launch_qk(const QkParams& p, cudaStream_t st) {
  const long long items = (p.run_rows ? (long long)p.N * (p.parts + (PAGED ? 1 : 0)) : 0) + (PAGED ? p.lens_items : 0);
  if (items <= 0) return cudaSuccess;
  const long long blocks = (items + kQkWarps - 1) / kQkWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kQkWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_rows_kernel<ET, L, PAGED>, p);
}

// Chunk pairs of a row: as the kernel deals them out.
int chunk_pairs(int cpr, int V, int layout, int rot_offset, int rot_dim) {
  const int half = rot_dim / 2;
  if (layout == 1 && rot_dim && rot_offset % V == 0 && half % V == 0) return half / V + (cpr - 2 * (half / V) + 1) / 2;
  return (cpr + 1) / 2;
}

template <typename ET, bool PAGED>
cudaError_t dispatch_qk(QkParams p, cudaStream_t st) {
  constexpr int V = Elem<ET>::kPerChunk;
  const int pairs = chunk_pairs(p.d / V, V, p.layout, p.rot_offset, p.rot_dim);
  const int L = pairs <= 4 ? 4 : pairs <= 8 ? 8 : pairs <= 16 ? 16 : 32;
  // Items per token: as few as keep 16 warps on each of the 152 SMs, at most one
  // round of loads each.
  const int rows = p.H + p.Hk, most = (rows + kQkRows * (32 / L) - 1) / (kQkRows * (32 / L));
  const long long want = (152 * 16 + (long long)p.N - 1) / (p.N > 0 ? p.N : 1);
  p.parts = rows == 0 ? 1 : (int)(want < 1 ? 1 : want > most ? most : want);
  switch (L) {
    case 4: return launch_qk<ET, 4, PAGED>(p, st);
    case 8: return launch_qk<ET, 8, PAGED>(p, st);
    case 16: return launch_qk<ET, 16, PAGED>(p, st);
    default: return launch_qk<ET, 32, PAGED>(p, st);
  }
}

}  // namespace

cudaError_t launch_qk_rows(const QkParams& p, int bf16, int paged, cudaStream_t st) {
  if (bf16) return paged ? dispatch_qk<__nv_bfloat16, true>(p, st) : dispatch_qk<__nv_bfloat16, false>(p, st);
  return paged ? dispatch_qk<float, true>(p, st) : dispatch_qk<float, false>(p, st);
}

}  // namespace gqa
