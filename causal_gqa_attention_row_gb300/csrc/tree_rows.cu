// tree_rows.cu -- attention of drafted rows (attn_tree_paged) where the tensor cores do not take the
// call: fp32, other head widths, other block sizes, a scale that is not positive.
//
//   out[r] = softmax over the history and the drafted rows that r sees of scale * q_r . k_j, times v_j
//
// An item is up to 64 rows (drafted rows times heads of one KV head), a unit a range of its keys
// (tree_part.cuh); keys come 64 at a time. The arithmetic is fp32 throughout: a thread forms 4 x 4 scores
// (16 bytes of four queries and four keys a step, packed products), its half warp owns those four rows,
// so the row maximum and the probabilities stay within it, then 4 rows x d_v / 16 columns of the
// output in registers. K and V share one tile in shared memory, which leaves room for two CTAs an SM (one
// beyond 128 columns); each is requested once the other has been worked on, so its way through memory stands open
// (held in registers meanwhile, they left too few: 16 sequences of one row, 32 heads on 8 of 128, behind 4,000 keys 311 us,
// so 272). Eight rows are a warp's, and warps without rows only load.
//
// A row's masked keys weigh nothing whatever they hold: their scores are set to -infinity, and
// in a tile that some row does not see whole a key of weight zero is left out of the second product, since
// 0 * NaN would not be 0. (In the other tiles the value of a key that scores -infinity counts, as 0 * v.)
//
// Where rows are many the fp32 rate bounds it, 4 d flops a row and key: tiles of 64 rows by 64 keys read 12 KB of
// shared memory a 16-byte step for 64 x 64 x 4 products, so issue and shared memory are about even. Where they
// are few it is the latency of the one warp that has them. Measured (fp32): 6 sequences of 3 to 24 rows, 8 heads
// on 2 of 64, up to 1,500 keys 21.6 us.

#include <atomic>

#include "attn_rows.cuh"
#include "tree_part.cuh"

namespace gqa {
namespace {

constexpr int kTreeThreads = 256;
constexpr int kTreeRows = 64, kTreeKeys = 64;
constexpr int kPStride = kTreeKeys + 4;

template <typename ET, int DK, int DV>
struct TreeCfg {
  static constexpr int kWide = DK > DV ? DK : DV, kStride = kWide + 4;
  static constexpr int kSeq = 16384;  // the line
  static constexpr int kQ = kSeq, kKV = kQ + kTreeRows * DK * 4, kP = kKV + kTreeKeys * kStride * 4;
  static constexpr int kRow = kP + kTreeRows * kPStride * 4;  // pool rows of two tiles, masks, positions
  static constexpr int kBytes = kRow + 2 * kTreeKeys * 8 + kTreeRows * 16 + kTreeKeys * 4 + kTreeRows * 4;
  static constexpr int kCtas = kBytes <= 113 * 1024 ? 2 : 1;
  static constexpr int kCh = Elem<ET>::kPerChunk;
  static constexpr int kLoadK = (kTreeKeys * DK / kCh + kTreeThreads - 1) / kTreeThreads;
  static constexpr int kLoadV = (kTreeKeys * DV / kCh + kTreeThreads - 1) / kTreeThreads;
  static constexpr int kLoad = kLoadK > kLoadV ? kLoadK : kLoadV;
  static_assert(kBytes <= 232448, "over the 227 KiB a CTA may use");
};

template <typename ET, int DK, int DV>
__global__ void __launch_bounds__(kTreeThreads, TreeCfg<ET, DK, DV>::kCtas)
    tree_rows_kernel(const __grid_constant__ TreeParams p) {
  using C = TreeCfg<ET, DK, DV>;
  constexpr int CH = C::kCh, kCols = DV >= 64 ? DV / 64 : 1;
  extern __shared__ __align__(128) unsigned char smem[];
  TreeSeq* seq = reinterpret_cast<TreeSeq*>(smem);
  float* sq = reinterpret_cast<float*>(smem + C::kQ);
  float* skv = reinterpret_cast<float*>(smem + C::kKV);
  float* sp = reinterpret_cast<float*>(smem + C::kP);
  long long* pool_row = reinterpret_cast<long long*>(smem + C::kRow);  // [2][keys], of the KV head; -1: no key
  long long* q_row = pool_row + 2 * kTreeKeys;  // [rows], of the queries; -1: none
  uint32_t* masks = reinterpret_cast<uint32_t*>(q_row + kTreeRows);  // [rows][2]
  int* key_pos = reinterpret_cast<int*>(masks + 2 * kTreeRows);
  int* row_pos = key_pos + kTreeKeys;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const TreeWork& w = p.w;
  grid_dep_wait();
  grid_dep_launch();
  tree_line<kTreeThreads>(w, seq, (int)blockIdx.x);
  tree_publish(w, seq, (int)blockIdx.x, (int)gridDim.x, tid, kTreeThreads);
  TreeWalk walk = tree_walk(w, seq, 1, (int)blockIdx.x);
  const bool placed = w.window > 0 || p.alibi;  // positions matter
  const float cap_k = p.softcap2 > 0.f ? 2.8853900817779268f / p.softcap2 : 0.f;  // 2 log2(e) / cap
  TreeUnit u;
  while (tree_next(w, seq, 1, 0, walk, u)) {
    const int i0 = u.tile * w.RPT, n_i = min(w.RPT, u.n - i0), rows = n_i * w.GH, head0 = u.hc * w.GH;
    const int kvh = head0 / p.G, n_tiles = (u.key1 - u.key0 + kTreeKeys - 1) / kTreeKeys;
    const bool busy = (tid >> 5) * 8 < rows;  // this warp's eight rows
    // places of tile t's keys, and where they stand
    const auto places = [&](int t) {
      if (tid < kTreeKeys) {
        const int key = u.key0 + t * kTreeKeys + tid;
        long long at = -1;
        if (t < n_tiles && key < u.key1) {
          const int e = __ldg(p.tables + (size_t)u.b * p.mbps + key / w.bs);
          if (e >= 0 && e < p.num_blocks) at = ((long long)e * p.Hkv + kvh) * w.bs + key % w.bs;
          else if (e >= 0 || key < u.hist) raise_error(w.err, kErrBounds);  // (below 0 behind it: no block was to be had)
        }
        pool_row[(t & 1) * kTreeKeys + tid] = at;
      }
    };
    uint4 held[C::kLoad];
    const auto load = [&](const void* pool, int d, int t) {
      const int cpr = d / CH;
#pragma unroll
      for (int x = 0; x < C::kLoad; ++x) {
        const int c = tid + x * kTreeThreads;
        held[x] = make_uint4(0, 0, 0, 0);
        if (c < kTreeKeys * cpr) {
          const long long at = pool_row[(t & 1) * kTreeKeys + c / cpr];
          if (at >= 0) held[x] = __ldg(reinterpret_cast<const uint4*>(static_cast<const ET*>(pool) + at * d + c % cpr * CH));
        }
      }
    };
    const auto store = [&](int d) {
      const int cpr = d / CH;
#pragma unroll
      for (int x = 0; x < C::kLoad; ++x) {
        const int c = tid + x * kTreeThreads;
        if (c < kTreeKeys * cpr) {
          float f[CH];
          Elem<ET>::chunk_to_f32(held[x], f);
          float* to = skv + c / cpr * C::kStride + c % cpr * CH;
#pragma unroll
          for (int e = 0; e < CH; e += 4) *reinterpret_cast<float4*>(to + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
        }
      }
    };
    __syncthreads();  // the unit before is done with everything
    places(0);
    if (tid >= kTreeThreads - kTreeRows) {
      const int r = tid - (kTreeThreads - kTreeRows);
      q_row[r] = r < rows ? (long long)(u.row0 + i0 + r / w.GH) * p.H + head0 + r % w.GH : -1;
    }
    __syncthreads();
    load(p.k, DK, 0);
    // (a warp's eight rows or none)
    for (int c = tid; c < (rows + 7) / 8 * 8 * (DK / CH); c += kTreeThreads) {
      const int r = c / (DK / CH), x = c % (DK / CH) * CH;
      float f[CH];
#pragma unroll
      for (int e = 0; e < CH; ++e) f[e] = 0.f;
      if (q_row[r] >= 0)
        Elem<ET>::chunk_to_f32(__ldg(reinterpret_cast<const uint4*>(static_cast<const ET*>(p.q) + q_row[r] * DK + x)), f);
#pragma unroll
      for (int e = 0; e < CH; e += 4)
        *reinterpret_cast<float4*>(sq + r * DK + x + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    }
    if (placed && tid < kTreeRows) {
      const int i = i0 + min(tid, rows - 1) / w.GH;
      row_pos[tid] = u.hist + tree_depth(w, u.row0 + i, i, u.n) - 1;
    }
    float slope2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      slope2[i] = p.alibi ? __ldg(p.alibi + head0 + min(ty * 4 + i, rows - 1) % w.GH) * kLog2e : 0.f;
    float2 o[4][kCols][2];
    float m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < kCols; ++c) o[i][c][0] = o[i][c][1] = make_float2(0.f, 0.f);
    }
#pragma unroll 1
    for (int t = 0; t < n_tiles; ++t) {
      const int j0 = u.key0 + t * kTreeKeys;
      // some row of the sequence does not see some key of the tile (the window's lower end moves with a row)
      const bool partly = j0 + kTreeKeys > u.hist || (w.window > 0 && j0 < u.hist + u.n - w.window);
      if (t > 0) load(p.k, DK, t);
      __syncthreads();  // the tile before is done with
      store(DK);
      if (placed && tid < kTreeKeys) {
        const int j = j0 + tid - u.hist;
        key_pos[tid] = j < 0 ? j0 + tid : j < u.n ? u.hist + tree_depth(w, u.row0 + j, j, u.n) - 1 : 0;
      }
      __syncthreads();
      if (partly && tid < 2 * kTreeRows) {
        const int r = tid >> 1, half = tid & 1, i = i0 + min(r, rows - 1) / w.GH;
        uint32_t x = tree_bits(w, u.row0 + i, i, u.n, j0 - u.hist + 32 * half);
        if (w.window > 0)
          for (int e = 0; e < 32; ++e)
            if (key_pos[32 * half + e] <= row_pos[r] - w.window) x &= ~(1u << e);
        masks[tid] = x;
      }
      places(t + 1);
      if (partly) __syncthreads();
      if (busy) {
        // ---- scores
        float2 acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int d = 0; d < DK; d += 4) {
          float4 a[4], b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(sq + (ty * 4 + i) * DK + d);
#pragma unroll
          for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(skv + (tx + 16 * j) * C::kStride + d);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[i][j] = __ffma2_rn(make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y), acc[i][j]);
              acc[i][j] = __ffma2_rn(make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w), acc[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = ty * 4 + i;
          float s[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[j] = (acc[i][j].x + acc[i][j].y) * p.qscale;
            if (p.softcap2 > 0.f) s[j] = softcap_log2(s[j], p.softcap2, cap_k);
            if (p.alibi) s[j] = fmaf(slope2[i], (float)(key_pos[tx + 16 * j] - row_pos[r]), s[j]);
            if (partly && !(masks[2 * r + (j >> 1)] >> ((tx + 16 * j) & 31) & 1u)) s[j] = -INFINITY;
          }
          float mx = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
#pragma unroll
          for (int off = 8; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
          const float mn = fmaxf(m[i], mx);
          const float at = mn == -INFINITY ? 0.f : mn, f = ex2(m[i] - at);  // (0 while no key has been seen)
          m[i] = mn;
          l[i] *= f;
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            o[i][c][0] = __fmul2_rn(o[i][c][0], make_float2(f, f));
            o[i][c][1] = __fmul2_rn(o[i][c][1], make_float2(f, f));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float e = ex2(s[j] - at);
            l[i] += e;
            sp[r * kPStride + tx + 16 * j] = e;
          }
        }
      }
      load(p.v, DV, t);
      __syncthreads();  // K is done with
      store(DV);
      __syncthreads();
      if (busy && tx * 4 < DV) {
        // ---- output
        if (!partly) {
#pragma unroll 2
          for (int k = 0; k < kTreeKeys; k += 4) {
            float4 pr[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) pr[i] = *reinterpret_cast<const float4*>(sp + (ty * 4 + i) * kPStride + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
              for (int c = 0; c < kCols; ++c) {
                const float4 v = *reinterpret_cast<const float4*>(skv + (k + kk) * C::kStride + tx * 4 + 64 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float e = kk == 0 ? pr[i].x : kk == 1 ? pr[i].y : kk == 2 ? pr[i].z : pr[i].w;
                  o[i][c][0] = __ffma2_rn(make_float2(e, e), make_float2(v.x, v.y), o[i][c][0]);
                  o[i][c][1] = __ffma2_rn(make_float2(e, e), make_float2(v.z, v.w), o[i][c][1]);
                }
              }
          }
        } else {
          const int some = min(kTreeKeys, u.key1 - j0);  // (the last tile's keys)
#pragma unroll 1
          for (int k = 0; k < some; k += 4) {
            float4 pr[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) pr[i] = *reinterpret_cast<const float4*>(sp + (ty * 4 + i) * kPStride + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
              for (int c = 0; c < kCols; ++c) {
                const float4 v = *reinterpret_cast<const float4*>(skv + (k + kk) * C::kStride + tx * 4 + 64 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float e = kk == 0 ? pr[i].x : kk == 1 ? pr[i].y : kk == 2 ? pr[i].z : pr[i].w;
                  if (e != 0.f) {
                    o[i][c][0] = __ffma2_rn(make_float2(e, e), make_float2(v.x, v.y), o[i][c][0]);
                    o[i][c][1] = __ffma2_rn(make_float2(e, e), make_float2(v.z, v.w), o[i][c][1]);
                  }
                }
              }
          }
        }
      }
    }
    // ---- the partial result
    if (busy) {
      float* part = p.partial + (size_t)u.index * dense_part_floats(w.R, DV);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
        if (r >= rows) continue;
        if (tx * 4 < DV)
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            *reinterpret_cast<float4*>(part + ((size_t)(tx + 16 * c) * w.R + r) * 4) =
                make_float4(o[i][c][0].x, o[i][c][0].y, o[i][c][1].x, o[i][c][1].y);
        if (tx == 0) {
          part[(size_t)w.R * DV + r] = m[i];
          part[(size_t)w.R * DV + w.R + r] = l[i];
        }
      }
    }
  }
}

template <typename ET, int DK, int DV>
cudaError_t launch_tr(const TreeParams& p, cudaStream_t st) {
  using C = TreeCfg<ET, DK, DV>;
  int dev = 0;
  cudaGetDevice(&dev);
  static std::atomic<unsigned long long> attr_done{0};  // per device, per instantiation
  if (dev >= 64 || !(attr_done.load(std::memory_order_acquire) >> dev & 1ull)) {
    const cudaError_t e =
        cudaFuncSetAttribute(tree_rows_kernel<ET, DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done.fetch_or(1ull << dev, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.w.slots);
  cfg.blockDim = dim3(kTreeThreads);
  cfg.dynamicSmemBytes = C::kBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_rows_kernel<ET, DK, DV>, p);
}

// F: what to do with the kernel's instantiation for a width.
template <typename ET, typename F>
auto by_width(int dk, int dv, F f) -> decltype(f.template operator()<ET, 64, 64>()) {
  if (dk == 192 && dv == 128) return f.template operator()<ET, 192, 128>();
  if (dk == dv) {
    if (dk == 16) return f.template operator()<ET, 16, 16>();
    if (dk == 32) return f.template operator()<ET, 32, 32>();
    if (dk == 64) return f.template operator()<ET, 64, 64>();
    if (dk == 128) return f.template operator()<ET, 128, 128>();
    if (dk == 256) return f.template operator()<ET, 256, 256>();
  }
  return {};
}
struct Ctas {
  template <typename ET, int DK, int DV>
  int operator()() const { return TreeCfg<ET, DK, DV>::kCtas; }
};
struct Launch {
  const TreeParams& p;
  cudaStream_t st;
  template <typename ET, int DK, int DV>
  cudaError_t operator()() const { return launch_tr<ET, DK, DV>(p, st); }
};

}  // namespace

int tree_rows_ctas(int bf16, int dk, int dv) {
  return bf16 ? by_width<__nv_bfloat16>(dk, dv, Ctas{}) : by_width<float>(dk, dv, Ctas{});
}

int tree_rows_tile() { return kTreeRows; }

cudaError_t launch_tree_rows(const TreeParams& p, int bf16, cudaStream_t st) {
  if (!tree_rows_ctas(bf16, p.dk, p.dv)) return cudaErrorNotSupported;
  return bf16 ? by_width<__nv_bfloat16>(p.dk, p.dv, Launch{p, st}) : by_width<float>(p.dk, p.dv, Launch{p, st});
}

}  // namespace gqa
