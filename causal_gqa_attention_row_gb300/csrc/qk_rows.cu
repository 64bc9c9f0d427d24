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
// partners of the first: the rotation then needs no exchange between lanes. The
// cosines and sines of the token are formed once per item by the whole warp; each
// lane multiplies them with its columns' weights into the four factors of a pair,
//   a' = rs * (a * (w_a m cos) - b * (w_b m sin)),  b' = rs * (a * (w_a m sin) + b * (w_b m cos)),
// which stay in registers over the rows of q, then of k: three packed operations
// per two columns and row, rs = 1 / sqrt(mean + eps) included. The row sums are
// fp32, by butterflies over the L lanes.
//
// Rows travel by cp.async through a ring of two rounds a warp, each lane its own 16
// bytes (no barrier), requested before the token's position and slot are known. Few
// tokens (a decode step): a token's rows are cut into as many items as fill the GPU,
// down to one round each; many tokens: one item per token, so that its angles and
// factors are formed once; many tokens of few rows: up to eight tokens a warp, side by
// side (dispatch_qk).
//
// Measured (32 + 8 heads of 128): 16384 tokens 63.9 us (5.3 TB/s of rows read and written,
// 0.78 of the copy bandwidth), four 2048-row chunks appended 37.5 us (5.4 TB/s); fp32 115.2
// and 63.4 us (5.8 and 6.4 TB/s).
// The first form (rows through registers, weights and rotation apart, a division per
// address) took 82.5 and 76.1 us at twice the instructions and half the warps. Two rows a
// round against one: 4.8 and 6.1 us for 2048 tokens of 14 + 2 heads of 64, alike for the
// long ones; four rounds in flight or fewer registers (5 or 6 CTAs an SM) gain nothing.

#include "common.cuh"
#include "internal.h"
#include "rope.cuh"

namespace gqa {
namespace {

constexpr int kQkWarps = 4;     // warps (items) per CTA
constexpr int kQkRows = 2;      // rows of a round per lane group
constexpr int kQkStages = 2;    // rounds in flight per warp (2 KB each)

// How pairs turn: columns that cross 16-byte chunks, half pairs by whole chunks,
// adjacent pairs by whole chunks (or no rotation).
enum { kTurnAny = 0, kTurnHalf = 1, kTurnAdjacent = 2 };

// 16 bytes from global to shared memory, asynchronously; each thread waits for its own.
__device__ __forceinline__ void async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void async_wait() {  // all but the last N groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 ld16(const void* p) { return *reinterpret_cast<const uint4*>(p); }

// A 16-byte chunk as float2 of neighbouring columns, and back (rounded to nearest).
template <typename ET>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  static __device__ __forceinline__ void unpack(const uint4& u, float2* f) {
    f[0] = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
    f[1] = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
    f[2] = make_float2(__uint_as_float(u.z << 16), __uint_as_float(u.z & 0xffff0000u));
    f[3] = make_float2(__uint_as_float(u.w << 16), __uint_as_float(u.w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 pack(const float2* f) {
    uint4 u;
    __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = __floats2bfloat162_rn(f[e].x, f[e].y);
    return u;
  }
};
template <>
struct Chunk<float> {
  static __device__ __forceinline__ void unpack(const uint4& u, float2* f) {
    f[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    f[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 pack(const float2* f) {
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                      __float_as_uint(f[1].y));
  }
};

// The sequence b that holds packed row `tok` (-1: none), its length and the row's
// index in it. Up to 31 sequences in one round trip, a lane each; more by a search
// over the ascending starts, 32 probes a step. The answer is verified, so a table
// that does not ascend gives -1 or a sequence that does hold the row, and no index
// leaves [0, B].
__device__ __forceinline__ int find_sequence(const QkParams& p, int tok, int lane, int& len, long long& row) {
  if (p.B < 32) {
    const int s = lane <= p.B ? __ldg(p.row_starts + lane) : 0;
    const int n = lane < p.B ? __ldg(p.lens_in + lane) : 0;
    const unsigned m = __ballot_sync(0xffffffffu, lane < p.B && s <= tok);
    const int b = 31 - __clz(m);  // -1 for none
    const int start = __shfl_sync(0xffffffffu, s, b & 31), end = __shfl_sync(0xffffffffu, s, (b + 1) & 31);
    len = __shfl_sync(0xffffffffu, n, b & 31);
    row = (long long)tok - start;
    return m != 0 && tok < end ? b : -1;
  }
  int lo = 0, n = p.B;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const bool in = (long long)lane * step < n;
    const bool le = in && __ldg(p.row_starts + lo + lane * step) <= tok;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    if (m == 0) return -1;
    const int at = (31 - __clz(m)) * step;
    lo += at;
    n = min(step, n - at);
  }
  const int start = __ldg(p.row_starts + lo), end = __ldg(p.row_starts + lo + 1);
  len = __ldg(p.lens_in + lo);
  row = (long long)tok - start;
  return start <= tok && tok < end ? lo : -1;
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

// L lanes per row: a power of two >= the row's chunk pairs. W tokens per warp, side by side (more
// than one: each a whole token).
template <typename ET, int L, int TURN, bool PAGED, int W>
__global__ void __launch_bounds__(kQkWarps * 32) qk_rows_kernel(const QkParams p) {
  constexpr int V = Elem<ET>::kPerChunk;  // elements of a 16-byte chunk
  constexpr int H2 = V / 2;
  constexpr int kSub = 32 / W;            // lanes of a token
  constexpr int kGroups = kSub / L;       // rows of a token side by side
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float2 cs_s[kQkWarps * W][L * V];  // (a row has at most 2 L V columns)
  // rounds of rows in flight: [stage][row][chunk][lane], each lane its own 16 bytes
  __shared__ uint4 ring_s[kQkWarps][kQkStages][kQkRows][2][32];
  // kTurnAny: the rows being turned, one per lane group
  __shared__ __align__(16) float row_s[TURN == kTurnAny ? kQkWarps : 1][TURN == kTurnAny ? 32 * 2 * V : 1];
  // launched as a programmatic dependent: everything read below may come from
  // the kernel before this one; the next launch may start setting up at once
  grid_dep_wait();
  grid_dep_launch();
  // block row y: share y of the tokens' rows; PAGED: then the tokens' values (with a single
  // share they go with it: half as many warps wait for a position), then the lengths
  const int item = (int)(blockIdx.x * kQkWarps) + warp, part = (int)blockIdx.y + p.first_part;
  if (PAGED && part == p.lens_part) {
    if (item < p.lens_items) advance_length(p, item, lane);
    return;
  }
  const long long first_tok = (long long)item * W;
  if (first_tok >= p.N) return;
  const int ts = lane / kSub, sl = lane % kSub;  // the token of this lane, the lane within it
  bool alive = W == 1 || first_tok + ts < p.N;   // (W > 1: the others' lanes come along and write nothing)
  const int tok = W == 1 ? item : alive ? (int)first_tok + ts : p.N - 1;
  const long long tb = PAGED ? 0 : tok / p.T, tt = PAGED ? tok : tok % p.T;

  // ---- this lane's two chunks of every row (-1: none)
  const int li = lane % L, grp = sl / L;
  const int cpr = p.d / V;
  const int half = p.rot_dim / 2;
  int c0, c1;
  if (TURN == kTurnHalf) {
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
  const auto turns = [&](int c) { return c >= 0 && c * V >= p.rot_offset && c * V < p.rot_offset + p.rot_dim; };
  const bool turn0 = turns(c0), turn1 = turns(c1);

  // ---- rows [r0, r1) of the token's q heads, then k heads
  const int r0 = part * p.part_rows, r1 = min(r0 + p.part_rows, p.H + p.Hk);
  const bool values = PAGED && p.parts > 1 && part == p.parts;
  // The item's rounds: those of its q rows, then those of its k rows. Round i is
  // requested into stage i % kQkStages.
  const int q_lo = min(r0, p.H), q_hi = min(r1, p.H), k_lo = max(r0 - p.H, 0), k_hi = max(r1 - p.H, 0);
  constexpr int kRound = kQkRows * kGroups;
  const int q_rounds = (q_hi - q_lo + kRound - 1) / kRound, rounds = q_rounds + (k_hi - k_lo + kRound - 1) / kRound;
  auto& ring = ring_s[warp];
  // this lane's chunk c0 (c1 lies `apart` columns on) of its row of the next round
  const int col0 = max(c0, 0) * V, apart = (c1 - c0) * V;
  const ET* next = static_cast<const ET*>(p.q.data) + tb * p.q.batch_stride + tt * p.q.token_stride +
                   (q_lo + grp) * p.q.head_stride + col0;
  long long step = kGroups * p.q.head_stride;
  int next_row = q_lo + grp, next_end = q_hi, next_round = 0;
  const auto request = [&]() {
    if (next_round == q_rounds) {  // on to the k rows
      next = static_cast<const ET*>(p.k.data) + tb * p.k.batch_stride + tt * p.k.token_stride +
             (k_lo + grp) * p.k.head_stride + col0;
      step = kGroups * p.k.head_stride;
      next_row = k_lo + grp;
      next_end = k_hi;
    }
    if (next_round < rounds) {
      uint4* slot = &ring[next_round % kQkStages][0][0][lane];
#pragma unroll
      for (int u = 0; u < kQkRows; ++u) {
        if (next_row < next_end) {
          if (c0 >= 0) async16(slot + u * 64, next);
          if (c1 >= 0) async16(slot + u * 64 + 32, next + apart);
        }
        next += step;
        next_row += kGroups;
      }
    }
    ++next_round;
    async_commit();  // (an empty group keeps the count)
  };
  // requested before the position is known: the rows do not depend on it
  if (!values) {
#pragma unroll
    for (int i = 0; i < kQkStages; ++i) request();
  }

  // ---- the token's position and, for the paged append, its slot
  int pos = 0;
  long long slot = 0;  // pool row of KV head 0: (block * Hkv) * bs + row
  if (PAGED) {
    int len = 0, b = -1;
    long long row = 0;
    if (W == 1) {
      b = find_sequence(p, tok, lane, len, row);
    } else {
#pragma unroll
      for (int w = 0; w < W; ++w) {
        int n;
        long long r;
        const int x = find_sequence(p, (int)min(first_tok + w, (long long)p.N - 1), lane, n, r);
        if (w == ts) {
          b = x;
          len = n;
          row = r;
        }
      }
    }
    alive = alive && b >= 0;  // behind the last sequence: left as it is
    if (W == 1 && !alive) {
      async_wait<0>();  // never exit with a copy in flight
      return;
    }
    const long long at = alive ? (long long)len + row : 0;
    const bool fits = alive && len >= 0 && at < (long long)p.mbps * p.bs;
    const int blk = fits ? __ldg(p.tables + (size_t)b * p.mbps + at / p.bs) : -1;
    if (alive && (blk < 0 || blk >= p.num_blocks)) {
      if (sl == 0) raise_error(p.err, kErrBounds);
      alive = false;
    }
    if (W == 1 ? !alive : !__any_sync(0xffffffffu, alive)) {
      async_wait<0>();
      return;
    }
    if (W == 1) alive = true;
    pos = alive ? (int)at : 0;
    slot = (long long)blk * p.Hkv * p.bs + at % p.bs;
    if (values || p.parts == 1) {  // the values, copied as they are, four chunks in flight per lane
      const int cpv = p.dv / V, n = p.Hkv * cpv;
      for (int i0 = sl; alive && i0 < n; i0 += 4 * kSub) {
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i0 + u * kSub;
          if (i < n)
            v[u] = ld16(static_cast<const ET*>(p.v.data) + tt * p.v.token_stride + (i / cpv) * p.v.head_stride +
                        (i % cpv) * V);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i0 + u * kSub;
          if (i < n)
            *reinterpret_cast<uint4*>(static_cast<ET*>(p.v_pool) + (slot + (long long)(i / cpv) * p.bs) * p.dv +
                                      (i % cpv) * V) = v[u];
        }
      }
      if (values) return;
    }
  } else if (p.rot_dim) {
    pos = __ldg(p.positions + tok);
  }
  float2* cs = cs_s[warp * W + ts];
  for (int t = sl; t < half; t += kSub) {
    const float2 w = __ldg(reinterpret_cast<const float2*>(p.freqs) + t);
    float c, s;
    rope_cos_sin_pair(pos, w.x, w.y, &c, &s);
    cs[t] = make_float2(c * p.magnitude, s * p.magnitude);
  }
  __syncwarp();

  const float inv_d = 1.f / (float)p.d;
  int round = 0;
#pragma unroll 1
  for (int seg = 0; seg < 2; ++seg) {  // q heads, then k heads
    const int lo = seg ? k_lo : q_lo, hi = seg ? k_hi : q_hi;
    if (lo >= hi) continue;
    ET* to;
    long long to_stride;
    if (seg && PAGED) {
      to = static_cast<ET*>(p.k_out.data) + slot * p.d;
      to_stride = (long long)p.bs * p.d;
    } else {
      const HeadsView& o = seg ? p.k_out : p.q_out;
      to = static_cast<ET*>(o.data) + tb * o.batch_stride + tt * o.token_stride;
      to_stride = o.head_stride;
    }
    to += (lo + grp) * to_stride + col0;
    to_stride *= kGroups;  // from a row of this lane to its next
    const ET* weight = static_cast<const ET*>(seg ? p.k_weight : p.q_weight);
    // ---- the columns' weights, and the factors of the pairs
    float2 g[2][H2];
#pragma unroll
    for (int e = 0; e < H2; ++e) g[0][e] = g[1][e] = make_float2(1.f, 1.f);
    if (weight && c0 >= 0) Chunk<ET>::unpack(ld16(weight + c0 * V), g[0]);
    if (weight && c1 >= 0) Chunk<ET>::unpack(ld16(weight + c1 * V), g[1]);
    // kTurnHalf: for columns (2e, 2e + 1) of c0 and their partners in c1, fa = w_a cos,
    // fb = -w_b sin, ha = w_a sin, hb = w_b cos. kTurnAdjacent: pair e of chunk s:
    // fa = (w_a cos, w_a sin), fb = (-w_b sin, w_b cos), chunk 1's in ha, hb.
    float2 fa[H2], fb[H2], ha[H2], hb[H2];
    if (TURN == kTurnHalf && turn0) {
#pragma unroll
      for (int e = 0; e < H2; ++e) {
        const int t = c0 * V + 2 * e - p.rot_offset;
        const float2 x = cs[t], z = cs[t + 1];
        fa[e] = make_float2(g[0][e].x * x.x, g[0][e].y * z.x);
        fb[e] = make_float2(-g[1][e].x * x.y, -g[1][e].y * z.y);
        ha[e] = make_float2(g[0][e].x * x.y, g[0][e].y * z.y);
        hb[e] = make_float2(g[1][e].x * x.x, g[1][e].y * z.x);
      }
    }
    if (TURN == kTurnAdjacent && (turn0 || turn1)) {
#pragma unroll
      for (int e = 0; e < H2; ++e) {
        const float2 x = turn0 ? cs[(c0 * V - p.rot_offset) / 2 + e] : make_float2(0.f, 0.f);
        const float2 z = turn1 ? cs[(c1 * V - p.rot_offset) / 2 + e] : make_float2(0.f, 0.f);
        fa[e] = make_float2(g[0][e].x * x.x, g[0][e].x * x.y);
        fb[e] = make_float2(-g[0][e].y * x.y, g[0][e].y * x.x);
        ha[e] = make_float2(g[1][e].x * z.x, g[1][e].x * z.y);
        hb[e] = make_float2(-g[1][e].y * z.y, g[1][e].y * z.x);
      }
    }
#pragma unroll 1
    for (int h = lo + grp; h - grp < hi; h += kRound, ++round) {
      async_wait<kQkStages - 1>();
      uint4 raw[kQkRows][2];
#pragma unroll
      for (int u = 0; u < kQkRows; ++u) {
        // (lanes without a chunk, and rows past the end, work on zeros)
        const bool row = h + u * kGroups < hi;
        raw[u][0] = row && c0 >= 0 ? ring[round % kQkStages][u][0][lane] : make_uint4(0, 0, 0, 0);
        raw[u][1] = row && c1 >= 0 ? ring[round % kQkStages][u][1][lane] : make_uint4(0, 0, 0, 0);
      }
      request();
#pragma unroll
      for (int u = 0; u < kQkRows; ++u) {
        const int r = h + u * kGroups;
        float2 y[2][H2];
        Chunk<ET>::unpack(raw[u][0], y[0]);
        Chunk<ET>::unpack(raw[u][1], y[1]);
        float rs = 1.f;
        if (weight) {
          float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < H2; ++e) s2 = __ffma2_rn(y[1][e], y[1][e], __ffma2_rn(y[0][e], y[0][e], s2));
          float ss = s2.x + s2.y;
#pragma unroll
          for (int off = L / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          rs = rsqrtf(fmaf(ss, inv_d, p.eps));  // within 2 ulp
        }
        const float2 rs2 = make_float2(rs, rs);
        if (TURN == kTurnHalf && turn0) {
#pragma unroll
          for (int e = 0; e < H2; ++e) {
            const float2 a = y[0][e], b = y[1][e];
            y[0][e] = __ffma2_rn(a, fa[e], __fmul2_rn(b, fb[e]));
            y[1][e] = __ffma2_rn(a, ha[e], __fmul2_rn(b, hb[e]));
          }
        } else if (TURN == kTurnAdjacent) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (s ? turn1 : turn0) {
#pragma unroll
              for (int e = 0; e < H2; ++e) {
                const float2 v = y[s][e];
                y[s][e] = __ffma2_rn(make_float2(v.x, v.x), s ? ha[e] : fa[e],
                                     __fmul2_rn(make_float2(v.y, v.y), s ? hb[e] : fb[e]));
              }
            } else if (weight) {
#pragma unroll
              for (int e = 0; e < H2; ++e) y[s][e] = __fmul2_rn(y[s][e], g[s][e]);
            }
          }
        } else if (weight) {
#pragma unroll
          for (int e = 0; e < H2; ++e) {
            y[0][e] = __fmul2_rn(y[0][e], g[0][e]);
            y[1][e] = __fmul2_rn(y[1][e], g[1][e]);
          }
        }
        if (TURN == kTurnAny) {
          // pairs that cross chunks: the weighted row through shared memory, column by column
          float* row = row_s[warp] + lane / L * (2 * L * V);
          __syncwarp();
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int c = s ? c1 : c0;
            if (c >= 0)
#pragma unroll
              for (int e = 0; e < H2; ++e) *reinterpret_cast<float2*>(row + c * V + 2 * e) = y[s][e];
          }
          __syncwarp();
          const auto turn = [&](int col, float v) {
            const int x = col - p.rot_offset;  // place in the rotated slice
            if (x < 0 || x >= p.rot_dim) return v;
            const int t = p.layout == 1 ? (x < half ? x : x - half) : x / 2;
            const bool second = p.layout == 1 ? x >= half : (x & 1) != 0;
            const int away = p.layout == 1 ? half : 1;
            const float other = row[second ? col - away : col + away];
            return second ? fmaf(other, cs[t].y, v * cs[t].x) : fmaf(v, cs[t].x, -other * cs[t].y);
          };
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int c = s ? c1 : c0;
            if (c >= 0)
#pragma unroll
              for (int e = 0; e < H2; ++e) {
                y[s][e].x = turn(c * V + 2 * e, y[s][e].x);
                y[s][e].y = turn(c * V + 2 * e + 1, y[s][e].y);
              }
          }
        }
        if (weight) {
#pragma unroll
          for (int e = 0; e < H2; ++e) {
            y[0][e] = __fmul2_rn(y[0][e], rs2);
            y[1][e] = __fmul2_rn(y[1][e], rs2);
          }
        }
        if (r < hi && alive) {
          if (c0 >= 0) *reinterpret_cast<uint4*>(to) = Chunk<ET>::pack(y[0]);
          if (c1 >= 0) *reinterpret_cast<uint4*>(to + apart) = Chunk<ET>::pack(y[1]);
        }
        to += to_stride;
      }
    }
  }
}

template <typename ET, int L, int TURN, bool PAGED, int W>
cudaError_t launch_qk(QkParams p, cudaStream_t st) {
  const int n = p.run_rows ? (int)(((long long)p.N + W - 1) / W) : 0, lens = PAGED ? p.lens_items : 0;
  const int most = n > lens ? n : lens;
  if (most == 0) return cudaSuccess;
  p.lens_part = p.parts > 1 ? p.parts + 1 : 1;
  p.first_part = n ? 0 : p.lens_part;  // the lengths alone
  const int last_part = !PAGED ? p.parts - 1 : lens ? p.lens_part : p.lens_part - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(((unsigned)most + kQkWarps - 1) / kQkWarps, (unsigned)(last_part - p.first_part + 1));
  cfg.blockDim = dim3(kQkWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_rows_kernel<ET, L, TURN, PAGED, W>, p);
}

template <typename ET, int TURN, bool PAGED>
cudaError_t dispatch_qk(QkParams p, cudaStream_t st) {
  constexpr int V = Elem<ET>::kPerChunk;
  const int cpr = p.d / V, np = p.rot_dim / 2 / V;
  const int pairs = TURN == kTurnHalf ? np + (cpr - 2 * np + 1) / 2 : (cpr + 1) / 2;  // chunk pairs of a row
  const int L = pairs <= 4 ? 4 : pairs <= 8 ? 8 : pairs <= 16 ? 16 : 32;
  // Items per token: as few as keep 16 warps on each of the 152 SMs, at most one
  // round of loads each.
  const int rows = p.H + p.Hk, rounds = (rows + kQkRows * (32 / L) - 1) / (kQkRows * (32 / L));
  const long long want = (152 * 16 + (long long)p.N - 1) / (p.N > 0 ? p.N : 1);
  const int parts = rows == 0 ? 1 : (int)(want < 1 ? 1 : want > rounds ? rounds : want);
  p.part_rows = rows == 0 ? 1 : (rows + parts - 1) / parts;
  p.parts = rows == 0 ? 1 : (rows + p.part_rows - 1) / p.part_rows;
  // Many tokens of few rows: a token for each L lanes, so that no lanes idle and what a token
  // takes beside its rows is shared by as many. Measured, a warp per token and side by side (bf16):
  // 524,288 tokens of 1 + 1 heads of 64 693 and 152 us, 16,384 of 8 + 2 of 128 27.7 and 19.3, of 32 +
  // 8 of 128 (five rounds a warp) 64.2 and 68.4; 8,192 of 14 + 2 of 64 14.0 and 10.0; 4,096 of 8 + 8
  // of 64 7.8 and 8.8, 2,048 of 14 + 2 of 64 (256 warps for the GPU) 4.8 and 8.9. An append's rows
  // may be padding in good part (7,261 rows of 14 + 2 + 2 heads of 64, half of them padding: 9.7
  // and 10.4), so twice as many are asked for.
  const bool side = p.parts == 1 && rounds <= 3 && p.N >= (PAGED ? 8 : 4) * 152 * (32 / L);
  switch (L) {
    case 4: return side ? launch_qk<ET, 4, TURN, PAGED, 8>(p, st) : launch_qk<ET, 4, TURN, PAGED, 1>(p, st);
    case 8: return side ? launch_qk<ET, 8, TURN, PAGED, 4>(p, st) : launch_qk<ET, 8, TURN, PAGED, 1>(p, st);
    case 16: return side ? launch_qk<ET, 16, TURN, PAGED, 2>(p, st) : launch_qk<ET, 16, TURN, PAGED, 1>(p, st);
    default: return launch_qk<ET, 32, TURN, PAGED, 1>(p, st);
  }
}

template <typename ET, bool PAGED>
cudaError_t dispatch_turn(const QkParams& p, cudaStream_t st) {
  constexpr int V = Elem<ET>::kPerChunk;
  const bool half = p.rot_dim && p.layout == 1;
  if (p.rot_offset % V || (half ? p.rot_dim / 2 : p.rot_dim) % V) return dispatch_qk<ET, kTurnAny, PAGED>(p, st);
  return half ? dispatch_qk<ET, kTurnHalf, PAGED>(p, st) : dispatch_qk<ET, kTurnAdjacent, PAGED>(p, st);
}

}  // namespace

cudaError_t launch_qk_rows(const QkParams& p, int bf16, int paged, cudaStream_t st) {
  if (bf16) return paged ? dispatch_turn<__nv_bfloat16, true>(p, st) : dispatch_turn<__nv_bfloat16, false>(p, st);
  return paged ? dispatch_turn<float, true>(p, st) : dispatch_turn<float, false>(p, st);
}

}  // namespace gqa
