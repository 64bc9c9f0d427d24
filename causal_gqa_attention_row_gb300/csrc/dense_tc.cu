// dense_tc.cu -- attention without a causal rule on the tcgen05 tensor cores
// (bf16; (d_k, d_v) = (64, 64), (128, 128) or (192, 128)): rows that all see the same
// keys, as decoder rows against an encoder's states (attn_cross), or the decode rows
// of sequences that share a prefix against that prefix (attn_decode_shared_prefix).
//
//   out[r] = softmax_{j < n_r}(scale * q_r . k_j) v_j,  n_r the keys of row r
//
// What is new against the causal prefill is the shape of the work: few rows and many
// keys. So the rows of a tile are (row i, head of the group) pairs: GH heads of one
// KV head times RPT rows i, GH * RPT <= 128, brought in by one TMA box per 64 columns
// from the [rows, H, d] queries as they lie. A K or V tile then serves all heads of
// the group at once (a group of 4 with 32 rows fills the 128 rows of the MMA; one head
// at a time would fill 32). And the keys are split over CTAs: a unit is a row tile and
// a range of key tiles; where there is more than one range, it leaves (m, l, o) in fp32
// and dense_combine_kernel joins them in a fixed order.
//
// The key loop is the causal prefill's: the roles of the warps, the rings, the two
// softmax warpgroups that take key tiles in turn with an O of their own in TMEM, the
// lazily moved reference max, P in bf16 for the second product (rounded once, a relative
// 2^-9 that averages over the keys; the row sum keeps the fp32 p). See prefill_tc.cu.
// Differences: no diagonal; a row's keys end at its own limit, and in the tile that
// holds the last key of a sequence the V rows behind it are zeroed in shared memory
// before the product reads them, since 0 * NaN of an unwritten row would not be 0;
// warps whose rows are all padding only keep the barriers going.

#include <atomic>

#include "attn_tc.cuh"
#include "tmap.h"

namespace gqa {
namespace {

struct DenseBars : Bars {
  uint64_t v_tail;  // the last V tile's copies, before its rows behind the last key are zeroed
};
static_assert(sizeof(DenseBars) <= 256, "barrier block");

template <int DK, int DV, bool ARMS>
__global__ void __launch_bounds__(kThreads, 1)
    dense_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                    const DenseParams p) {
  using C = Cfg<DK, DV>;
  constexpr int kTileK = C::kTileK, kTileV = C::kTileV, kStagesK = C::kStagesK, kStagesV = C::kStagesV;
  constexpr int kOffQ = C::kOffQ, kOffK = C::kOffK, kOffV = C::kOffV, kOffTab = C::kOffTab;
  constexpr int kOffOut = C::kOffOut, kOffML = C::kOffML;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  DenseBars* bars = reinterpret_cast<DenseBars*>(smem + C::kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == kProducerWarp && lane == 0) {
    mbar_init(&bars->q_full, 1);
    for (int s = 0; s < kStagesK; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
    }
    for (int s = 0; s < kStagesV; ++s) {
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 1);
    }
    for (int w = 0; w < kWG; ++w) {
      mbar_init(&bars->s_full[w], 1);
      mbar_init(&bars->s_free[w], 4);  // one arrival per softmax warp
      mbar_init(&bars->p_full[w], 4);
      mbar_init(&bars->p_half[w], 4);
      mbar_init(&bars->mma_final[w], 1);
      mbar_init(&bars->o_done[w], 1);
    }
    mbar_init(&bars->v_tail, 1);
    bars->abort_flag = 0;
    fence_barrier_init();
    tc::prefetch_tmap(&tm_q);
    tc::prefetch_tmap(&tm_k);
  }
  // the plan's units, the lengths and everything else may come from the kernel before
  grid_dep_wait();

  // ---- the unit: rows i0 .. i0 + n_i - 1 of heads head0 .. head0 + GH - 1, key tiles
  // t0 .. t1 - 1, keys below kv_hi
  DenseUnit u;
  int qb = 0;
  if (p.units) {
    if ((int)blockIdx.x >= __ldcg(p.n_units)) return;
    const int4 a = __ldcg(reinterpret_cast<const int4*>(p.units + blockIdx.x));
    const int4 c = __ldcg(reinterpret_cast<const int4*>(p.units + blockIdx.x) + 1);
    u = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
  } else {
    int x = (int)blockIdx.x;
    const int split = x % p.n_splits;
    x /= p.n_splits;
    u.i0 = (x % p.n_tiles) * p.RPT;
    x /= p.n_tiles;
    const int hc = x % p.n_hchunks;
    x /= p.n_hchunks;
    u.kvh = x % p.Hkv;
    u.seq = qb = x / p.Hkv;
    u.head0 = u.kvh * p.G + hc * p.GH;
    u.n_i = min(p.RPT, p.n_i - u.i0);
    u.kv_hi = p.kv_lens ? __ldg(p.kv_lens + u.seq) : p.S_kv;
    if (u.kv_hi < 0 || u.kv_hi > p.S_kv) {  // no such keys: zeros
      if (threadIdx.x == 0 && split == 0 && u.i0 == 0 && u.head0 == 0) raise_error(p.err, kErrBounds);
      u.kv_hi = 0;
    }
    u.t0 = min(split * p.split_tiles, (u.kv_hi + kBN - 1) / kBN);
    u.t1 = min((split + 1) * p.split_tiles, (u.kv_hi + kBN - 1) / kBN);
  }
  const int rows = u.n_i * p.GH;  // rows of the tile in use
  const int n_kv = u.t1 - u.t0;
  float* part = p.partial ? p.partial + (size_t)blockIdx.x * (kBM * (DV + 2)) : nullptr;
  if (n_kv <= 0) {  // no keys: an empty partial, or zeros
    for (int r = threadIdx.x; r < rows; r += kThreads) {
      if (part) {
        part[kBM * DV + r] = -INFINITY;
        part[kBM * DV + kBM + r] = 0.f;
      } else {
        uint4* o = reinterpret_cast<uint4*>(
            p.out + (((size_t)qb * p.n_i + u.i0 + r / p.GH) * p.H + u.head0 + r % p.GH) * DV);
        for (int c = 0; c < DV / 8; ++c) o[c] = make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }
  if (warp == kProducerWarp && lane == 0) {
    // Q and the first K tile load while the rest of the CTA sets up
    mbar_arrive_expect_tx(&bars->q_full, (uint32_t)(C::kCBK * p.GH * p.RPT * 128));
#pragma unroll
    for (int cb = 0; cb < C::kCBK; ++cb)
      tc::tma_load_4d(smem + kOffQ + cb * kBlk, &tm_q, cb * 64, u.head0, u.i0, qb, &bars->q_full);
    // test hook: withheld, the first K tile is never requested (nothing is left in
    // flight), so the first wait on it runs into its bound and the CTA gives up
    if (!p.debug_withhold)
      load_kv_tile<C::kCBK>(&tm_k, smem + kOffK, &bars->k_full[0], u.t0, u.kvh, u.seq, p, u.kv_hi);
  }
  if (warp == kMmaWarp0) {
    tc::tmem_alloc(&bars->tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  grid_dep_launch();  // the next launch may start setting up on the SMs this grid frees

  if (warp >= kProducerWarp) {
    regs_dec<kCtrlRegs>();  // the whole control warpgroup, right at the top of its branch
    if (warp == kProducerWarp || warp == kProducerVWarp) {
      // ================= TMA producers: Q and K (warp 8), V (warp 11) =================
      const bool is_k = warp == kProducerWarp;
      // Paged: the entries of the unit's blocks into shared memory first (the planner
      // keeps a unit within kTabEntries of them)
      const int* tab = nullptr;
      if (p.tables) {
        int* st_tab = reinterpret_cast<int*>(smem + kOffTab);
        const int first = u.t0 * (kBN / p.bs);
        const int n_tab = min(min(p.mbps, (min(u.kv_hi, u.t1 * kBN) + p.bs - 1) / p.bs) - first, kTabEntries);
        for (int i = (is_k ? 0 : 32) + lane; i < n_tab; i += 64)
          st_tab[i] = __ldg(p.tables + (size_t)u.seq * p.mbps + first + i);
        named_bar_sync(3, 64);
        tab = st_tab - first;  // indexed by the sequence's block
      }
      const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
      uint64_t* full = is_k ? bars->k_full : bars->v_full;
      uint64_t* empty = is_k ? bars->k_empty : bars->v_empty;
      unsigned char* ring = smem + (is_k ? kOffK : kOffV);
      const int tile_bytes = is_k ? kTileK : kTileV;
      const int stages = is_k ? kStagesK : kStagesV;
      if (!is_k && lane == 0) tc::prefetch_tmap(tm);
      int issued_last[kStagesK];
#pragma unroll
      for (int st = 0; st < kStagesK; ++st) issued_last[st] = -1;
      int j = 0;
      if (is_k) {  // Q and K_0 went out before the setup barrier
        issued_last[0] = p.debug_withhold ? -1 : 0;
        j = 1;
      }
      for (; j < n_kv; ++j) {
        const int st = j % stages;
        if (j >= stages) {
          bool w = true;
          if (lane == 0) w = wait_or_abort(&empty[st], ((j / stages) - 1) & 1, bars, p.err);
          if (!__shfl_sync(0xffffffffu, w, 0)) break;
        }
        if (is_k) {
          load_kv_tile_warp<C::kCBK>(tm, ring + st * tile_bytes, &full[st], u.t0 + j, u.kvh, u.seq, p, u.kv_hi, tab,
                                     lane);
        } else {
          const int valid = u.kv_hi - (u.t0 + j) * kBN;  // keys of the tile
          unsigned char* dst = ring + st * tile_bytes;
          if (valid >= kBN) {
            load_kv_tile_warp<C::kCBV>(tm, dst, &full[st], u.t0 + j, u.kvh, u.seq, p, u.kv_hi, tab, lane);
          } else {
            // the unit's last tile: its copies land on a barrier of their own, the rows
            // behind the last key are zeroed (every 64-column block; the swizzle moves
            // 16-byte chunks within a row only), then the stage is handed over
            load_kv_tile_warp<C::kCBV>(tm, dst, &bars->v_tail, u.t0 + j, u.kvh, u.seq, p, u.kv_hi, tab, lane);
            if (!warp_wait_tc(&bars->v_tail, 0, bars, p.err)) {
              mbar_wait(&bars->v_tail, 0);  // another warp gave up: still never leave with a copy in flight
              break;
            }
            for (int i = lane; i < (kBN - valid) * 8 * C::kCBV; i += 32) {
              const int chunk = i % 8, cb = (i / 8) % C::kCBV, row = valid + i / (8 * C::kCBV);
              *reinterpret_cast<uint4*>(dst + cb * kBlk + row * 128 + chunk * 16) = make_uint4(0, 0, 0, 0);
            }
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
          }
        }
        issued_last[st] = j;
      }
      if (lane == 0) {
        // never exit with a load in flight
        if (is_k && !mbar_wait(&bars->q_full, 0)) raise_error(p.err, kErrTimeout);
        for (int st = 0; st < stages; ++st)
          if (issued_last[st] >= 0 && !mbar_wait(&full[st], (issued_last[st] / stages) & 1))
            raise_error(p.err, kErrTimeout);
      }
    } else if (warp == kMmaWarp0 || warp == kMmaWarp0 + 1) {
      // ================= MMA issuers: warp 9 for warpgroup 0, warp 10 for warpgroup 1 =================
      const int w = warp - kMmaWarp0;
      if (lane == 0) {
        const int n_mine = (n_kv - w + 1) / 2;
        const uint32_t idS = tc::idesc_bf16_f32(kBM, kBN, false);
        const uint32_t idO = tc::idesc_bf16_f32(kBM, DV, true);
        constexpr uint64_t kHi = tc::desc_sw128_hi(0, 1024);
        const uint64_t dQ = kHi | (smem_u32(smem + kOffQ) >> 4);
        const uint64_t dK0 = kHi | (smem_u32(smem + kOffK) >> 4);
        const uint64_t dV0 = tc::desc_sw128_hi(C::kCBV > 1 ? kBlk : 0, 1024) | (smem_u32(smem + kOffV) >> 4);
        const uint32_t dS = tmem + C::col_s(w), dO = tmem + C::col_o(w), tP = tmem + C::col_p(w);
        auto issue_s = [&](int j) -> bool {  // S_w = Q K_j^T
          const int st = j % kStagesK;
          if (!wait_or_abort(&bars->k_full[st], (j / kStagesK) & 1, bars, p.err)) return false;
          tc::fence_after_sync();
          const uint64_t dK = dK0 + (uint64_t)((st * kTileK) >> 4);
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk) {
            const uint32_t at = (kk / 4) * kBlk + (kk % 4) * 32;
            tc::mma_f16_ss(dS, dQ + (at >> 4), dK + (at >> 4), idS, kk > 0);
          }
          tc::mma_commit(&bars->s_full[w]);
          tc::mma_commit(&bars->k_empty[st]);  // the K stage is free once S_j is done
          return true;
        };
        bool ok = n_mine > 0 && wait_or_abort(&bars->q_full, 0, bars, p.err) && issue_s(w);
        for (int k = 0; ok && k < n_mine; ++k) {
          const int j = 2 * k + w;
          if (!C::kAlias && k + 1 < n_mine) ok = wait_or_abort(&bars->s_free[w], k & 1, bars, p.err) && issue_s(j + 2);
          if (!ok || !wait_or_abort(C::kAlias ? &bars->p_half[w] : &bars->p_full[w], k & 1, bars, p.err)) break;
          const int st = j % kStagesV;
          if (!wait_or_abort(&bars->v_full[st], (j / kStagesV) & 1, bars, p.err)) break;
          tc::fence_after_sync();
          const uint64_t dV = dV0 + (uint64_t)((st * kTileV) >> 4);
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk) {
            if (C::kAlias && kk == kBN / 32) {
              ok = wait_or_abort(&bars->p_full[w], k & 1, bars, p.err);
              if (!ok) break;
              tc::fence_after_sync();
            }
            tc::mma_f16_ts(dO, tP + kk * 8, dV + kk * (2048 >> 4), idO, (k > 0 || kk > 0));
          }
          if (!ok) break;
          tc::mma_commit(&bars->o_done[w]);
          tc::mma_commit(&bars->v_empty[st]);
          // d_v = 128: P_j sits in S_w, so S_{j+2} waits for PV_j
          if (C::kAlias && k + 1 < n_mine) {
            ok = wait_or_abort(&bars->o_done[w], k & 1, bars, p.err);
            if (ok) {
              tc::fence_after_sync();
              ok = issue_s(j + 2);
            }
          }
        }
        // every MMA issued above has completed before TMEM is released
        tc::mma_commit(&bars->mma_final[w]);
        if (!mbar_wait(&bars->mma_final[w], 0)) raise_error(p.err, kErrTimeout);
      }
    }
  } else {
    // ================= softmax warpgroups =================
    regs_inc<kSoftmaxRegs>();  // both softmax warpgroups, right at the top of their branch
    const int wg = warp >> 2;
    const int quarter = warp & 3;       // TMEM lanes this warp may access
    const int r = quarter * 32 + lane;  // row of the tile
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const bool warp_live = quarter * 32 < rows;
    const int row_i = u.i0 + min(r, rows - 1) / p.GH, row_h = u.head0 + min(r, rows - 1) % p.GH;
    // keys of this row: [lo_key, lim)
    int lim = u.kv_hi, lo_key = 0, pos = 0;
    if (p.seq_lens) {  // a row is a sequence of its own length; its position is its last key's
      const int len = __ldg(p.seq_lens + row_i);
      pos = len - 1;
      lim = len >= 1 && len <= p.S_kv ? min(u.kv_hi, len) : 0;
      if (ARMS) lo_key = first_visible_key(pos, p.window);
    }
    if (r >= rows) lim = 0;
    // With the arms the scores are moved into log2 units before the max, so the
    // exponent's multiplier is 1; plain: the raw q.k and the scale folded into it.
    const float qs = ARMS ? 1.f : p.qscale;
    const float th = kRescaleLog2 / qs;
    const float alibi2 = ARMS && p.alibi ? __ldg(p.alibi + row_h) * kLog2e : 0.f;
    float m_ref = -INFINITY;
    float l_run = 0.f;  // the row sum of this warpgroup's p, against m_ref
    const uint32_t tS = tmem + lane_addr + C::col_s(wg);
    const uint32_t tO = tmem + lane_addr + C::col_o(wg);
    const uint32_t tP = tmem + lane_addr + C::col_p(wg);
    const float2 qs2 = make_float2(qs, qs);
    const int n_mine = (n_kv - wg + 1) / 2;  // key tiles this warpgroup handles
    bool alive = true;
    // d_v = 128: warpgroup 1 starts half a tile behind warpgroup 0 (see prefill_tc.cu)
    if (C::kAlias && wg == 1 && n_kv > 1) alive = warp_wait_tc(&bars->p_full[0], 0, bars, p.err);
    for (int k = 0; alive && k < n_mine; ++k) {
      const int j0 = (u.t0 + 2 * k + wg) * kBN;  // the tile's first key
      if (!warp_wait_tc(&bars->s_full[wg], k & 1, bars, p.err)) {
        alive = false;
        break;
      }
      if (!warp_live) {
        // padding rows: P may hold anything, only the barriers matter. At d_v = 64 S_{j+2}
        // is issued before PV_j, so this warp has to be held back here as the others are
        // by P_w, or its second arrival on p_full would stand in for another warp's first.
        if (!C::kAlias && k >= 1 && !warp_wait_tc(&bars->o_done[wg], (k - 1) & 1, bars, p.err)) {
          alive = false;
          break;
        }
        if (lane == 0) {
          mbar_arrive(&bars->s_free[wg]);
          if (C::kAlias) mbar_arrive(&bars->p_half[wg]);
          mbar_arrive(&bars->p_full[wg]);
        }
        continue;
      }
      tc::fence_after_sync();
      // ---- the S row into registers; S_w is then free for S_{j+2}
      uint32_t sv[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::tmem_ld_32x32b_x32(tS + c * 32, sv[c]);
      tc::tmem_ld_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->s_free[wg]);
      if (ARMS) {  // scale, softcap, ALiBi: log2 units, as in prefill_tc.cu
        const float base = alibi2 * (float)(j0 - pos);
        if (p.cap_out > 0.f) {
          const float2 k2 = make_float2(p.cap_in * 2.8853900817779268f, p.cap_in * 2.8853900817779268f);  // 2 log2(e)
          const float2 one2 = make_float2(1.f, 1.f);
          const float2 m2 = make_float2(-2.f * p.cap_out, -2.f * p.cap_out);
          const float2 a2 = make_float2(p.cap_out + base, p.cap_out + base);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 t = __fmul2_rn(make_float2(__uint_as_float(sv[c][e]), __uint_as_float(sv[c][e + 1])), k2);
              const float2 dn = __fadd2_rn(make_float2(ex2f(t.x), ex2f(t.y)), one2);
              const float2 y = __ffma2_rn(make_float2(rcpf(dn.x), rcpf(dn.y)), m2, a2);
              sv[c][e] = __float_as_uint(y.x);
              sv[c][e + 1] = __float_as_uint(y.y);
            }
        } else {
          const float2 q2 = make_float2(p.qscale, p.qscale), b2 = make_float2(base, base);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 y =
                  __ffma2_rn(make_float2(__uint_as_float(sv[c][e]), __uint_as_float(sv[c][e + 1])), q2, b2);
              sv[c][e] = __float_as_uint(y.x);
              sv[c][e + 1] = __float_as_uint(y.y);
            }
        }
        if (__any_sync(0xffffffffu, alibi2 != 0.f)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              sv[c][e] = __float_as_uint(fmaf(alibi2, (float)(c * 32 + e), __uint_as_float(sv[c][e])));
        }
      }
      // keys that some row of the warp does not see weigh zero for it
      if (__any_sync(0xffffffffu, j0 + kBN > lim || (ARMS && j0 < lo_key))) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int key = j0 + c * 32 + e;
            if (key >= lim || key < lo_key) sv[c][e] = __float_as_uint(-INFINITY);
          }
      }
      // ---- the tile's row max; the reference moves only past the threshold
      float mx8[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) mx8[e] = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 32; e += 2)
          mx8[(e >> 1) & 7] = fmax3(mx8[(e >> 1) & 7], __uint_as_float(sv[c][e]), __uint_as_float(sv[c][e + 1]));
      const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                             fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
      if (k == 0) {
        m_ref = mx;
      } else {
        const bool grow = mx > m_ref + th;
        if (__any_sync(0xffffffffu, grow)) {
          float f = 1.f;
          if (grow) {
            f = ex2f((m_ref - mx) * qs);  // 0 while m_ref = -inf
            m_ref = mx;
          }
          if (!C::kAlias && !warp_wait_tc(&bars->o_done[wg], (k - 1) & 1, bars, p.err)) {
            alive = false;
            break;
          }
          tc::fence_after_sync();
          uint32_t o[32];
#pragma unroll
          for (int c = 0; c < DV / 32; ++c) {
            tc::tmem_ld_32x32b_x32(tO + c * 32, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tc::tmem_st_32x32b_x32(tO + c * 32, o);
          }
          tc::tmem_st_wait();
          l_run *= f;
        }
      }
      // ---- p = 2^(s*qs - m*qs), the fp32 row sum of these p, and P as bf16 pairs
      const float mq = m_ref == -INFINITY ? 0.f : m_ref * qs;  // no visible key yet: all p are 0
      const float2 nmq2 = make_float2(-mq, -mq);
      float2 ls[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) ls[e] = make_float2(0.f, 0.f);
      uint32_t pw[4][16];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int t = 0; t < 16; ++t)
          pw[c][t] = exp2_pair(__uint_as_float(sv[c][2 * t]), __uint_as_float(sv[c][2 * t + 1]), qs2, nmq2, ls[t & 3]);
        if (C::kAlias) {  // P over S_j's own columns, already read; half of PV_j starts at half of P
          tc::tmem_st_32x32b_x16(tP + c * 16, pw[c]);
          if (c == 1) {
            tc::tmem_st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_half[wg]);
          }
        }
      }
      l_run += ((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y)) + ((ls[2].x + ls[2].y) + (ls[3].x + ls[3].y));
      // ---- d_v = 64: P_w is free once this warpgroup's previous PV has read it
      if (!C::kAlias) {
        if (k >= 1) {
          if (!warp_wait_tc(&bars->o_done[wg], (k - 1) & 1, bars, p.err)) {
            alive = false;
            break;
          }
          tc::fence_after_sync();
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::tmem_st_32x32b_x16(tP + c * 16, pw[c]);
      }
      tc::tmem_st_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->p_full[wg]);
    }
    // ---- the two warpgroups exchange (m, l); each merges half of the columns of O_0 and O_1
    bool have_o = alive && n_mine > 0;
    if (have_o) {
      have_o = warp_wait_tc(&bars->o_done[wg], (n_mine - 1) & 1, bars, p.err);
      tc::fence_after_sync();
    }
    float* ml = reinterpret_cast<float*>(smem + kOffML + wg * kTileK);  // K stage wg: consumed by now
    ml[r] = have_o ? m_ref : -INFINITY;
    ml[kBM + r] = have_o ? l_run : 0.f;  // l = 0: no visible key, or no tile at all
    tc::fence_before_sync();
    named_bar_sync(1, kWG * 128);
    tc::fence_after_sync();
    const float* ml0 = reinterpret_cast<const float*>(smem + kOffML);
    const float* ml1 = reinterpret_cast<const float*>(smem + kOffML + kTileK);
    const float m0 = ml0[r], l0 = ml0[kBM + r], m1 = ml1[r], l1 = ml1[kBM + r];
    // (a NaN among a row's scores makes its l NaN, and has to reach the output)
    const bool use0 = l0 != 0.f, use1 = l1 != 0.f;
    const float M = fmaxf(use0 ? m0 : -INFINITY, use1 ? m1 : -INFINITY);
    float c0 = use0 ? ex2f((m0 - M) * qs) : 0.f;
    float c1 = use1 ? ex2f((m1 - M) * qs) : 0.f;
    const float l = c0 * l0 + c1 * l1;
    if (part) {  // (m in log2 units, l) of the row, once
      if (wg == 0 && r < rows) {
        part[kBM * DV + r] = M * qs;
        part[kBM * DV + kBM + r] = l;
      }
    } else {
      const float inv = l != 0.f ? 1.f / l : 0.f;
      c0 *= inv;
      c1 *= inv;
    }
    unsigned char* so = smem + kOffOut;
#pragma unroll
    for (int cc = 0; cc < DV / 64; ++cc) {
      const int col0 = wg * (DV / 2) + cc * 32;
      uint32_t o0[32], o1[32];
      tc::tmem_ld_32x32b_x32(tmem + lane_addr + C::col_o(0) + col0, o0);
      if (n_kv > 1) tc::tmem_ld_32x32b_x32(tmem + lane_addr + C::col_o(1) + col0, o1);
      tc::tmem_ld_wait();
      float x[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        x[e] = use0 ? __uint_as_float(o0[e]) * c0 : 0.f;
        if (n_kv > 1 && use1) x[e] = fmaf(__uint_as_float(o1[e]), c1, x[e]);
      }
      if (part) {
        // [column / 4][row][4]: the 32 rows of a warp write 512 contiguous bytes
        if (r < rows) {
#pragma unroll
          for (int t = 0; t < 8; ++t)
            *reinterpret_cast<float4*>(part + ((size_t)(col0 / 4 + t) * kBM + r) * 4) =
                make_float4(x[4 * t], x[4 * t + 1], x[4 * t + 2], x[4 * t + 3]);
        }
      } else {
        // the output tile over Q, in the 128-byte swizzle of the output's tensor map
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          uint32_t w4[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) w4[v] = pack_bf16(x[t * 8 + 2 * v], x[t * 8 + 2 * v + 1]);
          const int col = col0 + t * 8;
          const int chunk = (col % 64) / 8;
          *reinterpret_cast<uint4*>(so + (col / 64) * kBlk + r * 128 + ((chunk ^ (r & 7)) * 16)) =
              make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
      }
    }
    if (!part) {
      tc::fence_async_smem();  // the tile visible to the TMA engine
      named_bar_sync(2, kWG * 128);
      if (threadIdx.x == 0) {
        // rows past the end of the sequence fall outside the tensor and are not written
#pragma unroll
        for (int cb = 0; cb < C::kCBV; ++cb) tc::tma_store_4d(&tm_o, so + cb * kBlk, cb * 64, u.head0, u.i0, qb);
        tc::bulk_commit_group();
        tc::bulk_wait_group_read0();  // shared memory stays valid until the store has read it
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMmaWarp0) tc::tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------------------
// Joins the partial results of a row, in a fixed order (key ranges of the row's tile,
// then, for the shared-prefix step, the splits of the sequence's own rows):
//   M = max m_s (and the sink logit),  out = sum 2^(m_s - M) o_s / sum 2^(m_s - M) l_s
// A warp per row; lane c takes columns 4c .. 4c + 3. Latency bounds it: the loads of
// four ranges are in flight at a time.
__global__ void __launch_bounds__(256) dense_combine_kernel(const DenseCombine p) {
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= p.n_rows) return;
  const int h = (int)(row % p.H);
  const int i = (int)(row / p.H % p.n_i);  // shared prefix: the sequence
  const int b = (int)(row / p.H / p.n_i);
  const int kvh = h / p.G, hc = h % p.G / p.GH;
  // ---- the row's units: n of them from unit0, one after another
  long long unit0 = 0;
  int n = 0, in_tile = 0, s_lo = 0, s_n = 0;
  if (p.groups) {
    const int len = __ldg(p.seq_lens + i);
    if (len < 1 || len > p.capacity) return;  // the attention kernel wrote zeros
    const int lo = __ldcg(p.kv_lo + i);
    s_n = (len + p.split_rows - 1) / p.split_rows;
    s_lo = max(first_visible_key(len - 1, p.window), lo) / p.split_rows;
    if (lo == 0) {
      if (s_n - s_lo <= 1) return;  // the attention kernel wrote the output itself
    } else {
      if (lo >= len) s_n = s_lo;  // no rows of its own
      const DenseGroup g = p.groups[__ldcg(p.group_of + i)];
      n = g.n_splits;
      in_tile = i - g.first;
      unit0 = g.unit0 + ((long long)(kvh * p.n_hchunks + hc) * g.tiles + in_tile / p.RPT) * n;
      in_tile = in_tile % p.RPT * p.GH + h % p.GH;
    }
  } else {
    n = p.n_splits;
    unit0 = ((((long long)b * p.Hkv + kvh) * p.n_hchunks + hc) * p.n_tiles + i / p.RPT) * n;
    in_tile = i % p.RPT * p.GH + h % p.GH;
  }
  const int dv = p.dv;
  const size_t unit_floats = (size_t)kBM * (dv + 2);
  const float* U = p.partial + (size_t)unit0 * unit_floats;
  const float* R = p.rows_partial ? p.rows_partial + (size_t)row * p.max_splits * (dv + 2) : nullptr;
  const float z2 = p.sinks ? __ldg(p.sinks + h) * kLog2e : -INFINITY;
  float M = z2;
  for (int s = lane; s < n; s += 32) M = fmaxf(M, __ldcg(U + s * unit_floats + kBM * dv + in_tile));
  for (int s = s_lo + lane; s < s_n; s += 32) M = fmaxf(M, __ldcg(R + (size_t)s * (dv + 2)));
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const int c = lane;
  const bool col = 4 * c < dv;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = p.sinks && M != -INFINITY ? exp2f(z2 - M) : 0.f;
  const int total = n + (s_n - s_lo);
  constexpr int kFlight = 4;
  for (int s0 = 0; s0 < total; s0 += kFlight) {
    float4 o[kFlight];
    float m[kFlight], l[kFlight];
#pragma unroll
    for (int t = 0; t < kFlight; ++t) {
      const int s = s0 + t;
      m[t] = -INFINITY;
      l[t] = 0.f;
      o[t] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s >= total) continue;
      if (s < n) {
        const float* u = U + s * unit_floats;
        m[t] = __ldcg(u + kBM * dv + in_tile);
        l[t] = __ldcg(u + kBM * dv + kBM + in_tile);
        if (col) o[t] = __ldcg(reinterpret_cast<const float4*>(u) + (size_t)c * kBM + in_tile);
      } else {
        const float* u = R + (size_t)(s_lo + s - n) * (dv + 2);
        m[t] = __ldcg(u);
        l[t] = __ldcg(u + 1);
        if (col) {
          const float2 a = __ldcg(reinterpret_cast<const float2*>(u + 2) + 2 * c);
          const float2 d = __ldcg(reinterpret_cast<const float2*>(u + 2) + 2 * c + 1);
          o[t] = make_float4(a.x, a.y, d.x, d.y);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kFlight; ++t) {
      if (l[t] == 0.f) continue;  // no visible key: o was not written
      const float w = exp2f(m[t] - M);
      den = fmaf(w, l[t], den);
      acc.x = fmaf(w, o[t].x, acc.x);
      acc.y = fmaf(w, o[t].y, acc.y);
      acc.z = fmaf(w, o[t].z, acc.z);
      acc.w = fmaf(w, o[t].w, acc.w);
    }
  }
  if (!col) return;
  const float inv = den != 0.f ? 1.f / den : 0.f;
  uint2 v;
  v.x = pack_bf16(acc.x * inv, acc.y * inv);
  v.y = pack_bf16(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(p.out + (size_t)row * dv + 4 * c) = v;
}

// A 4-D bf16 tensor of rows of d elements; box = 64 x b1 x b2 x 1, 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, int d, uint64_t d1, uint64_t d2, uint64_t d3, uint32_t box1,
              uint32_t box2) {
  const uint64_t dims[4] = {(uint64_t)d, d1, d2, d3};
  const uint64_t strides[3] = {(uint64_t)d * 2, (uint64_t)d * 2 * d1, (uint64_t)d * 2 * d1 * d2};
  const uint32_t box[4] = {64, box1, box2, 1};
  return make_tmap_bf16(m, base, dims, strides, box);
}

template <int DK, int DV, bool ARMS>
cudaError_t launch_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& to,
                     const DenseParams& p, long long units, cudaStream_t st) {
  using C = Cfg<DK, DV>;
  int dev = 0;
  cudaGetDevice(&dev);
  static std::atomic<unsigned long long> attr_done{0};  // per device, per instantiation
  if (dev >= 64 || !(attr_done.load(std::memory_order_acquire) >> dev & 1ull)) {
    // The register hand-over inside the kernel assumes exactly kLaunchRegs per
    // thread at launch; a build with any other allocation is refused.
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, dense_tc_kernel<DK, DV, ARMS>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kLaunchRegs) return cudaErrorNotSupported;
    e = cudaFuncSetAttribute(dense_tc_kernel<DK, DV, ARMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done.fetch_or(1ull << dev, std::memory_order_release);
  }
  if (units <= 0) return cudaSuccess;
  if (units > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)units);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dense_tc_kernel<DK, DV, ARMS>, tq, tk, tv, to, p);
}

}  // namespace

bool dense_tc_supported(int bf16, int dk, int dv, int bs) {
  const bool widths = (dk == 64 && dv == 64) || (dk == 128 && dv == 128) || (dk == 192 && dv == 128);
  return bf16 == 1 && widths && (bs == 0 || (bs % 8 == 0 && kBN % bs == 0));
}

void dense_rows(int G, int* GH, int* RPT) {
  int g = G < kBM ? G : kBM;
  while (G % g) --g;
  *GH = g;
  *RPT = kBM / g;
}

// The queries [n_b, n_i, H, d_k] and outputs [n_b, n_i, H, d_v]; k, v contiguous
// [n_b, Hkv, S_kv, d] (p.tables NULL) or pools [num_blocks, Hkv, bs, d].
cudaError_t launch_dense_tc(const void* q, const void* k, const void* v, const DenseParams& p, int n_b, int dk, int dv,
                            long long units, bool arms, cudaStream_t st) {
  if (!dense_tc_supported(1, dk, dv, p.tables ? p.bs : 0) || !(p.qscale > 0.f)) return cudaErrorNotSupported;
  CUtensorMap tq, tk, tv, to;
  if (!make_map(&tq, q, dk, p.H, p.n_i, n_b, p.GH, p.RPT)) return cudaErrorInvalidValue;
  if (p.tables) {
    if (!make_map(&tk, k, dk, p.bs, p.Hkv, p.num_blocks, p.bs, 1)) return cudaErrorInvalidValue;
    if (!make_map(&tv, v, dv, p.bs, p.Hkv, p.num_blocks, p.bs, 1)) return cudaErrorInvalidValue;
  } else {
    if (!make_map(&tk, k, dk, p.S_kv, p.Hkv, n_b, kBN, 1)) return cudaErrorInvalidValue;
    if (!make_map(&tv, v, dv, p.S_kv, p.Hkv, n_b, kBN, 1)) return cudaErrorInvalidValue;
  }
  if (!make_map(&to, p.out, dv, p.H, p.n_i, n_b, p.GH, p.RPT)) return cudaErrorInvalidValue;
  if (arms) {
    if (dk == 64) return launch_d<64, 64, true>(tq, tk, tv, to, p, units, st);
    if (dk == 128) return launch_d<128, 128, true>(tq, tk, tv, to, p, units, st);
    return launch_d<192, 128, true>(tq, tk, tv, to, p, units, st);
  }
  if (dk == 64) return launch_d<64, 64, false>(tq, tk, tv, to, p, units, st);
  if (dk == 128) return launch_d<128, 128, false>(tq, tk, tv, to, p, units, st);
  return launch_d<192, 128, false>(tq, tk, tv, to, p, units, st);
}

cudaError_t launch_dense_combine(const DenseCombine& p, cudaStream_t st) {
  if (p.n_rows <= 0) return cudaSuccess;
  const long long blocks = (p.n_rows + 7) / 8;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dense_combine_kernel, p);
}

}  // namespace gqa
