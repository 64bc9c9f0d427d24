// dense_tc.cu -- attention without a causal rule on the tcgen05 tensor cores
// (bf16; (d_k, d_v) = (64, 64), (128, 128) or (192, 128)): rows that all see the same
// keys, as decoder rows against an encoder's states (attn_cross), the decode rows of
// sequences that share a prefix against that prefix, and a sequence's decode row against
// its own keys (attn_decode_shared_prefix).
//
//   out[r] = softmax_{j < n_r}(scale * q_r . k_j) v_j,  n_r the keys of row r
//
// What is new against the causal prefill is the shape of the work: few rows and many
// keys. So the rows of a tile are (row i, head of the group) pairs: GH heads of one
// KV head times RPT rows i, GH * RPT <= 128, brought in by one TMA box per 64 columns
// from the [rows, H, d] queries as they lie. A K or V tile then serves all heads of
// the group at once (a group of 4 with 32 rows fills the 128 rows of the MMA; one head
// at a time would fill 32). The keys are split: a unit is a row tile and a range of
// keys; where a row has more than one range, each leaves (m, l, o) in fp32 and
// dense_combine_kernel joins them in a fixed order.
//
// A tile of 128 keys (64 KB of K and V at d = 128) takes a CTA about 1.1 us whatever rows it
// has: 58 GB/s, above the 45 GB/s that is an SM's share of HBM. So rows that stream their
// own keys (M = 4 of 128 rows in use) run here too, in the same list as the prefixes, and
// the two share the GPU without a boundary between them.
//
// The kernel is persistent: a CTA per SM with two independent halves, each a softmax
// warpgroup with a producer warp and an MMA warp of its own, its own Q buffer, K and V
// stages and TMEM (S, P, O), working off units slot, slot + slots, ... (slot = CTA + CTAs *
// half, so that a list shorter than the slots spreads over the SMs first). While one half
// is in its softmax the other's products run. The producer runs ahead into the next unit
// as stages come free, so a unit costs its tiles plus one epilogue, not a launch, a set-up
// and a first load. The shared prefixes' units are drawn from a ticket counter; those of
// attn_cross go round by slot: alike but for lengths on the device, which shorten a sequence's
// last unit and leave those behind it empty.
//
// Measured at 32 heads on 8 KV heads of 128, plan and combine included: 64 sequences behind
// a prefix of 8,192 keys with up to 512 of their own 42 us; 256 sequences behind four prefixes
// of 16,384 keys with up to 1,024 of their own 170 us (4.7 TB/s of rows read once, 0.70 of the
// copy bandwidth); attn_cross of 8 x 1,024 rows on 2,048 to 4,096 keys (364 GFLOP) 282 us in a burst
// at 2,070 MHz (1.29 PFLOP/s, 0.68 of the measured bf16 rate), 292 us after seconds at the power
// cap (1,390 W, 1,980 MHz). What bounds them is a half's time from tile to tile, of 1,024 cycles
// of products: in the last case about 3,200 cycles, S, softmax and PV of a half one after
// another; in the second a third more, for K and V that come from HBM through one stage each.
//
//   warps 0-3, 4-7   softmax of half 0, 1: thread t owns row t of the tile (TMEM lane t)
//   warps 8, 11      TMA producer of half 0, 1 (Q once a unit, then K and V tiles; paged:
//                    a lane per block, its table entry fetched a tile ahead)
//   warps 9, 10      MMA of half 0, 1 (warp 9 also allocates and frees TMEM)
//
// Per tile and half, as in the causal prefill (see prefill_tc.cu): S into registers, row
// max, lazily moved reference max, fp32 exponentials, P in bf16 for the second product
// (rounded once, a relative 2^-8 at most that averages over the keys; the row sum keeps the fp32
// p). At d_v = 64 S_{j+1} is issued as soon as S_j is in registers; at d_v = 128 P lies over
// S, so S_{j+1} waits for PV_j, of which half is issued at half of P. All rows of a unit see
// the same keys: those behind the last one, and those in a sequence's own first tile that its
// window hides, weigh zero, and their V rows are zeroed in shared memory before the product
// reads them, since 0 * NaN of an unwritten row would not be 0. Warps whose rows are all
// padding only keep the barriers going.

#include <atomic>
#include <climits>

#include "attn_tc.cuh"
#include "tmap.h"

namespace gqa {
namespace {

// Sizes for head widths DK, DV. Halves per CTA: two, one where two do not fit.
template <int DK, int DV>
struct DenseCfg {
  static constexpr int kCBK = DK / 64, kCBV = DV / 64;
  static constexpr int kTileK = kCBK * kBlk, kTileV = kCBV * kBlk;
  static constexpr bool kAlias = DV > 64;  // P over the first 64 columns of S
  static constexpr int kHalves = DK > 128 ? 1 : 2;
  static constexpr int kStages = DK > 128 ? 2 : DK > 64 ? 1 : 2;  // K and V stages of a half
  __host__ __device__ static constexpr uint32_t col_s(int w) { return kAlias ? (128 + DV) * w : 128 * w; }
  __host__ __device__ static constexpr uint32_t col_o(int w) { return kAlias ? (128 + DV) * w + 128 : 256 + 64 * w; }
  __host__ __device__ static constexpr uint32_t col_p(int w) { return kAlias ? (128 + DV) * w : 384 + 64 * w; }
  // shared memory of a half: Q, K stages, V stages
  static constexpr int kOffK = kTileK, kOffV = kOffK + kStages * kTileK;
  static constexpr int kHalfBytes = kOffV + kStages * kTileV;
  static constexpr int kOffOut = kHalves * kHalfBytes;  // 64 columns of a half's output tile
  static constexpr int kOffBar = kOffOut + kHalves * kBlk;
  static constexpr int kSmemBytes = kOffBar + 1024 + 1024;  // + alignment slack
  static_assert(kSmemBytes <= 232448, "over the 227 KiB a CTA may use");
};

constexpr int kDenseStagesMax = 2;

struct HalfBars {
  uint64_t q_full[2];     // a unit's record (and its Q) is in place; by unit parity
  uint64_t unit_free[2];  // the MMA warp has read the record, the softmax warps are done with the unit
  uint64_t k_full[kDenseStagesMax], k_empty[kDenseStagesMax], v_full[kDenseStagesMax], v_empty[kDenseStagesMax];
  uint64_t s_full, s_free, p_half, p_full, o_done;  // a phase per tile
  uint64_t mma_final;
  uint64_t out_turn;  // the four softmax warps have come to a step of an output tile
  DenseUnit unit[2];  // n_i = 0: no more units
};
struct DenseBars {
  HalfBars half[2];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(DenseBars) <= 1024, "barrier block");

// A value that the compiler takes for a new one.
__device__ __forceinline__ uint32_t fresh(uint32_t x) {
  asm volatile("" : "+r"(x));
  return x;
}

// Unit x of an attn_cross call.
__device__ __forceinline__ DenseUnit cross_unit(const DenseParams& p, int x, int dv) {
  DenseUnit u;
  u.part = p.n_splits > 1 ? (int)(x * (dense_part_floats(kBM, dv) / 4)) : -1;
  const int split = x % p.n_splits;
  x /= p.n_splits;
  u.i0 = (x % p.n_tiles) * p.RPT;
  x /= p.n_tiles;
  const int hc = x % p.n_hchunks;
  x /= p.n_hchunks;
  u.head0 = x % p.Hkv * p.G + hc * p.GH;
  u.seq = u.batch_or_own = x / p.Hkv;
  u.n_i = min(p.RPT, p.n_i - u.i0);
  int n = p.kv_lens ? __ldg(p.kv_lens + u.seq) : p.S_kv;
  if (n < 0 || n > p.S_kv) {  // no such keys: zeros
    raise_error(p.err, kErrBounds);
    n = 0;
  }
  u.key0 = min(split * p.split_tiles * kBN, n);
  u.key1 = min((split + 1) * p.split_tiles * kBN, n);
  return u;
}

__device__ __forceinline__ int unit_tiles(const DenseUnit& u) { return (u.key1 - u.key0 + kBN - 1) / kBN; }

template <int DK, int DV, bool ARMS, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
    dense_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_q1,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_o, const DenseParams p) {
  using C = DenseCfg<DK, DV>;
  constexpr int kTileK = C::kTileK, kTileV = C::kTileV, kStages = C::kStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  DenseBars* bars = reinterpret_cast<DenseBars*>(smem + C::kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == kProducerWarp && lane == 0) {
    for (int w = 0; w < C::kHalves; ++w) {
      HalfBars& h = bars->half[w];
      for (int s = 0; s < 2; ++s) {
        mbar_init(&h.q_full[s], 1);
        mbar_init(&h.unit_free[s], 5);  // four softmax warps and the MMA warp
      }
      for (int s = 0; s < kStages; ++s) {
        mbar_init(&h.k_full[s], 1);
        mbar_init(&h.k_empty[s], 1);
        mbar_init(&h.v_full[s], 1);
        mbar_init(&h.v_empty[s], 1);
      }
      mbar_init(&h.s_full, 1);
      mbar_init(&h.s_free, 4);  // one arrival per softmax warp
      mbar_init(&h.p_half, 4);
      mbar_init(&h.p_full, 4);
      mbar_init(&h.o_done, 1);
      mbar_init(&h.mma_final, 1);
      mbar_init(&h.out_turn, 4);
    }
    bars->abort_flag = 0;
    fence_barrier_init();
    tc::prefetch_tmap(&tm_q);
    tc::prefetch_tmap(&tm_k);
    tc::prefetch_tmap(&tm_v);
  }
  if (warp == kMmaWarp0) {
    tc::tmem_alloc(&bars->tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  // the plan's units, the lengths and everything else may come from the kernel before
  grid_dep_wait();
  grid_dep_launch();  // the next launch may start setting up on the SMs this grid frees
  const int n_units = PAGED ? __ldcg(p.units_listed) : p.n_units;
  const int slots = (int)gridDim.x * C::kHalves;

  if (warp >= kProducerWarp) {
    regs_dec<kCtrlRegs>();  // the whole control warpgroup, right at the top of its branch
    const bool producer = warp == kProducerWarp || warp == kProducerVWarp;
    const int w = warp == kProducerWarp || warp == kMmaWarp0 ? 0 : 1;
    HalfBars& hb = bars->half[w];
    unsigned char* sm = smem + w * C::kHalfBytes;
    if (w < C::kHalves && producer) {
      // ================= TMA producer of half w =================
      int n = 0;        // units so far
      int t_all = 0;    // tiles so far
      int k_sent = 0, v_sent = 0;        // K and V tiles requested
      int last_q[2] = {-1, -1};          // the last unit of each parity, if a Q copy was requested for it
      bool alive = true;
      // The units of a plan differ in length: the first of each half is its slot, the others
      // come by ticket. A unit's ticket, record and first table entry are three round trips
      // to memory, so they are fetched step by step while the unit before sends its tiles.
      int next_x = (int)blockIdx.x + (int)gridDim.x * w, ahead = 1;  // steps done: 1 number, 2 record, 3 entry
      DenseUnit next_u = {};
      int next_e = 0;
      // paged: lane y < per brings block y of a tile and holds its table entry
      const int per = PAGED ? kBN / p.bs : 1;
      const int my_block = lane % per;
      // table entry of this lane's rows of tile j (num_blocks where it holds no key); checked
      // where it is used
      const auto entry = [&](const DenseUnit& u, int j) {
        const int t = (u.key0 + j * kBN) / p.bs + my_block;
        return t < p.mbps && t * p.bs < u.key1 ? __ldg(p.tables + (size_t)u.seq * p.mbps + t) : p.num_blocks;
      };
      const auto fetch_ahead = [&] {
        if (ahead == 0) {
          if (PAGED) {
            if (lane == 0) next_x = slots + atomicAdd(p.ticket, 1);
          } else {
            next_x += slots;
          }
          ahead = 1;
        } else if (ahead == 1) {
          if (PAGED) next_x = __shfl_sync(0xffffffffu, next_x, 0);
          next_u = DenseUnit{};
          if (next_x < n_units) {
            if (PAGED) {
              const int4 a = __ldcg(reinterpret_cast<const int4*>(p.units + next_x));
              const int4 c = __ldcg(reinterpret_cast<const int4*>(p.units + next_x) + 1);
              next_u = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
            } else {
              next_u = cross_unit(p, next_x, DV);
            }
          }
          ahead = 2;
        } else if (ahead == 2) {
          if (PAGED) next_e = entry(next_u, 0);
          // its Q and (contiguous) first K and V tiles on their way to L2: units that end
          // together would all wait for HBM at their next one's start
          if (next_u.n_i && next_u.key1 > next_u.key0) {
            const int own = PAGED && next_u.batch_or_own, seq = PAGED ? 0 : next_u.batch_or_own;
            if (lane < C::kCBK)
              tc::tma_prefetch_4d(own ? &tm_q1 : &tm_q, lane * 64, next_u.head0, next_u.i0, seq);
            if (!PAGED && lane < C::kCBK)
              tc::tma_prefetch_4d(&tm_k, lane * 64, next_u.key0, next_u.head0 / p.G, next_u.seq);
            if (!PAGED && lane < C::kCBV)
              tc::tma_prefetch_4d(&tm_v, lane * 64, next_u.key0, next_u.head0 / p.G, next_u.seq);
          }
          ahead = 3;
        }
      };
      for (; alive; ++n) {
        const int us = n & 1;
        while (ahead < 3) fetch_ahead();
        const DenseUnit u = next_u;
        int e = next_e;
        ahead = 0;
        const int tiles = u.n_i ? unit_tiles(u) : 0;
        const int kvh = u.head0 / p.G;
        // the record's slot is free once the unit before last has been taken; Q once the
        // last S of the previous unit is done
        bool ok = true;
        if (n >= 2) ok = warp_wait_tc(&hb.unit_free[us], ((n >> 1) - 1) & 1, bars, p.err);
        if (ok && t_all > 0)
          ok = warp_wait_tc(&hb.k_empty[(t_all - 1) % kStages], ((t_all - 1) / kStages) & 1, bars, p.err);
        if (!ok) break;
        const bool small = PAGED && u.batch_or_own;
        if (lane == 0) {
          hb.unit[us] = u;
          if (tiles > 0)
            mbar_arrive_expect_tx(&hb.q_full[us], (uint32_t)(C::kCBK * p.GH * (small ? 1 : p.RPT) * 128));
          else
            mbar_arrive(&hb.q_full[us]);
        }
        __syncwarp();
        // (a record without a copy completes a phase of its own: the copy two units before
        // it has long landed, and its phase can no longer be told from this one)
        last_q[us] = tiles > 0 ? n : -1;
        if (u.n_i == 0) break;  // the end
        if (tiles > 0 && lane < C::kCBK)
          tc::tma_load_4d(sm + lane * kBlk, small ? &tm_q1 : &tm_q, lane * 64, u.head0, u.i0,
                          PAGED ? 0 : u.batch_or_own, &hb.q_full[us]);
        for (int j = 0; j < tiles; ++j, ++t_all) {
          const int st = t_all % kStages;
          // a block that holds no key, or whose entry is out of range (flagged), loads from
          // past the end of the pool: the TMA engine fills it with zeros
          int blk = e;
          if (PAGED) {
            if ((blk < 0 || blk >= p.num_blocks) && u.key0 + j * kBN + my_block * p.bs < u.key1) {
              raise_error(p.err, kErrBounds);
              blk = p.num_blocks;
            }
            if (j + 1 < tiles) e = entry(u, j + 1);
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {  // the K tile, then the V tile
            uint64_t* full = kv ? &hb.v_full[st] : &hb.k_full[st];
            if (t_all >= kStages) {
              ok = warp_wait_tc(kv ? &hb.v_empty[st] : &hb.k_empty[st], (t_all / kStages - 1) & 1, bars, p.err);
              if (!ok) break;
            }
            // test hook: withheld, the first K tile is never requested (nothing is left in
            // flight), so the first wait on it runs into its bound and the half gives up
            if (p.debug_withhold && t_all == 0 && !kv) continue;
            const int ncb = kv ? C::kCBV : C::kCBK;
            unsigned char* dst = sm + (kv ? C::kOffV + st * kTileV : C::kOffK + st * kTileK);
            const CUtensorMap* tm = kv ? &tm_v : &tm_k;
            if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(ncb * kBlk));
            __syncwarp();
            if (!PAGED) {
              if (lane < ncb) tc::tma_load_4d(dst + lane * kBlk, tm, lane * 64, u.key0 + j * kBN, kvh, u.seq, full);
            } else if (lane < per) {
              tc::tma_load_4d(dst + lane * p.bs * 128 * ncb, tm, 0, 0, 0, (blk * p.Hkv + kvh) * (p.bs / 8), full);
            }
            __syncwarp();
            (kv ? v_sent : k_sent) = t_all + 1;
          }
          if (!ok) {
            alive = false;
            break;
          }
          fetch_ahead();  // one step a tile
        }
      }
      if (lane == 0) {
        // never exit with a load in flight (on the normal path all of these have landed)
        bool landed = true;
        for (int s = 0; s < 2; ++s)
          if (last_q[s] >= 0) landed &= mbar_wait(&hb.q_full[s], (last_q[s] >> 1) & 1);
        for (int s = 0; s < kStages; ++s) {
          const int k_last = (k_sent - 1 - s) / kStages, v_last = (v_sent - 1 - s) / kStages;  // phase of the last tile
          if (k_sent > s && !(p.debug_withhold && k_last == 0 && s == 0)) landed &= mbar_wait(&hb.k_full[s], k_last & 1);
          if (v_sent > s) landed &= mbar_wait(&hb.v_full[s], v_last & 1);
        }
        if (!landed) raise_error(p.err, kErrTimeout);
      }
    } else if (w < C::kHalves) {
      // ================= MMA warp of half w =================
      // The warp runs the loop converged, waits included, and an elected lane issues a product's
      // MMAs and its commits in one turn. (Waits and MMAs from lane 0 alone: attn_cross of 8 x 1024
      // rows 389 us; two MMAs an election 333, a whole product 306.)
      const uint32_t idS = tc::idesc_bf16_f32(kBM, kBN, false), idO = tc::idesc_bf16_f32(kBM, DV, true);
      // a K or V tile: squares of 8 rows x 64 columns, 1 KB each; those of the next columns and of
      // the next rows (paged: a block's columns next to one another, see make_pool_map)
      constexpr uint32_t kNextCols = PAGED ? 1024 : kBlk;
      constexpr uint32_t kNextRowsK = PAGED ? 1024 * C::kCBK : 1024, kNextRowsV = PAGED ? 1024 * C::kCBV : 1024;
      constexpr uint64_t kHiQ = tc::desc_sw128_hi(0, 1024), kHiK = tc::desc_sw128_hi(0, kNextRowsK);
      constexpr uint64_t kHiV = tc::desc_sw128_hi(C::kCBV > 1 ? kNextCols : 0, kNextRowsV);
      const uint32_t dS0 = tmem + C::col_s(w), dO = tmem + C::col_o(w), tP0 = tmem + C::col_p(w);
      // One place that issues S and one that issues PV, whatever tile or unit they are for: a
      // second copy of either, run once a unit, was fetched from L2 instruction by instruction
      // (2,000 cycles for eight MMAs). At d_v = 64 PV runs a tile behind S.
      constexpr int kLag = C::kAlias ? 0 : 1;
      bool ok = true;
      int t_all = 0;  // tiles before this unit
      for (int n = 0; ok; ++n) {
        const int us = n & 1;
        ok = warp_wait_tc(&hb.q_full[us], (n >> 1) & 1, bars, p.err);
        if (!ok) break;
        const int n_i = hb.unit[us].n_i, keys = hb.unit[us].key1 - hb.unit[us].key0;
        // keys at the start of a sequence's own, on the first one's block, that its window hides
        int hidden = 0;
        if (ARMS && p.window > 0 && hb.unit[us].batch_or_own)
          hidden = first_visible_key(__ldg(p.seq_lens + hb.unit[us].seq) - 1, p.window) - hb.unit[us].key0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&hb.unit_free[us]);
        if (n_i == 0) break;
        const int tiles = (keys + kBN - 1) / kBN;
#pragma unroll 1
        for (int i = 0; ok && i < tiles + kLag && tiles > 0; ++i) {
          if (i < tiles) {  // S = Q K^T of tile i
            const int t = t_all + i, st = t % kStages;
            // its columns are free once the previous tile's S is in registers (d_v = 64), or its
            // PV has read the P that lies over them (d_v = 128)
            if (t > 0) ok = warp_wait_tc(C::kAlias ? &hb.o_done : &hb.s_free, (t - 1) & 1, bars, p.err);
            ok = ok && warp_wait_tc(&hb.k_full[st], (t / kStages) & 1, bars, p.err);
            if (!ok) break;
            tc::fence_after_sync();
            // (the descriptors are built here from the buffers' addresses: as loop invariants
            // all of them were kept, in more registers than the control warps have)
            const uint64_t dQ = kHiQ | fresh(smem_u32(sm) >> 4);
            const uint64_t dK = kHiK | fresh(smem_u32(sm + C::kOffK + st * kTileK) >> 4);
            if (tc::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < DK / 16; ++kk) {
                const uint32_t at = (kk / 4) * kBlk + (kk % 4) * 32, at_k = (kk / 4) * kNextCols + (kk % 4) * 32;
                tc::mma_f16_ss(dS0, dQ + (at >> 4), dK + (at_k >> 4), idS, kk > 0);
              }
              tc::mma_commit(&hb.s_full);
              tc::mma_commit(&hb.k_empty[st]);  // the K stage is free once S is done
            }
            __syncwarp();
          }
          const int k = i - kLag;
          if (k >= 0) {  // O += P V of tile k
            const int t = t_all + k, st = t % kStages;
            ok = warp_wait_tc(&hb.v_full[st], (t / kStages) & 1, bars, p.err);
            if (!ok) break;
            // zeros for the rows behind the last key and for those before the first one that the row
            // sees (the swizzle moves chunks within a row only)
            const int valid = keys - k * kBN, skip = ARMS ? hidden - k * kBN : 0;
            if (valid < kBN || (ARMS && skip > 0)) {
              unsigned char* dst = sm + C::kOffV + st * kTileV + lane / 8 % C::kCBV * kNextCols + lane % 8 * 16;
#pragma unroll 1
              for (int row = (ARMS && skip > 0 ? 0 : valid) + lane / (8 * C::kCBV); row < kBN; row += 4 / C::kCBV)
                if (!ARMS || row >= valid || row < skip)
                  *reinterpret_cast<uint4*>(dst + row / 8 * kNextRowsV + row % 8 * 128) = make_uint4(0, 0, 0, 0);
              tc::fence_async_smem();
              __syncwarp();
            }
            ok = warp_wait_tc(C::kAlias ? &hb.p_half : &hb.p_full, t & 1, bars, p.err);
            if (!ok) break;
            tc::fence_after_sync();
            const uint64_t dV = kHiV | fresh(smem_u32(sm + C::kOffV + st * kTileV) >> 4);
            constexpr int kSteps = kBN / 16, kTurn = C::kAlias ? kSteps / 2 : kSteps;
#pragma unroll
            for (int k0 = 0; k0 < kSteps; k0 += kTurn) {
              if (k0 > 0) {
                ok = warp_wait_tc(&hb.p_full, t & 1, bars, p.err);
                if (!ok) break;
                tc::fence_after_sync();
              }
              if (tc::elect_one()) {
#pragma unroll
                for (int kk = k0; kk < k0 + kTurn; ++kk)
                  tc::mma_f16_ts(dO, tP0 + kk * 8, dV + kk * (kNextRowsV >> 3), idO, (k > 0 || kk > 0));
                if (k0 + kTurn == kSteps) {
                  tc::mma_commit(&hb.o_done);
                  tc::mma_commit(&hb.v_empty[st]);
                }
              }
              __syncwarp();
            }
          }
        }
        t_all += tiles;
      }
      // every MMA issued above has completed before TMEM is released
      if (tc::elect_one()) {  // (the lane that issued them)
        tc::mma_commit(&hb.mma_final);
        if (!mbar_wait(&hb.mma_final, 0)) raise_error(p.err, kErrTimeout);
      }
      __syncwarp();
    }
  } else {
    // ================= softmax warpgroups =================
    regs_inc<kSoftmaxRegs>();  // both softmax warpgroups, right at the top of their branch
    const int wg = warp >> 2;
    const int quarter = warp & 3;       // TMEM lanes this warp may access
    const int r = quarter * 32 + lane;  // row of the tile
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    HalfBars& hb = bars->half[wg];
    // With the arms the scores are moved into log2 units before the max, so the
    // exponent's multiplier is 1; plain: the raw q.k and the scale folded into it.
    const float qs = ARMS ? 1.f : p.qscale;
    const uint32_t tS = tmem + lane_addr + C::col_s(wg);
    const uint32_t tO = tmem + lane_addr + C::col_o(wg);
    const uint32_t tP = tmem + lane_addr + C::col_p(wg);
    const float2 qs2 = make_float2(qs, qs);
    bool alive = wg < C::kHalves;
    int t_all = 0;  // tiles so far: the phase of every barrier of the tile loop
    int turn = 0;   // steps of output tiles so far: the phase of out_turn
    for (int n = 0; alive; ++n) {
      const int us = n & 1;
      if (!warp_wait_tc(&hb.q_full[us], (n >> 1) & 1, bars, p.err)) break;
      // (the record stays until this warp lets go of it at the unit's end: what the tile
      // loop does not need is read again there, not held in registers)
      const volatile DenseUnit& u = hb.unit[us];
      if (u.n_i == 0) break;
      const int key0 = u.key0, tiles = (u.key1 - key0 + kBN - 1) / kBN;
      // keys of this row: [lo_key, lim)
      int lim, lo_key = 0, pos = 0;
      float th;  // the reference max moves when a score passes it by this much
      float alibi2 = 0.f;
      bool warp_live;
      {
        const int rows = u.n_i * p.GH;  // rows of the tile in use
        warp_live = quarter * 32 < rows;
        lim = u.key1;
        if (ARMS) {  // a row is a sequence of its own length; its position is its last key's
          pos = __ldg(p.seq_lens + u.i0 + min(r, rows - 1) / p.GH) - 1;
          if (u.batch_or_own) lo_key = first_visible_key(pos, p.window);
        }
        // a padding row beside live ones needs no mask and never moves its reference: whatever
        // it holds stays in its own row
        if (r >= rows) lim = INT_MAX;
        th = r < rows ? kRescaleLog2 / qs : INFINITY;
        if (ARMS && p.alibi) alibi2 = __ldg(p.alibi + u.head0 + min(r, rows - 1) % p.GH) * kLog2e;
      }
      float m_ref = -INFINITY;
      float l_run = 0.f;  // the row sum of p, against m_ref
      for (int k = 0; k < tiles; ++k, ++t_all) {
        const int j0 = key0 + k * kBN;  // the tile's first key
        if (!warp_wait_tc(&hb.s_full, t_all & 1, bars, p.err)) {
          alive = false;
          break;
        }
        if (!warp_live) {
          // padding rows: P may hold anything, only the barriers matter. At d_v = 64 S of the
          // next tile is issued before this tile's PV, so this warp has to be held back as the
          // others are by P, or its second arrival on p_full would stand in for another's first.
          if (!C::kAlias && t_all >= 1 && !warp_wait_tc(&hb.o_done, (t_all - 1) & 1, bars, p.err)) {
            alive = false;
            break;
          }
          if (lane == 0) {
            if (!C::kAlias) mbar_arrive(&hb.s_free);
            if (C::kAlias) mbar_arrive(&hb.p_half);
            mbar_arrive(&hb.p_full);
          }
          continue;
        }
        tc::fence_after_sync();
        // ---- the S row into registers; S's columns are then free
        uint32_t sv[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::tmem_ld_32x32b_x32(tS + c * 32, sv[c]);
        tc::tmem_ld_wait();
        if (!C::kAlias) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&hb.s_free);
        }
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
        if (__any_sync(0xffffffffu, j0 > lim - kBN || (ARMS && j0 < lo_key))) {
          const int end = lim - j0, begin = ARMS ? lo_key - j0 : 0;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c * 32 + e >= end || (ARMS && c * 32 + e < begin)) sv[c][e] = __float_as_uint(-INFINITY);
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
            if (!C::kAlias && !warp_wait_tc(&hb.o_done, (t_all - 1) & 1, bars, p.err)) {
              alive = false;
              break;
            }
            tc::fence_after_sync();
            uint32_t o[32];
#pragma unroll 1  // (rare, and the tile loop's code has to stay in the instruction cache)
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
              if (lane == 0) mbar_arrive(&hb.p_half);
            }
          }
        }
        l_run += ((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y)) + ((ls[2].x + ls[2].y) + (ls[3].x + ls[3].y));
        // ---- d_v = 64: P is free once the previous tile's PV has read it
        if (!C::kAlias) {
          if (t_all >= 1) {
            if (!warp_wait_tc(&hb.o_done, (t_all - 1) & 1, bars, p.err)) {
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
        if (lane == 0) mbar_arrive(&hb.p_full);
      }
      if (!alive) break;
      // ---- the unit's result: a partial one, or the output (every column of the row by its thread)
      if (tiles > 0) {
        if (!warp_wait_tc(&hb.o_done, (t_all - 1) & 1, bars, p.err)) break;
        tc::fence_after_sync();
      }
      // (a NaN among a row's scores makes its l NaN, and has to reach the output)
      const bool some = l_run != 0.f;
      const int at = u.part;
      if (PAGED || at >= 0) {
        if (warp_live) {
          const int rows = u.n_i * p.GH, R = PAGED && u.batch_or_own ? p.own_rows : kBM;
          float* part = p.partial + (size_t)at * 4;
#pragma unroll 1
          for (int cc = 0; cc < DV / 32; ++cc) {
            // (a unit without keys reads whatever O holds, and writes zeros)
            uint32_t o[32];
            tc::tmem_ld_32x32b_x32(tO + cc * 32, o);
            tc::tmem_ld_wait();
            if (r < rows) {
              // [column / 4][row][4]: the rows of a warp write contiguous bytes
#pragma unroll
              for (int t = 0; t < 8; ++t)
                *reinterpret_cast<uint4*>(part + ((size_t)(cc * 8 + t) * R + r) * 4) =
                    some ? make_uint4(o[4 * t], o[4 * t + 1], o[4 * t + 2], o[4 * t + 3]) : make_uint4(0, 0, 0, 0);
            }
            __syncwarp();  // the next columns are loaded by the whole warp
          }
          if (r < rows) {
            part[(size_t)R * DV + r] = m_ref * qs;
            part[(size_t)R * DV + R + r] = l_run;
          }
        }
      } else {
        // 64 columns at a time through shared memory (the output map's 128-byte swizzle) and
        // out by TMA: stored from the registers, each row's 16 bytes on a line of its own, a
        // tile held the load/store unit for 8,000 cycles, the other half's barriers with it
        const float inv = some ? 1.f / l_run : 0.f;
        unsigned char* so = smem + C::kOffOut + wg * kBlk;
        // Two steps for each 64 columns: the rows into the buffer once the last store has read it,
        // the store once all rows are there. The warps meet before each on an mbarrier, whose wait
        // has a bound: a warp that gave up does not come, and a hardware barrier would wait for it
        // without end. (8 x 1,024 rows: 279 us, with hardware barriers 276; with an mbarrier for each
        // step, so that only the storing warp waits before the store, 284: a second wait in the code.)
#pragma unroll 1
        for (int x = 0; x < 2 * C::kCBV; ++x, ++turn) {
          const int cb = x >> 1;
          if (!(x & 1) && (threadIdx.x & 127) == 0) tc::bulk_wait_group_read0();
          __syncwarp();
          if (lane == 0) mbar_arrive(&hb.out_turn);
          if (!warp_wait_tc(&hb.out_turn, turn & 1, bars, p.err)) {
            alive = false;
            break;
          }
          if (!(x & 1)) {
            if (warp_live) {
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                uint32_t o[32];
                tc::tmem_ld_32x32b_x32(tO + cb * 64 + hf * 32, o);
                tc::tmem_ld_wait();
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                  uint32_t w4[4];
#pragma unroll
                  for (int v = 0; v < 4; ++v) {
                    const float x0 = __uint_as_float(o[t * 8 + 2 * v]) * inv, x1 = __uint_as_float(o[t * 8 + 2 * v + 1]) * inv;
                    w4[v] = some ? pack_bf16(x0, x1) : 0u;
                  }
                  *reinterpret_cast<uint4*>(so + r * 128 + (((hf * 4 + t) ^ (r & 7)) * 16)) =
                      make_uint4(w4[0], w4[1], w4[2], w4[3]);
                }
              }
            }
            tc::fence_async_smem();
          } else if ((threadIdx.x & 127) == 0) {
            // rows past the end of the sequence fall outside the tensor and are not written
            tc::tma_store_4d(&tm_o, so, cb * 64, u.head0, u.i0, u.batch_or_own);
            tc::bulk_commit_group();
          }
        }
      }
      if (!alive) break;
      tc::fence_before_sync();  // O is read: the next unit's first PV may overwrite it
      __syncwarp();
      if (lane == 0) mbar_arrive(&hb.unit_free[us]);
    }
    if (!PAGED && (threadIdx.x & 127) == 0) tc::bulk_wait_group_read0();  // shared memory stays valid until then
  }

  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMmaWarp0) tc::tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------------------
// Joins the partial results of a row, in a fixed order (key ranges of the row's tile,
// then, for the shared-prefix step, the parts of the sequence's own keys):
//   M = max m_s (and the sink logit),  out = sum 2^(m_s - M) o_s / sum 2^(m_s - M) l_s
// A CTA takes rows (i, head) of one head chunk, next to one another in the parts, rows along
// the lanes, so that a warp's loads of a part fall on few lines: rows by d_v / 4 threads of four
// columns by `groups` shares of the parts (four parts at a time in turn, joined at the end in the
// shares' order; more than one where few rows would leave SMs without work: 9 sequences of 7 heads
// behind 10,600 keys 41.4 us, with eight shares 19.9). Latency bounds it:
// four parts are in flight a thread, M moves from round to round as the sums are rescaled. (A
// row per warp touched 32 lines a part; on an SM whose shared memory the kernel above had just
// used, with 28 KB left for L1, each round of loads took 3 us. The L1 is asked for in full at
// the launch.)
// SHARES: groups > 1 (an instantiation of its own: with the shared memory and the shares in one
// kernel 256 sequences behind four prefixes took 186 us instead of 173).
template <bool SHARES>
__global__ void __launch_bounds__(256) dense_combine_kernel(const DenseCombine p, int shares) {
  __shared__ float4 acc_s[SHARES ? 256 : 1];
  __shared__ float2 md_s[SHARES ? 256 : 1];
  const int groups = SHARES ? shares : 1;
  grid_dep_wait();
  const int dv = p.dv, rows_here = 1024 / dv / groups;  // powers of two, as dv is
  const int r = threadIdx.x & (rows_here - 1), c = threadIdx.x / rows_here % (dv / 4);
  const int share = SHARES ? threadIdx.x / (256 / groups) : 0;
  const int chunks = p.H / p.GH, per_chunk = (p.n_i * p.GH + rows_here - 1) / rows_here;
  int x = blockIdx.x;
  const int in_chunk = x % per_chunk * rows_here + r;
  const bool live = in_chunk < p.n_i * p.GH;
  if (!SHARES && !live) return;
  const int at_row = live ? in_chunk : p.n_i * p.GH - 1;  // i * GH + head within the chunk
  x /= per_chunk;
  const int chunk = x % chunks, b = x / chunks;  // chunk: (KV head, head chunk)
  const int i = at_row / p.GH, g = at_row - i * p.GH;  // shared prefix: i is the sequence
  // ---- the row's parts: n units of 128 rows, then n_own of own_rows
  const size_t unit_floats = dense_part_floats(kBM, dv), own_floats = dense_part_floats(p.own_rows, dv);
  int n = p.n_splits, n_own = 0, in_tile;
  const float *U, *R = nullptr;
  if (p.seq) {
    const int4 s0 = __ldcg(reinterpret_cast<const int4*>(p.seq + i));
    const int4 s1 = __ldcg(reinterpret_cast<const int4*>(p.seq + i) + 1);
    n = s0.x;
    U = p.partial + (size_t)(s0.y + chunk * s0.z) * unit_floats;
    in_tile = s0.w + g;
    n_own = s1.x;
    R = p.own_partial + (size_t)(s1.y + chunk * n_own) * own_floats;
  } else {
    const int tile = i / p.RPT;
    U = p.partial + (size_t)((b * chunks + chunk) * p.n_tiles + tile) * n * unit_floats;
    in_tile = at_row - tile * p.RPT * p.GH;
  }
  const int total = n + n_own;
  const float z2 = p.sinks ? __ldg(p.sinks + chunk * p.GH + g) * kLog2e : -INFINITY;
  float M = share == 0 ? z2 : -INFINITY, den = M != -INFINITY ? 1.f : 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int s0 = 4 * share; s0 < total; s0 += 4 * groups) {
    float4 o[4];
    float m[4], l[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int s = s0 + t;
      m[t] = -INFINITY;
      l[t] = 0.f;
      o[t] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < total) {
        const bool own = s >= n;
        const float* u = own ? R + (s - n) * own_floats : U + s * unit_floats;
        const int rows = own ? p.own_rows : kBM, at = own ? g : in_tile;
        m[t] = __ldcg(u + rows * dv + at);
        l[t] = __ldcg(u + rows * dv + rows + at);
        o[t] = __ldcg(reinterpret_cast<const float4*>(u) + (size_t)c * rows + at);
      }
    }
    const float Mn = fmaxf(fmaxf(fmaxf(M, m[0]), fmaxf(m[1], m[2])), m[3]);
    const float f = M == -INFINITY ? 0.f : ex2f(M - Mn);
    den = den == 0.f ? 0.f : den * f;
    acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
    M = Mn;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (l[t] == 0.f) continue;  // no visible key, whatever m and o hold (a NaN in l goes through)
      const float w = ex2f(m[t] - M);
      den = fmaf(w, l[t], den);
      acc.x = fmaf(w, o[t].x, acc.x);
      acc.y = fmaf(w, o[t].y, acc.y);
      acc.z = fmaf(w, o[t].z, acc.z);
      acc.w = fmaf(w, o[t].w, acc.w);
    }
  }
  if (SHARES) {
    md_s[threadIdx.x] = make_float2(M, den);
    acc_s[threadIdx.x] = acc;
    __syncthreads();
    if (share > 0) return;
    for (int k = 1; k < groups; ++k) {
      const float2 md = md_s[threadIdx.x + k * (256 / groups)];
      const float4 a = acc_s[threadIdx.x + k * (256 / groups)];
      if (md.y == 0.f) continue;
      const float Mn = fmaxf(M, md.x), f = den == 0.f ? 0.f : ex2f(M - Mn), w = ex2f(md.x - Mn);
      den = fmaf(w, md.y, den == 0.f ? 0.f : den * f);
      acc = make_float4(fmaf(w, a.x, acc.x * f), fmaf(w, a.y, acc.y * f), fmaf(w, a.z, acc.z * f),
                        fmaf(w, a.w, acc.w * f));
      M = Mn;
    }
  }
  if (!live) return;
  const float inv = den != 0.f ? 1.f / den : 0.f;
  const size_t row = ((size_t)b * p.n_i + i) * p.H + chunk * p.GH + g;
  *reinterpret_cast<uint2*>(p.out + row * dv + 4 * c) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

// A 4-D bf16 tensor of rows of d elements; box = 64 x b1 x b2 x 1, 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, int d, uint64_t d1, uint64_t d2, uint64_t d3, uint32_t box1,
              uint32_t box2) {
  const uint64_t dims[4] = {(uint64_t)d, d1, d2, d3};
  const uint64_t strides[3] = {(uint64_t)d * 2, (uint64_t)d * 2 * d1, (uint64_t)d * 2 * d1 * d2};
  const uint32_t box[4] = {64, box1, box2, 1};
  return make_tmap_bf16(m, base, dims, strides, box);
}

// The pool as [groups of 8 rows, d / 64, 8, 64]: a block of a KV head, all its columns, is one
// box, and in shared memory a group's squares of 8 x 64 lie next to one another. (A box of each 64
// columns, twice as many at 128 columns: 256 sequences behind four prefixes 193 us, so 184.)
bool make_pool_map(CUtensorMap* m, const void* base, int d, const DenseParams& p) {
  const uint64_t groups = (uint64_t)p.num_blocks * p.Hkv * (p.bs / 8);
  // (the block past the end, which stands for none, has to have a coordinate too)
  if (groups + (uint64_t)p.Hkv * (p.bs / 8) > INT_MAX) return false;
  const uint64_t dims[4] = {64, 8, (uint64_t)d / 64, groups};
  const uint64_t strides[3] = {(uint64_t)d * 2, 128, (uint64_t)d * 16};
  const uint32_t box[4] = {64, 8, (uint32_t)d / 64, (uint32_t)p.bs / 8};
  return make_tmap_bf16(m, base, dims, strides, box);
}

template <int DK, int DV, bool ARMS, bool PAGED>
cudaError_t launch_d(const CUtensorMap& tq, const CUtensorMap& tq1, const CUtensorMap& tk, const CUtensorMap& tv,
                     const CUtensorMap& to, const DenseParams& p, cudaStream_t st) {
  using C = DenseCfg<DK, DV>;
  int dev = 0;
  cudaGetDevice(&dev);
  static std::atomic<unsigned long long> attr_done{0};  // per device, per instantiation
  if (dev >= 64 || !(attr_done.load(std::memory_order_acquire) >> dev & 1ull)) {
    // The register hand-over inside the kernel assumes exactly kLaunchRegs per
    // thread at launch; a build with any other allocation is refused.
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, dense_tc_kernel<DK, DV, ARMS, PAGED>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kLaunchRegs) return cudaErrorNotSupported;
    e = cudaFuncSetAttribute(dense_tc_kernel<DK, DV, ARMS, PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done.fetch_or(1ull << dev, std::memory_order_release);
  }
  const int grid = p.units || p.n_units > kDenseSms ? kDenseSms : p.n_units;
  if (grid <= 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dense_tc_kernel<DK, DV, ARMS, PAGED>, tq, tq1, tk, tv, to, p);
}

// (the arms belong to the shared-prefix step, which is paged)
template <int DK, int DV>
cudaError_t launch_w(const CUtensorMap& tq, const CUtensorMap& tq1, const CUtensorMap& tk, const CUtensorMap& tv,
                     const CUtensorMap& to, const DenseParams& p, bool arms, cudaStream_t st) {
  if (!p.tables) return launch_d<DK, DV, false, false>(tq, tq1, tk, tv, to, p, st);
  return arms ? launch_d<DK, DV, true, true>(tq, tq1, tk, tv, to, p, st)
              : launch_d<DK, DV, false, true>(tq, tq1, tk, tv, to, p, st);
}

}  // namespace

bool dense_tc_supported(int bf16, int dk, int dv, int bs) {
  const bool widths = (dk == 64 && dv == 64) || (dk == 128 && dv == 128) || (dk == 192 && dv == 128);
  return bf16 == 1 && widths && (bs == 0 || (bs % 8 == 0 && kBN % bs == 0));
}

int dense_tc_slots(int dk) { return dk > 128 ? kDenseSms : 2 * kDenseSms; }

void dense_rows(int G, int* GH, int* RPT) {
  int g = G < kBM ? G : kBM;
  while (G % g) --g;
  *GH = g;
  *RPT = kBM / g;
}

// The queries [n_b, n_i, H, d_k] and outputs [n_b, n_i, H, d_v]; k, v contiguous
// [n_b, Hkv, S_kv, d] (p.tables NULL) or pools [num_blocks, Hkv, bs, d].
cudaError_t launch_dense_tc(const void* q, const void* k, const void* v, const DenseParams& p, int n_b, int dk, int dv,
                            bool arms, cudaStream_t st) {
  if (!dense_tc_supported(1, dk, dv, p.tables ? p.bs : 0) || !(p.qscale > 0.f)) return cudaErrorNotSupported;
  CUtensorMap tq, tq1, tk, tv, to;
  if (!make_map(&tq, q, dk, p.H, p.n_i, n_b, p.GH, p.RPT)) return cudaErrorInvalidValue;
  if (!make_map(&tq1, q, dk, p.H, p.n_i, n_b, p.GH, 1)) return cudaErrorInvalidValue;
  if (p.tables) {
    if (!make_pool_map(&tk, k, dk, p) || !make_pool_map(&tv, v, dv, p)) return cudaErrorInvalidValue;
  } else {
    if (!make_map(&tk, k, dk, p.S_kv, p.Hkv, n_b, kBN, 1)) return cudaErrorInvalidValue;
    if (!make_map(&tv, v, dv, p.S_kv, p.Hkv, n_b, kBN, 1)) return cudaErrorInvalidValue;
  }
  if (!make_map(&to, p.out, dv, p.H, p.n_i, n_b, p.GH, p.RPT)) return cudaErrorInvalidValue;
  if (dk == 64) return launch_w<64, 64>(tq, tq1, tk, tv, to, p, arms, st);
  if (dk == 128) return launch_w<128, 128>(tq, tq1, tk, tv, to, p, arms, st);
  return launch_w<192, 128>(tq, tq1, tk, tv, to, p, arms, st);
}

cudaError_t launch_dense_combine(const DenseCombine& p, cudaStream_t st) {
  int dev = 0;
  cudaGetDevice(&dev);
  static std::atomic<unsigned long long> attr_done{0};  // per device
  if (dev >= 64 || !(attr_done.load(std::memory_order_acquire) >> dev & 1ull)) {
    cudaError_t e = cudaFuncSetAttribute(dense_combine_kernel<false>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                         cudaSharedmemCarveoutMaxL1);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(dense_combine_kernel<true>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxL1);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_done.fetch_or(1ull << dev, std::memory_order_release);
  }
  int rows_here = 1024 / p.dv, groups = 1;
  const auto blocks_of = [&](int rows) {
    return (long long)p.n_b * (p.H / p.GH) * (((long long)p.n_i * p.GH + rows - 1) / rows);
  };
  while (rows_here > 1 && groups < 8 && blocks_of(rows_here / 2) <= 2 * kDenseSms) {
    rows_here /= 2;
    groups *= 2;
  }
  const long long blocks = blocks_of(rows_here);
  if (blocks <= 0) return cudaSuccess;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return groups > 1 ? cudaLaunchKernelEx(&cfg, dense_combine_kernel<true>, p, groups)
                    : cudaLaunchKernelEx(&cfg, dense_combine_kernel<false>, p, groups);
}

}  // namespace gqa
