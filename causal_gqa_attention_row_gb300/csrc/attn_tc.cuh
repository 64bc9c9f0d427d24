// attn_tc.cuh -- what the tcgen05 attention kernels (prefill_tc.cu, dense_tc.cu)
// share: the roles of the warps, the shared-memory and TMEM maps, bounded waits,
// the exponential and packing steps, register hand-over, and the loads of K and V
// tiles (contiguous, or gathered from a paged pool).
//
// The parameter struct P of the loads has the fields tables (NULL: contiguous),
// mbps, bs, num_blocks and err.
#pragma once

#include "tc_ptx.cuh"

namespace gqa {

constexpr int kBM = 128;         // query rows per tile
constexpr int kBN = 128;         // keys per tile
constexpr int kBlk = kBM * 128;  // 16 KiB: 128 rows of one 64-column block
constexpr int kWG = 2;           // softmax warpgroups
constexpr int kThreads = (kWG + 1) * 128;  // two softmax warpgroups + one control warpgroup
constexpr int kProducerWarp = 8, kMmaWarp0 = 9, kProducerVWarp = 11;
// Registers per thread: 168 at launch (384 threads); the control warpgroup
// gives up 96 per thread and the softmax warpgroups take 48 more:
// 128 * 72 + 256 * 216 = 384 * 168. (88 / 208 measured the same at d = 64 and
// d = 128 and up to 1% slower for the arms, the MLA widths and the paged chunks;
// 56 / 224 the same as 72 / 216.)
constexpr int kLaunchRegs = 168, kCtrlRegs = 72, kSoftmaxRegs = 216;
static_assert(128 * kCtrlRegs + kWG * 128 * kSoftmaxRegs <= kThreads * kLaunchRegs, "register split over budget");
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.0f;
constexpr int kTabEntries = 4096;  // paged: the CTA's block-table entries
constexpr int kMaxStages = 4;

// Sizes and maps of the kernel for head widths DK (Q, K) and DV (V, out).
template <int DK, int DV>
struct Cfg {
  static constexpr int kCBK = DK / 64, kCBV = DV / 64;  // 64-column blocks of a Q/K row, of a V/out row
  static constexpr int kTileK = kCBK * kBlk;            // one Q or K tile (128 rows)
  static constexpr int kTileV = kCBV * kBlk;            // one V or output tile
  static constexpr bool kAlias = DV > 64;               // P_w over the first 64 columns of S_w
  // rings: stage s only ever holds key tiles of warpgroup s % 2
  static constexpr int kStagesK = DK > 64 ? 2 : 4, kStagesV = DK > 64 ? 2 : 4;
  static_assert(kStagesK % kWG == 0 && kStagesV % kWG == 0 && kStagesK <= kMaxStages && kStagesV <= kMaxStages,
                "ring stages shared between warpgroups");
  static_assert(DV <= DK, "the output tile is staged over Q");
  // TMEM columns of S_w, O_w and P_w
  __host__ __device__ static constexpr uint32_t col_s(int w) { return kAlias ? (128 + DV) * w : 128 * w; }
  __host__ __device__ static constexpr uint32_t col_o(int w) { return kAlias ? (128 + DV) * w + 128 : 256 + 64 * w; }
  __host__ __device__ static constexpr uint32_t col_p(int w) { return kAlias ? (128 + DV) * w : 384 + 64 * w; }
  static_assert(col_o(kWG - 1) + DV <= kTmemCols && col_p(kWG - 1) + 64 <= kTmemCols, "TMEM map");
  // shared-memory map (from a 1024-byte aligned base)
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kTileK;                             // K ring
  static constexpr int kOffV = kOffK + kStagesK * kTileK;          // V ring
  static constexpr int kOffTab = kOffV + kStagesV * kTileV;        // paged: block-table entries
  static constexpr int kOffBar = kOffTab + kTabEntries * 4;
  static constexpr int kSmemBytes = kOffBar + 256 + 1024;          // + alignment slack
  // At the end, once every MMA is done: the output tile over Q, and warpgroup
  // w's row max and sum over K stage w (which only ever held warpgroup w's tiles).
  static constexpr int kOffOut = kOffQ;
  static constexpr int kOffML = kOffK;
  static_assert(kSmemBytes <= 232448, "over the 227 KiB a CTA may use");
};

struct Bars {
  uint64_t q_full, k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t s_full[kWG], s_free[kWG], p_full[kWG], mma_final[kWG];
  uint64_t p_half[kWG];  // P over S (d_v = 128): keys 0-63 of the warpgroup's P are in place
  uint64_t o_done[kWG];  // every PV of warpgroup w issued so far is done (a phase per PV)
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

template <typename BarsT>
__device__ __forceinline__ bool aborted(BarsT* bars) {
  return *reinterpret_cast<volatile int*>(&bars->abort_flag);
}

// Each probe of an mbarrier suspends a waiter for at most this long. A waiter
// resumes when the phase completes whatever the hint: 20, 200 and 2000 ns gave
// the same times (prefill and absorbed MLA decode, same box), so the hint only
// sets how often a long wait re-checks its time limit and the abort flag.
constexpr uint32_t kWaitHintNs = 20;

// Single-thread wait of the producer and MMA issuers (bounded). A phase that
// has completed is taken at once (the abort flag, a shared-memory load on the
// critical path, is only read when the wait has to wait).
template <typename BarsT>
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, BarsT* bars, unsigned* err) {
  if (mbar_test_parity_nb(bar, parity)) return true;
  if (aborted(bars)) return false;
  if (mbar_wait_hint(bar, parity, kWaitHintNs)) return true;
  *reinterpret_cast<volatile int*>(&bars->abort_flag) = 1;
  raise_error(err, kErrTimeout);
  return false;
}

// Whole-warp version: every lane agrees on the outcome.
template <typename BarsT>
__device__ __forceinline__ bool warp_wait_tc(uint64_t* bar, uint32_t parity, BarsT* bars, unsigned* err) {
  bool ok = mbar_test_parity_nb(bar, parity) || (!aborted(bars) && mbar_wait_hint(bar, parity, kWaitHintNs));
  ok = __all_sync(0xffffffffu, ok);
  if (!ok && (threadIdx.x & 31) == 0) {
    *reinterpret_cast<volatile int*>(&bars->abort_flag) = 1;
    raise_error(err, kErrTimeout);
  }
  return ok;
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// p = 2^(s*qs - mq) for two scores: fp32 exponentials (one special-function
// operation per score; the bf16x2 form costs the same per score and needs
// unpacking), added to the fp32 row sum `acc`, and returned rounded to the bf16
// pair that P stores.
__device__ __forceinline__ uint32_t exp2_pair(float s0, float s1, float2 qs2, float2 nmq2, float2& acc) {
  const float2 x = __ffma2_rn(make_float2(s0, s1), qs2, nmq2);
  const float2 e = make_float2(ex2f(x.x), ex2f(x.y));
  acc = __fadd2_rn(acc, e);
  return pack_bf16(e.x, e.y);
}

__device__ __forceinline__ float rcpf(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max(a, b, c) in one instruction.
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void named_bar_sync(int id, int nthreads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// The TMA loads of key tile j (128 rows of D) of KV head kvh, sequence b, into
// `dst`, completing a tile's bytes on `bar`: one box per 64-column block of the
// rows, at that block's 16 KiB slot. Contiguous: the tile's 128 rows in one box
// per block. Paged: one box per pool block and column block, addressed through
// the block table (the 128-byte swizzle is a function of the shared address, so
// the pool blocks land exactly where one box would put them). A pool block that
// holds no key below kv_hi, or whose table entry is out of range (flagged),
// loads from past the end of the pool: the TMA engine fills it with zeros.
template <typename P>
__device__ __forceinline__ int pool_block(const P& p, int t, int kv_hi, int e) {
  if (t >= p.mbps || t * p.bs >= kv_hi) return p.num_blocks;
  if (e >= 0 && e < p.num_blocks) return e;
  raise_error(p.err, kErrBounds);
  return p.num_blocks;
}

// One thread, the table read from global memory (the first tile, before the
// CTA's shared copy of the table exists).
template <int NCB, typename P>
__device__ __forceinline__ void load_kv_tile(const CUtensorMap* tm, unsigned char* dst, uint64_t* bar, int j, int kvh,
                                             int b, const P& p, int kv_hi) {
  mbar_arrive_expect_tx(bar, NCB * kBlk);
  if (!p.tables) {
#pragma unroll
    for (int cb = 0; cb < NCB; ++cb) tc::tma_load_4d(dst + cb * kBlk, tm, cb * 64, j * kBN, kvh, b, bar);
    return;
  }
  const int per = kBN / p.bs;
  for (int i = 0; i < per; ++i) {
    const int t = j * per + i;
    const int e = (t < p.mbps && t * p.bs < kv_hi) ? __ldg(p.tables + (size_t)b * p.mbps + t) : 0;
    const int blk = pool_block(p, t, kv_hi, e);
#pragma unroll
    for (int cb = 0; cb < NCB; ++cb)
      tc::tma_load_4d(dst + cb * kBlk + i * p.bs * 128, tm, cb * 64, 0, kvh, blk, bar);
  }
}

// The whole producer warp: lane 0 sets the expected bytes, then each lane issues
// one box (each TMA instruction holds its thread for a few hundred cycles, so
// the boxes of a tile go out side by side), the entries read from the CTA's
// shared copy of its table row.
template <int NCB, typename P>
__device__ __forceinline__ void load_kv_tile_warp(const CUtensorMap* tm, unsigned char* dst, uint64_t* bar, int j,
                                                  int kvh, int b, const P& p, int kv_hi, const int* tab, int lane) {
  if (lane == 0) mbar_arrive_expect_tx(bar, NCB * kBlk);
  __syncwarp();
  if (!p.tables) {
    if (lane < NCB) tc::tma_load_4d(dst + lane * kBlk, tm, lane * 64, j * kBN, kvh, b, bar);
  } else {
    const int per = kBN / p.bs;  // per * NCB boxes: one lane each while they fit the warp
    for (int x = lane; x < per * NCB; x += 32) {
      const int i = x % per, cb = x / per;
      const int t = j * per + i;
      const int e = (t < p.mbps && t * p.bs < kv_hi) ? tab[t] : 0;  // the shared copy covers every such t
      tc::tma_load_4d(dst + cb * kBlk + i * p.bs * 128, tm, cb * 64, 0, kvh, pool_block(p, t, kv_hi, e), bar);
    }
  }
  __syncwarp();
}

}  // namespace gqa
