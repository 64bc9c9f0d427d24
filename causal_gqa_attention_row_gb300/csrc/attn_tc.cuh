// attn_tc.cuh -- what the tcgen05 attention kernels (prefill_tc.cu, dense_tc.cu)
// share: the roles of the warps and their registers, bounded waits, and the exponential
// and packing steps.
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

}  // namespace gqa
