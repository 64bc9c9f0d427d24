// api.cu -- the extern "C" entry points of libgqa_attn.so (include/gqa_attn.h):
// host-side argument checks, work decomposition, and launches. No device
// memory is allocated here; the only device state is the error word below.
#include <atomic>
#include <cmath>
#include <climits>
#include <cstdint>

#include "gqa_attn.h"
#include "internal.h"

// Sticky device error word (bits gqa::kErrBounds, gqa::kErrTimeout), one per
// device that loads the library. Kernels in other translation units receive its
// device address as a parameter.
__device__ unsigned int g_gqa_error_word = 0;

namespace {

int g_withhold_first_tile = 0;

// Device address of the error word on the current device, looked up once per
// device; the cache is atomic, so concurrent first calls from several host
// threads are safe (each stores the same value).
unsigned* error_word() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  static std::atomic<void*> cache[64];
  void* p = cache[dev].load(std::memory_order_acquire);
  if (!p) {
    if (cudaGetSymbolAddress(&p, g_gqa_error_word) != cudaSuccess || p == nullptr) return nullptr;
    cache[dev].store(p, std::memory_order_release);
  }
  return static_cast<unsigned*>(p);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool heads_ok(int H, int Hkv) { return H > 0 && Hkv > 0 && H % Hkv == 0; }

bool width_ok(int d) { return d > 0 && d % 8 == 0 && d <= 256; }

int dtype_flag(gqa_dtype dt) { return dt == GQA_BF16 ? 1 : (dt == GQA_F32 ? 0 : -1); }

// Largest power of two <= cap that divides n.
int pow2_divisor(int n, int cap) {
  int g = 1;
  while (g * 2 <= cap && n % (g * 2) == 0) g *= 2;
  return g;
}

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

gqa_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return GQA_OK;
  if (e == cudaErrorNotSupported) return GQA_ERR_UNSUPPORTED;
  return GQA_ERR_CUDA;
}

gqa_status launch_rows(const gqa::RowsParams& p, int bf16, int dk, int dv, int drot, int nv, cudaStream_t st) {
  if (p.sched) {
    const cudaError_t ep = gqa::launch_plan_units(p, st);
    if (ep != cudaSuccess) return from_cuda(ep);
  }
  cudaError_t e = bf16 ? gqa::launch_attn_rows_bf16(p, dk, dv, drot, nv, st)
                       : gqa::launch_attn_rows_f32(p, dk, dv, drot, nv, st);
  if (e != cudaSuccess) return from_cuda(e);
  if (p.max_splits > 1) return from_cuda(gqa::launch_split_combine(p, dv, bf16, st));
  return GQA_OK;
}

// The arms of the attention row into the kernel parameters; true when any is on.
gqa_status apply_arms(gqa::RowsParams& p, const gqa_arms* arms, bool* active) {
  *active = false;
  if (!arms) return GQA_OK;
  if (!std::isfinite(arms->softcap)) return GQA_ERR_INVALID_ARG;
  if ((arms->sinks && reinterpret_cast<uintptr_t>(arms->sinks) % 4) ||
      (arms->alibi_slopes && reinterpret_cast<uintptr_t>(arms->alibi_slopes) % 4))
    return GQA_ERR_INVALID_ARG;
  p.window = arms->window > 0 ? arms->window : 0;
  p.softcap2 = arms->softcap > 0.f ? arms->softcap * gqa::kLog2e : 0.f;
  p.sinks = arms->sinks;
  p.alibi = arms->alibi_slopes;
  *active = p.window > 0 || p.softcap2 > 0.f || p.sinks || p.alibi;
  return GQA_OK;
}

}  // namespace

extern "C" {

size_t attn_decode_workspace_bytes(int B, int H, int d_v, int max_len_upper_bound) {
  if (B <= 0 || H <= 0 || d_v <= 0 || max_len_upper_bound <= gqa::kSplitRows) return 0;
  const size_t splits = (size_t)ceil_div(max_len_upper_bound, gqa::kSplitRows);
  const size_t units = (size_t)B * (size_t)H * splits;  // at least the (item, split) units of a call
  return gqa::plan_bytes(units) + units * (size_t)(d_v + 2) * sizeof(float);
}

static gqa_status decode_common(gqa::RowsParams& p, int bf16, int d_k, int d_v, int d_rot, void* workspace,
                                size_t workspace_bytes, cudaStream_t st) {
  const int nvmax = gqa::rows_max_nv(bf16, d_k, d_v, d_rot);
  if (nvmax == 0) return GQA_ERR_UNSUPPORTED;
  p.G = p.H / p.Hkv;
  p.GH = pow2_divisor(p.G, nvmax);
  p.QR = 1;
  p.n_hchunks = p.G / p.GH;
  p.n_rblocks = 1;
  p.seq_q = 1;
  p.split_rows = gqa::kSplitRows;
  p.max_splits = ceil_div(p.capacity, gqa::kSplitRows);
  const size_t need = attn_decode_workspace_bytes(p.B, p.H, d_v, p.capacity);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return GQA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GQA_ERR_INVALID_ARG;
  }
  if (need > 0) {
    const size_t units = (size_t)p.B * (size_t)p.H * (size_t)p.max_splits;
    p.sched = static_cast<int*>(workspace);
    p.units = reinterpret_cast<int2*>(static_cast<char*>(workspace) + gqa::kPlanHeaderBytes);
    p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + gqa::plan_bytes(units));
  }
  p.err = error_word();
  if (!p.err) return GQA_ERR_CUDA;
  p.debug_withhold = g_withhold_first_tile;
  return launch_rows(p, bf16, d_k, d_v, d_rot, p.GH, st);
}

gqa_status attn_decode_contig_ex(const void* q, const void* k_cache, const void* v_cache, const void* k_rot_shared,
                                 int d_rot, const int32_t* seq_lens, void* out, int B, int max_len, int H, int Hkv,
                                 int d_k, int d_v, float attention_scale, gqa_dtype dt, void* workspace,
                                 size_t workspace_bytes, const gqa_arms* arms, void* stream) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || B < 0 || max_len <= 0 || !heads_ok(H, Hkv) || !width_ok(d_k) || !width_ok(d_v))
    return GQA_ERR_INVALID_ARG;
  if (d_rot < 0 || d_rot >= d_k || d_rot % 8 || (k_rot_shared == nullptr) != (d_rot == 0))
    return GQA_ERR_INVALID_ARG;
  if (B == 0) return GQA_OK;
  if (!q || !k_cache || !v_cache || !seq_lens || !out) return GQA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      (k_rot_shared && !aligned16(k_rot_shared)))
    return GQA_ERR_INVALID_ARG;
  gqa::RowsParams p{};
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.k_rot = k_rot_shared;
  p.out = out;
  p.kv_len = seq_lens;
  p.paged = 0;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.max_len = max_len;
  p.capacity = max_len;
  p.qscale = attention_scale * 1.4426950408889634f;
  bool arms_on;
  const gqa_status sa = apply_arms(p, arms, &arms_on);
  if (sa != GQA_OK) return sa;
  return decode_common(p, bf16, d_k, d_v, d_rot, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

gqa_status attn_decode_paged_ex(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_tables,
                                const int32_t* seq_lens, void* out, int B, int max_blocks_per_seq, int num_blocks,
                                int block_size, int H, int Hkv, int d_k, int d_v, float attention_scale,
                                gqa_dtype dt, void* workspace, size_t workspace_bytes, const gqa_arms* arms,
                                void* stream) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || B < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || block_size <= 0 || !heads_ok(H, Hkv) ||
      !width_ok(d_k) || !width_ok(d_v))
    return GQA_ERR_INVALID_ARG;
  if ((long long)max_blocks_per_seq * block_size > INT_MAX / 2) return GQA_ERR_INVALID_ARG;
  if (B == 0) return GQA_OK;
  if (!q || !k_pool || !v_pool || !block_tables || !seq_lens || !out) return GQA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out)) return GQA_ERR_INVALID_ARG;
  gqa::RowsParams p{};
  p.q = q;
  p.k = k_pool;
  p.v = v_pool;
  p.out = out;
  p.kv_len = seq_lens;
  p.tables = block_tables;
  p.paged = 1;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.max_len = 0;
  p.capacity = max_blocks_per_seq * block_size;
  p.mbps = max_blocks_per_seq;
  p.bs = block_size;
  p.num_blocks = num_blocks;
  p.qscale = attention_scale * 1.4426950408889634f;
  bool arms_on;
  const gqa_status sa = apply_arms(p, arms, &arms_on);
  if (sa != GQA_OK) return sa;
  return decode_common(p, bf16, d_k, d_v, 0, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

// Prefill, contiguous or paged (p holds the pointers, shapes and arms): the
// tcgen05 kernel for the shapes it takes, else the SIMT kernel with one split
// per work item (every item covers its whole key range; no workspace).
static gqa_status prefill_common(gqa::RowsParams& p, int bf16, int d_k, int d_v, float attention_scale, bool arms_on,
                                 cudaStream_t st) {
  p.err = error_word();
  if (!p.err) return GQA_ERR_CUDA;
  const float qscale = attention_scale * 1.4426950408889634f;
  if (gqa::prefill_tc_supported(bf16, d_k, d_v, p.paged ? p.bs : 0, p.mbps) && attention_scale > 0.f) {
    const gqa::TcArms tc_arms{p.window, p.softcap2, p.sinks, p.alibi};
    return from_cuda(gqa::launch_prefill_tc(p.q, p.k, p.v, p.out, p.B, p.seq_q, p.capacity, p.offsets, p.H, p.Hkv,
                                            d_k, d_v, qscale, p.err, st, p.paged ? p.tables : nullptr, p.mbps, p.bs,
                                            p.num_blocks, arms_on ? &tc_arms : nullptr, g_withhold_first_tile));
  }
  const int nvmax = gqa::rows_max_nv(bf16, d_k, d_v, 0);
  if (nvmax == 0) return GQA_ERR_UNSUPPORTED;
  p.G = p.H / p.Hkv;
  p.GH = pow2_divisor(p.G, nvmax);
  p.QR = 1;
  while (p.GH * p.QR * 2 <= nvmax && p.QR < p.seq_q) p.QR *= 2;
  p.n_hchunks = p.G / p.GH;
  p.n_rblocks = ceil_div(p.seq_q, p.QR);
  p.split_rows = p.capacity;
  p.max_splits = 1;
  p.qscale = qscale;
  return launch_rows(p, bf16, d_k, d_v, 0, p.GH * p.QR, st);
}

gqa_status attn_prefill_causal_ex(const void* q, const void* k, const void* v, void* out, int B, int seq_q,
                                  int seq_kv_max, const int32_t* position_offset, int H, int Hkv, int d_k, int d_v,
                                  float attention_scale, gqa_dtype dt, const gqa_arms* arms, void* stream) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || B < 0 || seq_q < 0 || seq_kv_max <= 0 || seq_q > seq_kv_max || !heads_ok(H, Hkv) ||
      !width_ok(d_k) || !width_ok(d_v))
    return GQA_ERR_INVALID_ARG;
  if (B == 0 || seq_q == 0) return GQA_OK;
  if (!q || !k || !v || !out) return GQA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return GQA_ERR_INVALID_ARG;
  gqa::RowsParams p{};
  bool arms_on;
  const gqa_status sa = apply_arms(p, arms, &arms_on);
  if (sa != GQA_OK) return sa;
  p.q = q;
  p.k = k;
  p.v = v;
  p.out = out;
  p.offsets = position_offset;
  p.paged = 0;
  p.B = B;
  p.seq_q = seq_q;
  p.H = H;
  p.Hkv = Hkv;
  p.max_len = seq_kv_max;
  p.capacity = seq_kv_max;
  return prefill_common(p, bf16, d_k, d_v, attention_scale, arms_on, static_cast<cudaStream_t>(stream));
}

gqa_status attn_prefill_paged_ex(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_tables,
                                 const int32_t* position_offset, void* out, int B, int seq_q, int max_blocks_per_seq,
                                 int num_blocks, int block_size, int H, int Hkv, int d_k, int d_v,
                                 float attention_scale, gqa_dtype dt, const gqa_arms* arms, void* stream) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || B < 0 || seq_q < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || block_size <= 0 ||
      !heads_ok(H, Hkv) || !width_ok(d_k) || !width_ok(d_v))
    return GQA_ERR_INVALID_ARG;
  if ((long long)max_blocks_per_seq * block_size > INT_MAX / 2) return GQA_ERR_INVALID_ARG;
  if (seq_q > max_blocks_per_seq * block_size) return GQA_ERR_INVALID_ARG;
  if (B == 0 || seq_q == 0) return GQA_OK;
  if (!q || !k_pool || !v_pool || !block_tables || !out) return GQA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out)) return GQA_ERR_INVALID_ARG;
  gqa::RowsParams p{};
  bool arms_on;
  const gqa_status sa = apply_arms(p, arms, &arms_on);
  if (sa != GQA_OK) return sa;
  p.q = q;
  p.k = k_pool;
  p.v = v_pool;
  p.out = out;
  p.offsets = position_offset;
  p.tables = block_tables;
  p.paged = 1;
  p.B = B;
  p.seq_q = seq_q;
  p.H = H;
  p.Hkv = Hkv;
  p.max_len = 0;
  p.capacity = max_blocks_per_seq * block_size;
  p.mbps = max_blocks_per_seq;
  p.bs = block_size;
  p.num_blocks = num_blocks;
  return prefill_common(p, bf16, d_k, d_v, attention_scale, arms_on, static_cast<cudaStream_t>(stream));
}

// The plain calls: the _ex calls with no arms.
gqa_status attn_decode_contig(const void* q, const void* k_cache, const void* v_cache, const void* k_rot_shared,
                              int d_rot, const int32_t* seq_lens, void* out, int B, int max_len, int H, int Hkv,
                              int d_k, int d_v, float attention_scale, gqa_dtype dt, void* workspace,
                              size_t workspace_bytes, void* stream) {
  return attn_decode_contig_ex(q, k_cache, v_cache, k_rot_shared, d_rot, seq_lens, out, B, max_len, H, Hkv, d_k, d_v,
                               attention_scale, dt, workspace, workspace_bytes, nullptr, stream);
}

gqa_status attn_decode_paged(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_tables,
                             const int32_t* seq_lens, void* out, int B, int max_blocks_per_seq, int num_blocks,
                             int block_size, int H, int Hkv, int d_k, int d_v, float attention_scale, gqa_dtype dt,
                             void* workspace, size_t workspace_bytes, void* stream) {
  return attn_decode_paged_ex(q, k_pool, v_pool, block_tables, seq_lens, out, B, max_blocks_per_seq, num_blocks,
                              block_size, H, Hkv, d_k, d_v, attention_scale, dt, workspace, workspace_bytes, nullptr,
                              stream);
}

gqa_status attn_prefill_causal(const void* q, const void* k, const void* v, void* out, int B, int seq_q,
                               int seq_kv_max, const int32_t* position_offset, int H, int Hkv, int d_k, int d_v,
                               float attention_scale, gqa_dtype dt, void* stream) {
  return attn_prefill_causal_ex(q, k, v, out, B, seq_q, seq_kv_max, position_offset, H, Hkv, d_k, d_v,
                                attention_scale, dt, nullptr, stream);
}

gqa_status attn_prefill_paged(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_tables,
                              const int32_t* position_offset, void* out, int B, int seq_q, int max_blocks_per_seq,
                              int num_blocks, int block_size, int H, int Hkv, int d_k, int d_v, float attention_scale,
                              gqa_dtype dt, void* stream) {
  return attn_prefill_paged_ex(q, k_pool, v_pool, block_tables, position_offset, out, B, seq_q, max_blocks_per_seq,
                               num_blocks, block_size, H, Hkv, d_k, d_v, attention_scale, dt, nullptr, stream);
}

// ---- attn_decode_shared_prefix ------------------------------------------------
namespace {

// The workspace of a shared-prefix step: header, the plan's records, the list of units,
// the partial results of the prefixes' units and of the own parts.
struct SharedLayout {
  int GH, RPT, n_hchunks, own_rows, max_prefix_units;
  size_t groups, seq, units, partial, own, bytes;
};

SharedLayout shared_layout(int B, int H, int Hkv, int d_v, int capacity, int n_groups) {
  SharedLayout s{};
  const int G = H / Hkv;
  gqa::dense_rows(G, &s.GH, &s.RPT);
  s.n_hchunks = G / s.GH;
  s.own_rows = (s.GH + 3) / 4 * 4;  // a whole number of 16-byte steps per part
  // row tiles of the groups that count (two members or more), each with one key range or
  // more: as many more as two rounds of the SMs' two slots take, at most one per key tile
  const int counted = n_groups < B / 2 ? n_groups : B / 2;
  const long long heads = (long long)Hkv * s.n_hchunks;
  const long long tiles = counted ? heads * (B / s.RPT + counted) : 0;
  const long long each = tiles * ((capacity + 127) / 128), some = tiles ? tiles + 4 * gqa::kDenseSms : 0;
  const long long units = each < some ? each : some;
  s.max_prefix_units = units > INT_MAX ? INT_MAX : (int)units;
  const size_t parts = 2 * (size_t)B * (size_t)heads + gqa::kOwnExtra;
  size_t at = 256;  // [0]: units listed, [1]: ticket counter
  const auto take = [&](size_t n) {
    const size_t a = at;
    at += gqa::round_up256(n);
    return a;
  };
  s.groups = take((size_t)n_groups * sizeof(gqa::DenseGroup));
  s.seq = take((size_t)B * sizeof(gqa::SeqPlan));
  s.units = take(((size_t)s.max_prefix_units + parts) * sizeof(gqa::DenseUnit));
  s.partial = take((size_t)s.max_prefix_units * gqa::dense_part_floats(128, d_v) * 4);
  s.own = take(parts * gqa::dense_part_floats(s.own_rows, d_v) * 4);
  s.bytes = at;
  return s;
}

}  // namespace

size_t attn_decode_shared_prefix_workspace_bytes(int B, int H, int Hkv, int d_v, int max_len, int n_groups) {
  if (B <= 0 || !heads_ok(H, Hkv) || d_v <= 0 || max_len <= 0 || n_groups < 0) return 0;
  // (a shape that the tensor-core kernel does not take needs attn_decode_paged's workspace)
  const size_t shared = shared_layout(B, H, Hkv, d_v, max_len, n_groups).bytes;
  const size_t paged = attn_decode_workspace_bytes(B, H, d_v, max_len);
  return shared > paged ? shared : paged;
}

gqa_status attn_decode_shared_prefix(const void* q, const void* k_pool, const void* v_pool,
                                     const int32_t* block_tables, const int32_t* seq_lens,
                                     const int32_t* group_starts, const int32_t* shared_blocks, void* out, int B,
                                     int n_groups, int max_blocks_per_seq, int num_blocks, int block_size, int H,
                                     int Hkv, int d_k, int d_v, float attention_scale, gqa_dtype dt, void* workspace,
                                     size_t workspace_bytes, const gqa_arms* arms, void* stream) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || B < 0 || n_groups < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || block_size <= 0 ||
      !heads_ok(H, Hkv) || !width_ok(d_k) || !width_ok(d_v))
    return GQA_ERR_INVALID_ARG;
  if ((long long)max_blocks_per_seq * block_size > INT_MAX / 2) return GQA_ERR_INVALID_ARG;
  if (B == 0) return GQA_OK;
  if (!q || !k_pool || !v_pool || !block_tables || !seq_lens || !out) return GQA_ERR_INVALID_ARG;
  if (n_groups > 0 && (!group_starts || !shared_blocks)) return GQA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out)) return GQA_ERR_INVALID_ARG;
  const int capacity = max_blocks_per_seq * block_size;
  if (!workspace ||
      workspace_bytes < attn_decode_shared_prefix_workspace_bytes(B, H, Hkv, d_v, capacity, n_groups))
    return GQA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return GQA_ERR_INVALID_ARG;
  gqa::RowsParams arm{};  // (the arms in the kernels' units)
  bool arms_on;
  const gqa_status sa = apply_arms(arm, arms, &arms_on);
  if (sa != GQA_OK) return sa;
  if (!gqa::dense_tc_supported(bf16, d_k, d_v, block_size) || !(attention_scale > 0.f))
    return attn_decode_paged_ex(q, k_pool, v_pool, block_tables, seq_lens, out, B, max_blocks_per_seq, num_blocks,
                                block_size, H, Hkv, d_k, d_v, attention_scale, dt, workspace, workspace_bytes, arms,
                                stream);
  const SharedLayout s = shared_layout(B, H, Hkv, d_v, capacity, n_groups);
  // offsets of partial results are 32-bit counts of 16 bytes; units, and the key tiles of all
  // sequences (two ranges each), are counted in 32 bits
  if ((s.bytes - s.partial) / 16 > (size_t)INT_MAX || (s.own - s.partial) % 16 ||
      (long long)B * H > INT_MAX / 2 || (long long)B * (capacity / 128 + 2) > INT_MAX)
    return GQA_ERR_INVALID_ARG;
  unsigned* err = error_word();
  if (!err) return GQA_ERR_CUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);

  gqa::SharedPlan plan{};
  plan.seq_lens = seq_lens;
  plan.group_starts = group_starts;
  plan.shared_blocks = shared_blocks;
  plan.B = B;
  plan.Hkv = Hkv;
  plan.capacity = capacity;
  plan.bs = block_size;
  plan.mbps = max_blocks_per_seq;
  plan.window = arm.window;
  plan.dv = d_v;
  plan.n_groups = n_groups;
  plan.max_prefix_units = s.max_prefix_units;
  plan.slots = gqa::dense_tc_slots(d_k);
  plan.GH = s.GH;
  plan.RPT = s.RPT;
  plan.n_hchunks = s.n_hchunks;
  plan.own_rows = s.own_rows;
  plan.own_part_at = (int)((s.own - s.partial) / 16);
  plan.groups = reinterpret_cast<gqa::DenseGroup*>(ws + s.groups);
  plan.seq = reinterpret_cast<gqa::SeqPlan*>(ws + s.seq);
  plan.units = reinterpret_cast<gqa::DenseUnit*>(ws + s.units);
  plan.units_listed = reinterpret_cast<int*>(ws);
  plan.err = err;
  cudaError_t e = gqa::launch_shared_plan(plan, st);
  if (e != cudaSuccess) return from_cuda(e);

  gqa::DenseParams d{};
  d.H = H;
  d.Hkv = Hkv;
  d.G = H / Hkv;
  d.GH = s.GH;
  d.RPT = s.RPT;
  d.n_hchunks = s.n_hchunks;
  d.n_i = B;
  d.S_kv = capacity;
  d.units = plan.units;
  d.units_listed = plan.units_listed;
  d.ticket = plan.units_listed + 1;
  d.seq_lens = seq_lens;
  d.own_rows = s.own_rows;
  d.tables = block_tables;
  d.mbps = max_blocks_per_seq;
  d.bs = block_size;
  d.num_blocks = num_blocks;
  d.partial = reinterpret_cast<float*>(ws + s.partial);
  d.out = static_cast<__nv_bfloat16*>(out);
  d.qscale = attention_scale * gqa::kLog2e;
  d.err = err;
  d.debug_withhold = g_withhold_first_tile;
  d.window = arm.window;
  d.cap_out = arm.softcap2;
  d.cap_in = arm.softcap2 > 0.f ? d.qscale / arm.softcap2 : 0.f;
  d.alibi = arm.alibi;
  const bool score_arms = arm.window > 0 || arm.softcap2 > 0.f || arm.alibi;  // sinks join in the combine
  e = gqa::launch_dense_tc(q, k_pool, v_pool, d, 1, d_k, d_v, score_arms, st);
  if (e != cudaSuccess) return from_cuda(e);

  gqa::DenseCombine c{};
  c.n_b = 1;
  c.n_i = B;
  c.H = H;
  c.GH = s.GH;
  c.RPT = s.RPT;
  c.dv = d_v;
  c.partial = d.partial;
  c.seq = plan.seq;
  c.own_partial = reinterpret_cast<const float*>(ws + s.own);
  c.own_rows = s.own_rows;
  c.sinks = arm.sinks;
  c.out = d.out;
  return from_cuda(gqa::launch_dense_combine(c, st));
}

// ---- attn_cross ----------------------------------------------------------------
namespace {

// How a cross attention runs: on the tensor cores (row tiles and key ranges), or on
// the SIMT kernel (splits of one query row's keys), with the workspace of each.
struct CrossPlan {
  bool tc;
  int GH, RPT, n_hchunks, n_tiles, n_splits, split_tiles;
  long long units;
  int simt_GH, simt_QR, split_rows, max_splits;
  size_t bytes;
  size_t bound;  // of the bytes of every smaller B and every shorter L: fewer items make more splits
};

// Rows of a KV head (query rows times heads of its group) from which the tensor cores
// are taken: the SIMT kernel reads the keys once for up to NV rows (a power of two), the
// tensor-core kernel once for 128. Measured (SIMT, tensor cores) at 64 sequences of up to 1500
// keys: one row of 16 KV heads of 64 39.9 and 48.8 us, of 128 64 and 84 us; two rows of 64 58 and
// 55, of 8 heads of 128 60 and 51; four rows of 64 85 and 53; at 4 sequences of up to 4000 keys,
// 8 heads of 64, one row 17.0 and 15.4 us, two 70 and 15.4 (the SIMT kernel splits single rows
// only).
constexpr int kCrossTcRows = 2;

bool cross_plan(int B, int S, int L, int H, int Hkv, int d_k, int d_v, int bf16, bool scale_ok, CrossPlan* c) {
  *c = CrossPlan{};
  const int G = H / Hkv;
  c->tc = scale_ok && gqa::dense_tc_supported(bf16, d_k, d_v) && (long long)S * G >= kCrossTcRows;
  if (c->tc) {
    gqa::dense_rows(G, &c->GH, &c->RPT);
    if (c->RPT > S) c->RPT = S;
    c->n_hchunks = G / c->GH;
    c->n_tiles = ceil_div(S, c->RPT);
    const long long tiles = (long long)B * Hkv * c->n_hchunks * c->n_tiles;
    const int nt = ceil_div(L, 128), slots = gqa::dense_tc_slots(d_k);
    // key ranges of st tiles: the fewest rounds * (st + a unit's own cost); one range
    // writes the result itself, more leave partial results to join (a further cost)
    long long best = -1;
    for (int ns = 1; ns <= nt && (ns == 1 || tiles * ns <= 4 * slots); ++ns) {
      const int st = ceil_div(nt, ns), n = ceil_div(nt, st);
      const long long rounds = (tiles * n + slots - 1) / slots;
      const long long cost = rounds * (st + gqa::kDenseUnitTiles) + (n > 1 ? 2 : 0);
      if (best < 0 || cost < best) {
        best = cost;
        c->n_splits = n;
        c->split_tiles = st;
      }
    }
    c->units = tiles * c->n_splits;
    const size_t part = gqa::dense_part_floats(128, d_v) * 4;
    c->bytes = c->n_splits > 1 ? (size_t)c->units * part : 0;
    // more ranges than one leave at most 4 * slots units (the loop's condition, from one sequence on)
    if (nt > 1 && tiles / B * 2 <= 4 * slots) c->bound = (size_t)(tiles * nt < 4 * slots ? tiles * nt : 4 * slots) * part;
    return true;
  }
  const int nvmax = gqa::rows_max_nv(bf16, d_k, d_v, 0);
  if (nvmax == 0) return false;
  c->simt_GH = pow2_divisor(G, nvmax);
  c->simt_QR = 1;
  while (c->simt_GH * c->simt_QR * 2 <= nvmax && c->simt_QR < S) c->simt_QR *= 2;
  c->split_rows = L;
  c->max_splits = 1;
  if (S == 1) {
    // splits of 2048 keys, halved to 512 until there are several units for each of the
    // kernel's 456 resident CTAs, and to 256 while SMs would go without work. Measured: 1024
    // items of up to 1500 keys 51.6 us whole, 42.2 / 40.9 / 43.2 us in splits of 1024 / 512 /
    // 256; 16 items of 4000 keys 40.2, 24.9, 17.4, 15.1 us.
    const long long items = (long long)B * Hkv * (G / c->simt_GH);
    const auto few = [](int r) { return r > 512 ? 3 * 1024 : r > gqa::kLeastSplitRows ? 2 * gqa::kDenseSms : 0; };
    const auto bytes_of = [&](size_t units) { return gqa::plan_bytes(units) + units * (size_t)(d_v + 2) * 4; };
    int r = gqa::kSplitRows;
    while (items * ceil_div(L, r) < few(r)) r /= 2;
    c->max_splits = ceil_div(L, r);
    if (c->max_splits > 1) {
      c->split_rows = r;
      c->bytes = bytes_of((size_t)B * (size_t)H * (size_t)c->max_splits);
    }
    // splits of r rows are taken where those of 2r were fewer than few(2r), so they are fewer than twice that
    for (r = gqa::kSplitRows; r >= gqa::kLeastSplitRows; r /= 2) {
      const long long all = items * ceil_div(L, r), most = r == gqa::kSplitRows ? all : 2 * few(2 * r);
      const size_t n = bytes_of((size_t)(all < most ? all : most) * c->simt_GH);
      if (ceil_div(L, r) > 1 && n > c->bound) c->bound = n;
    }
  }
  return true;
}

}  // namespace

size_t attn_cross_workspace_bytes(int B, int seq_q, int seq_kv_max, int H, int Hkv, int d_k, int d_v, gqa_dtype dt) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || B <= 0 || seq_q <= 0 || seq_kv_max <= 0 || !heads_ok(H, Hkv) || !width_ok(d_k) || !width_ok(d_v))
    return 0;
  size_t n = 0;
  for (int scale_ok = 0; scale_ok < 2; ++scale_ok) {  // (a scale that is not positive takes the SIMT kernel)
    CrossPlan c;
    if (cross_plan(B, seq_q, seq_kv_max, H, Hkv, d_k, d_v, bf16, scale_ok, &c) && c.bound > n) n = c.bound;
  }
  return n;
}

gqa_status attn_cross(const void* q, const void* k, const void* v, const int32_t* kv_lens, void* out, int B, int seq_q,
                      int seq_kv_max, int H, int Hkv, int d_k, int d_v, float attention_scale, gqa_dtype dt,
                      void* workspace, size_t workspace_bytes, void* stream) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || B < 0 || seq_q < 0 || seq_kv_max <= 0 || seq_kv_max > INT_MAX / 2 || !heads_ok(H, Hkv) ||
      !width_ok(d_k) || !width_ok(d_v) || (long long)B * seq_q > INT_MAX || !std::isfinite(attention_scale))
    return GQA_ERR_INVALID_ARG;
  if (B == 0 || seq_q == 0) return GQA_OK;
  if (!q || !k || !v || !out) return GQA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return GQA_ERR_INVALID_ARG;
  CrossPlan c;
  if (!cross_plan(B, seq_q, seq_kv_max, H, Hkv, d_k, d_v, bf16, attention_scale > 0.f, &c)) return GQA_ERR_UNSUPPORTED;
  if (c.bytes > 0) {
    if (!workspace || workspace_bytes < c.bytes) return GQA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GQA_ERR_INVALID_ARG;
  }
  unsigned* err = error_word();
  if (!err) return GQA_ERR_CUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const float qscale = attention_scale * gqa::kLog2e;
  if (c.tc) {
    gqa::DenseParams d{};
    d.H = H;
    d.Hkv = Hkv;
    d.G = H / Hkv;
    d.GH = c.GH;
    d.RPT = c.RPT;
    d.n_hchunks = c.n_hchunks;
    d.n_i = seq_q;
    d.S_kv = seq_kv_max;
    d.kv_lens = kv_lens;
    d.n_units = (int)c.units;
    d.n_tiles = c.n_tiles;
    d.n_splits = c.n_splits;
    d.split_tiles = c.split_tiles;
    d.partial = c.n_splits > 1 ? static_cast<float*>(workspace) : nullptr;
    d.out = static_cast<__nv_bfloat16*>(out);
    d.qscale = qscale;
    d.err = err;
    d.debug_withhold = g_withhold_first_tile;
    if (c.units > INT_MAX / 2 || c.bytes / 16 > (size_t)INT_MAX) return GQA_ERR_INVALID_ARG;
    const cudaError_t e = gqa::launch_dense_tc(q, k, v, d, B, d_k, d_v, false, st);
    if (e != cudaSuccess || c.n_splits == 1) return from_cuda(e);
    gqa::DenseCombine m{};
    m.n_b = B;
    m.n_i = seq_q;
    m.H = H;
    m.GH = c.GH;
    m.RPT = c.RPT;
    m.dv = d_v;
    m.n_tiles = c.n_tiles;
    m.n_splits = c.n_splits;
    m.partial = d.partial;
    m.out = d.out;
    return from_cuda(gqa::launch_dense_combine(m, st));
  }
  gqa::RowsParams p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.out = out;
  p.kv_len = kv_lens;
  p.full = 1;
  p.B = B;
  p.seq_q = seq_q;
  p.H = H;
  p.Hkv = Hkv;
  p.max_len = seq_kv_max;
  p.capacity = seq_kv_max;
  p.G = H / Hkv;
  p.GH = c.simt_GH;
  p.QR = c.simt_QR;
  p.n_hchunks = p.G / p.GH;
  p.n_rblocks = ceil_div(seq_q, p.QR);
  p.split_rows = c.split_rows;
  p.max_splits = c.max_splits;
  p.qscale = qscale;
  p.err = err;
  p.debug_withhold = g_withhold_first_tile;
  if (c.max_splits > 1) {
    const size_t units = (size_t)B * (size_t)H * (size_t)c.max_splits;
    p.sched = static_cast<int*>(workspace);
    p.units = reinterpret_cast<int2*>(static_cast<char*>(workspace) + gqa::kPlanHeaderBytes);
    p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + gqa::plan_bytes(units));
  }
  return launch_rows(p, bf16, d_k, d_v, 0, p.GH * p.QR, st);
}

gqa_status kv_append_paged(void* q, const void* k_new, const void* v_new, void* k_pool, void* v_pool,
                           const int32_t* block_tables, const int32_t* seq_lens_in, int32_t* seq_lens_out, int B,
                           int max_blocks_per_seq, int num_blocks, int block_size, int H, int Hkv, int d_k, int d_v,
                           double rope_theta, int rot_offset, int rot_dim, gqa_dtype dt, void* stream) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || B < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || block_size <= 0 || !heads_ok(H, Hkv) ||
      d_k <= 0 || d_v <= 0 || d_k % 2)
    return GQA_ERR_INVALID_ARG;
  if (rope_theta > 0.0 && (rot_dim <= 0 || rot_dim % 2 || rot_offset < 0 || rot_offset + rot_dim > d_k))
    return GQA_ERR_INVALID_ARG;
  if ((long long)max_blocks_per_seq * block_size > INT_MAX / 2) return GQA_ERR_INVALID_ARG;
  if (B == 0) return GQA_OK;
  if (!q || !k_new || !v_new || !k_pool || !v_pool || !block_tables || !seq_lens_in || !seq_lens_out)
    return GQA_ERR_INVALID_ARG;
  unsigned* err = error_word();
  if (!err) return GQA_ERR_CUDA;
  return from_cuda(gqa::launch_append(q, k_new, v_new, k_pool, v_pool, block_tables, seq_lens_in, seq_lens_out, B,
                                      max_blocks_per_seq, num_blocks, block_size, H, Hkv, d_k, d_v, rope_theta,
                                      rot_offset, rope_theta > 0.0 ? rot_dim : 0, bf16, err,
                                      static_cast<cudaStream_t>(stream)));
}

gqa_status attn_rope_interleaved(void* x, const int32_t* positions, int B, int T, int heads, int d, int heads_outer,
                                 int rot_offset, int rot_dim, double theta, gqa_dtype dt, void* stream) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || B < 0 || T < 0 || heads <= 0 || d <= 0 || d % 2 || rot_dim <= 0 || rot_dim % 2 ||
      rot_offset < 0 || rot_offset % 2 || rot_offset + rot_dim > d || !(theta > 0.0) ||
      (heads_outer != 0 && heads_outer != 1))
    return GQA_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return GQA_OK;
  if (!x || !positions || !aligned16(x)) return GQA_ERR_INVALID_ARG;
  return from_cuda(gqa::launch_rope(x, positions, B, T, heads, d, heads_outer, rot_offset, rot_dim, theta, bf16,
                                    static_cast<cudaStream_t>(stream)));
}

gqa_status attn_rope_interleaved_qk(void* q, void* k, const int32_t* positions, int B, int T, int heads_q, int heads_k,
                                    int d, int q_heads_outer, int k_heads_outer, int rot_offset, int rot_dim,
                                    double theta, gqa_dtype dt, void* stream) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || B < 0 || T < 0 || heads_q <= 0 || heads_k <= 0 || d <= 0 || d % 2 || rot_dim <= 0 ||
      rot_dim % 2 || rot_offset < 0 || rot_offset % 2 || rot_offset + rot_dim > d || !(theta > 0.0) ||
      (q_heads_outer != 0 && q_heads_outer != 1) || (k_heads_outer != 0 && k_heads_outer != 1))
    return GQA_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return GQA_OK;
  if (!q || !k || !positions || !aligned16(q) || !aligned16(k)) return GQA_ERR_INVALID_ARG;
  return from_cuda(gqa::launch_rope(q, positions, B, T, heads_q, d, q_heads_outer, rot_offset, rot_dim, theta, bf16,
                                    static_cast<cudaStream_t>(stream), k, heads_k, k_heads_outer));
}

gqa_status gqa_rope_frequencies(float* freqs_host, float* magnitude, int rot_dim, double theta,
                                const gqa_rope_scaling* scaling) {
  if (!freqs_host || !magnitude || rot_dim <= 0 || rot_dim % 2 || rot_dim > 256 || !(theta > 0.0) ||
      !std::isfinite(theta))
    return GQA_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586;
  const int kind = scaling ? scaling->kind : GQA_ROPE_SCALING_NONE;
  if (kind < GQA_ROPE_SCALING_NONE || kind > GQA_ROPE_SCALING_INDEX) return GQA_ERR_INVALID_ARG;
  if (kind != GQA_ROPE_SCALING_NONE && !(scaling->factor > 0.0 && std::isfinite(scaling->factor)))
    return GQA_ERR_INVALID_ARG;
  const bool blend = kind == GQA_ROPE_SCALING_TURNS || kind == GQA_ROPE_SCALING_INDEX;
  if (blend && !(scaling->original_max > 0.0 && std::isfinite(scaling->original_max) && scaling->low > 0.0 &&
                 scaling->high > scaling->low && std::isfinite(scaling->high)))
    return GQA_ERR_INVALID_ARG;
  if (scaling && !(scaling->magnitude >= 0.0 && std::isfinite(scaling->magnitude))) return GQA_ERR_INVALID_ARG;
  double first = 0.0, last = 0.0;
  if (kind == GQA_ROPE_SCALING_INDEX) {
    if (!(theta > 1.0)) return GQA_ERR_INVALID_ARG;  // the index of a pair needs falling frequencies
    const auto index = [&](double turns) {
      return rot_dim * std::log(scaling->original_max / (two_pi * turns)) / (2.0 * std::log(theta));
    };
    first = std::fmax(0.0, std::floor(index(scaling->high)));
    last = std::fmin(rot_dim - 1.0, std::ceil(index(scaling->low)));
  }
  for (int t = 0; t < rot_dim / 2; ++t) {
    double w = std::pow(theta, -2.0 * t / rot_dim);
    if (scaling && scaling->divisors) {
      if (!(scaling->divisors[t] > 0.0)) return GQA_ERR_INVALID_ARG;
      w /= scaling->divisors[t];
    }
    double keep = 1.0;
    if (kind == GQA_ROPE_SCALING_LINEAR) keep = 0.0;
    if (kind == GQA_ROPE_SCALING_TURNS)
      keep = (scaling->original_max * w / two_pi - scaling->low) / (scaling->high - scaling->low);
    if (kind == GQA_ROPE_SCALING_INDEX) keep = 1.0 - (t - first) / std::fmax(last - first, 0.001);
    keep = std::fmin(1.0, std::fmax(0.0, keep));
    if (kind != GQA_ROPE_SCALING_NONE) w = keep * w + (1.0 - keep) * w / scaling->factor;
    const float hi = (float)w;
    freqs_host[2 * t] = hi;
    freqs_host[2 * t + 1] = (float)(w - (double)hi);
  }
  double m = scaling ? scaling->magnitude : 1.0;
  if (m == 0.0) m = kind == GQA_ROPE_SCALING_INDEX ? 0.1 * std::log(scaling->factor) + 1.0 : 1.0;
  *magnitude = (float)m;
  return GQA_OK;
}

// A call's view of a tensor of B sequences (0: no batch axis), T tokens, heads heads:
// an axis of one element has no stride.
static gqa::HeadsView heads_view(const gqa_heads* x, int B, int T, int heads) {
  if (!x) return {};
  return {x->data, B > 1 ? x->batch_stride : 0, T > 1 ? x->token_stride : 0, heads > 1 ? x->head_stride : 0};
}

static bool heads_view_ok(const gqa::HeadsView& x, int bf16) {
  const int v = bf16 ? 8 : 4;  // elements of 16 bytes
  return x.data && aligned16(x.data) && x.batch_stride % v == 0 && x.token_stride % v == 0 && x.head_stride % v == 0;
}

// An output that starts where its input does has to be the same view.
static bool in_place_ok(const gqa::HeadsView& x, const gqa::HeadsView& y) {
  return x.data != y.data ||
         (x.batch_stride == y.batch_stride && x.token_stride == y.token_stride && x.head_stride == y.head_stride);
}

// The checks that attn_qk_norm_rope and kv_append_paged_rows share, and the norm
// and the rotation into the kernel's parameters.
static gqa_status qk_norm_and_rope(gqa::QkParams& p, const void* q_weight, const void* k_weight, float eps,
                                   const gqa_rope* rope, int d) {
  if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight))) return GQA_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return GQA_ERR_INVALID_ARG;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.eps = eps;
  p.d = d;
  if (!rope) return GQA_OK;
  if ((rope->layout != GQA_ROPE_ADJACENT && rope->layout != GQA_ROPE_HALF) || rope->rot_dim <= 0 ||
      rope->rot_dim % 2 || rope->rot_dim > 256 || rope->rot_offset < 0 || rope->rot_offset > d - rope->rot_dim ||
      !rope->freqs || reinterpret_cast<uintptr_t>(rope->freqs) % 8 || !std::isfinite(rope->magnitude))
    return GQA_ERR_INVALID_ARG;
  p.layout = rope->layout;
  p.rot_offset = rope->rot_offset;
  p.rot_dim = rope->rot_dim;
  p.magnitude = rope->magnitude;
  p.freqs = rope->freqs;
  return GQA_OK;
}

gqa_status attn_qk_norm_rope(const gqa_heads* q, const gqa_heads* k, const gqa_heads* q_out, const gqa_heads* k_out,
                             const void* q_weight, const void* k_weight, float eps, const int32_t* positions, int B,
                             int T, int H, int Hkv, int d, const gqa_rope* rope, gqa_dtype dt, void* stream) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || B < 0 || T < 0 || H < 0 || Hkv < 0 || !width_ok(d) || (long long)B * T > INT_MAX ||
      (long long)H + Hkv > INT_MAX / 2)
    return GQA_ERR_INVALID_ARG;
  if ((q == nullptr) != (H == 0) || (k == nullptr) != (Hkv == 0) || (q == nullptr) != (q_out == nullptr) ||
      (k == nullptr) != (k_out == nullptr))
    return GQA_ERR_INVALID_ARG;
  gqa::QkParams p{};
  const gqa_status s = qk_norm_and_rope(p, q_weight, k_weight, eps, rope, d);
  if (s != GQA_OK) return s;
  if (B == 0 || T == 0 || H + Hkv == 0) return GQA_OK;
  p.q = heads_view(q, B, T, H);
  p.q_out = heads_view(q_out, B, T, H);
  p.k = heads_view(k, B, T, Hkv);
  p.k_out = heads_view(k_out, B, T, Hkv);
  if ((q && (!heads_view_ok(p.q, bf16) || !heads_view_ok(p.q_out, bf16) || !in_place_ok(p.q, p.q_out))) ||
      (k && (!heads_view_ok(p.k, bf16) || !heads_view_ok(p.k_out, bf16) || !in_place_ok(p.k, p.k_out))))
    return GQA_ERR_INVALID_ARG;
  if (rope && !positions) return GQA_ERR_INVALID_ARG;
  p.positions = positions;
  p.N = B * T;
  p.T = T;
  p.B = B;
  p.H = H;
  p.Hk = p.Hkv = Hkv;
  p.run_rows = 1;
  return from_cuda(gqa::launch_qk_rows(p, bf16, 0, static_cast<cudaStream_t>(stream)));
}

gqa_status kv_append_paged_rows(const gqa_heads* q, const gqa_heads* k_new, const gqa_heads* v_new,
                                const gqa_heads* q_out, void* k_pool, void* v_pool, const int32_t* block_tables,
                                const int32_t* row_starts, const int32_t* seq_lens_in, int32_t* seq_lens_out, int N,
                                int B, int max_blocks_per_seq, int num_blocks, int block_size, int H, int Hkv, int d_k,
                                int d_v, const void* q_weight, const void* k_weight, float eps, const gqa_rope* rope,
                                gqa_dtype dt, void* stream) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || N < 0 || B < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || block_size <= 0 || H < 0 ||
      Hkv <= 0 || !width_ok(d_k) || !width_ok(d_v) || (long long)H + Hkv > INT_MAX / 2)
    return GQA_ERR_INVALID_ARG;
  if ((long long)max_blocks_per_seq * block_size > INT_MAX / 2) return GQA_ERR_INVALID_ARG;
  if ((q == nullptr) != (H == 0) || (q == nullptr) != (q_out == nullptr)) return GQA_ERR_INVALID_ARG;
  gqa::QkParams p{};
  const gqa_status s = qk_norm_and_rope(p, q_weight, k_weight, eps, rope, d_k);
  if (s != GQA_OK) return s;
  if (B == 0) return GQA_OK;
  if (!k_new || !v_new || !k_pool || !v_pool || !block_tables || !row_starts || !seq_lens_in || !seq_lens_out)
    return GQA_ERR_INVALID_ARG;
  p.q = heads_view(q, 0, N, H);
  p.q_out = heads_view(q_out, 0, N, H);
  p.k = heads_view(k_new, 0, N, Hkv);
  p.v = heads_view(v_new, 0, N, Hkv);
  if (N > 0 && (!heads_view_ok(p.k, bf16) || !heads_view_ok(p.v, bf16) ||
                (q && (!heads_view_ok(p.q, bf16) || !heads_view_ok(p.q_out, bf16) || !in_place_ok(p.q, p.q_out)))))
    return GQA_ERR_INVALID_ARG;
  if (!aligned16(k_pool) || !aligned16(v_pool)) return GQA_ERR_INVALID_ARG;
  const bool same_lens = seq_lens_in == seq_lens_out;
  if (!same_lens && seq_lens_in < seq_lens_out + B && seq_lens_out < seq_lens_in + B) return GQA_ERR_INVALID_ARG;
  p.k_out.data = k_pool;
  p.v_pool = v_pool;
  p.tables = block_tables;
  p.row_starts = row_starts;
  p.lens_in = seq_lens_in;
  p.lens_out = seq_lens_out;
  p.err = error_word();
  if (!p.err) return GQA_ERR_CUDA;
  p.N = N;
  p.B = B;
  p.H = H;
  p.Hk = p.Hkv = Hkv;
  p.dv = d_v;
  p.mbps = max_blocks_per_seq;
  p.bs = block_size;
  p.num_blocks = num_blocks;
  p.run_rows = 1;
  // the lengths are read by every row: written in the same launch only to another array
  p.lens_items = same_lens ? 0 : B;
  const cudaError_t e = gqa::launch_qk_rows(p, bf16, 1, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess || !same_lens) return from_cuda(e);
  p.run_rows = 0;
  p.lens_items = B;
  return from_cuda(gqa::launch_qk_rows(p, bf16, 1, static_cast<cudaStream_t>(stream)));
}

size_t attn_decode_mla_absorbed_workspace_bytes(int B, int H, int d_c, int max_len) {
  if (B <= 0 || H <= 0 || d_c <= 0 || max_len <= 0) return 0;
  const int chunk = gqa::mla_chunk_rows(B, H, max_len);
  if (max_len <= chunk) return 0;
  const size_t splits = (size_t)ceil_div(max_len, chunk);
  return (size_t)B * (size_t)H * splits * (size_t)(d_c + 2) * sizeof(float);
}

// The absorbed MLA decode, contiguous latent cache (tables NULL) or paged pool.
static gqa_status mla_absorbed_common(const void* q_abs, const void* latent, const int32_t* seq_lens, void* out_lat,
                                      int B, int capacity, int H, int d_c, int d_r, float attention_scale, int bf16,
                                      void* workspace, size_t workspace_bytes, cudaStream_t st,
                                      const int32_t* tables, int mbps, int bs, int num_blocks) {
  if (!gqa::mla_absorbed_tc_supported(bf16, d_c, d_r) || !(attention_scale > 0.f)) return GQA_ERR_UNSUPPORTED;
  if (B == 0) return GQA_OK;
  if (!q_abs || !latent || !seq_lens || !out_lat) return GQA_ERR_INVALID_ARG;
  if (!aligned16(q_abs) || !aligned16(latent) || !aligned16(out_lat)) return GQA_ERR_INVALID_ARG;
  const size_t need = attn_decode_mla_absorbed_workspace_bytes(B, H, d_c, capacity);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return GQA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GQA_ERR_INVALID_ARG;
  }
  unsigned* err = error_word();
  if (!err) return GQA_ERR_CUDA;
  const float qscale = attention_scale * 1.4426950408889634f;
  float* partial = need > 0 ? static_cast<float*>(workspace) : nullptr;
  const int chunk = gqa::mla_chunk_rows(B, H, capacity);
  const cudaError_t e = gqa::launch_mla_absorbed_tc(q_abs, latent, seq_lens, out_lat, partial, B, capacity, H, d_c,
                                                    d_r, chunk, qscale, err, st, tables, mbps, bs,
                                                    num_blocks, g_withhold_first_tile);
  if (e != cudaSuccess || need == 0) return from_cuda(e);
  // the splits of each (sequence, head) merged into out_lat
  gqa::RowsParams p{};
  p.out = out_lat;
  p.partial = partial;
  p.kv_len = seq_lens;
  p.B = B;
  p.seq_q = 1;
  p.H = H;
  p.capacity = capacity;
  p.split_rows = chunk;
  p.max_splits = ceil_div(capacity, chunk);
  p.window = 0;
  p.err = err;
  return from_cuda(gqa::launch_split_combine(p, d_c, 1, st));
}

gqa_status attn_decode_mla_absorbed(const void* q_abs, const void* latent, const int32_t* seq_lens, void* out_lat,
                                    int B, int max_len, int H, int d_c, int d_r, float attention_scale, gqa_dtype dt,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || B < 0 || max_len <= 0 || H <= 0 || d_c <= 0 || d_r < 0 || !std::isfinite(attention_scale))
    return GQA_ERR_INVALID_ARG;
  return mla_absorbed_common(q_abs, latent, seq_lens, out_lat, B, max_len, H, d_c, d_r, attention_scale, bf16,
                             workspace, workspace_bytes, static_cast<cudaStream_t>(stream), nullptr, 0, 0, 0);
}

gqa_status attn_decode_mla_absorbed_paged(const void* q_abs, const void* latent_pool, const int32_t* block_tables,
                                          const int32_t* seq_lens, void* out_lat, int B, int max_blocks_per_seq,
                                          int num_blocks, int block_size, int H, int d_c, int d_r,
                                          float attention_scale, gqa_dtype dt, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || B < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || block_size <= 0 || H <= 0 || d_c <= 0 ||
      d_r < 0 || !std::isfinite(attention_scale))
    return GQA_ERR_INVALID_ARG;
  if ((long long)max_blocks_per_seq * block_size > INT_MAX / 2) return GQA_ERR_INVALID_ARG;
  if (!gqa::mla_absorbed_paged_block_ok(block_size)) return GQA_ERR_UNSUPPORTED;
  if (B > 0 && !block_tables) return GQA_ERR_INVALID_ARG;
  return mla_absorbed_common(q_abs, latent_pool, seq_lens, out_lat, B, max_blocks_per_seq * block_size, H, d_c, d_r,
                             attention_scale, bf16, workspace, workspace_bytes, static_cast<cudaStream_t>(stream),
                             block_tables, max_blocks_per_seq, block_size, num_blocks);
}

// y[b, h, :M] = W[h] x[b, h, :K] (+ the tail columns copied): the tensor-core
// kernel for the shapes it takes, else the SIMT one.
static gqa_status head_projection(const void* W, const void* x, int x_stride, void* y, int y_stride, int B, int H,
                                  int M, int K, int tail, cudaStream_t st) {
  if (gqa::head_proj_tc_supported(M, K)) {
    unsigned* err = error_word();
    if (!err) return GQA_ERR_CUDA;
    return from_cuda(gqa::launch_head_proj_tc(W, x, x_stride, y, y_stride, B, H, M, K, tail, err, st));
  }
  return from_cuda(gqa::launch_head_matvec(W, x, x_stride, y, y_stride, B, H, M, K, tail, st));
}

gqa_status mla_absorb_q(const void* q, const void* k_b, void* q_abs, int B, int H, int d_nope, int d_rope, int d_c,
                        gqa_dtype dt, void* stream) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || B < 0 || H <= 0 || d_nope <= 0 || d_rope < 0 || d_c <= 0) return GQA_ERR_INVALID_ARG;
  if (bf16 != 1) return GQA_ERR_UNSUPPORTED;
  if (B == 0) return GQA_OK;
  if (!q || !k_b || !q_abs || q == q_abs) return GQA_ERR_INVALID_ARG;
  if (d_nope % 8 || d_rope % 8 || !aligned16(q) || !aligned16(k_b)) return GQA_ERR_INVALID_ARG;
  return head_projection(k_b, q, d_nope + d_rope, q_abs, d_c + d_rope, B, H, d_c, d_nope, d_rope,
                         static_cast<cudaStream_t>(stream));
}

gqa_status mla_unabsorb_out(const void* out_lat, const void* v_b, void* out, int B, int H, int d_c, int d_v,
                            gqa_dtype dt, void* stream) {
  const int bf16 = dtype_flag(dt);
  if (bf16 < 0 || B < 0 || H <= 0 || d_c <= 0 || d_v <= 0) return GQA_ERR_INVALID_ARG;
  if (bf16 != 1) return GQA_ERR_UNSUPPORTED;
  if (B == 0) return GQA_OK;
  if (!out_lat || !v_b || !out || out == out_lat) return GQA_ERR_INVALID_ARG;
  if (d_c % 8 || !aligned16(out_lat) || !aligned16(v_b)) return GQA_ERR_INVALID_ARG;
  return head_projection(v_b, out_lat, d_c, out, d_v, B, H, d_v, d_c, 0, static_cast<cudaStream_t>(stream));
}

gqa_status attn_get_device_error(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return GQA_ERR_CUDA;
  unsigned word = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&word, g_gqa_error_word, sizeof word) != cudaSuccess) return GQA_ERR_CUDA;
  if (word && cudaMemcpyToSymbol(g_gqa_error_word, &zero, sizeof zero) != cudaSuccess) return GQA_ERR_CUDA;
  if (word & gqa::kErrTimeout) return GQA_ERR_DEVICE_TIMEOUT;
  if (word & gqa::kErrBounds) return GQA_ERR_DEVICE_BOUNDS;
  return GQA_OK;
}

const char* gqa_status_string(gqa_status s) {
  switch (s) {
    case GQA_OK: return "ok";
    case GQA_ERR_INVALID_ARG: return "invalid argument";
    case GQA_ERR_UNSUPPORTED: return "unsupported shape";
    case GQA_ERR_CUDA: return "CUDA error";
    case GQA_ERR_WORKSPACE: return "workspace missing or too small";
    case GQA_ERR_DEVICE_BOUNDS: return "device saw an index or length out of range";
    case GQA_ERR_DEVICE_TIMEOUT: return "a bounded device wait gave up";
  }
  return "unknown status";
}

int gqa_debug_withhold_first_tile(int enable) {
  const int prev = g_withhold_first_tile;
  g_withhold_first_tile = enable ? 1 : 0;
  return prev;
}

}  // extern "C"
