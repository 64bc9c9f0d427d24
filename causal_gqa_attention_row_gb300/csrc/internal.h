// internal.h -- host-side declarations shared by the translation units of
// libgqa_attn.so (not part of the public ABI; see include/gqa_attn.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gqa {

// Bits of the device error word.
enum : unsigned { kErrBounds = 1u, kErrTimeout = 2u };

// Rows of one split-K work item of the decodes. Their split boundaries are multiples of
// this, a fixed number independent of the layout and of the rest of the batch, so the
// paged and contiguous decodes of one history do identical arithmetic.
constexpr int kSplitRows = 2048;
// The shortest split that attn_cross takes (from there up to kSplitRows by powers of two).
constexpr int kLeastSplitRows = 256;

// Parameters of the SIMT attention kernel (decode, and prefill shapes that the
// tensor-core kernel does not take). All pointers are device pointers.
struct RowsParams {
  const void* q;            // [B, seq_q, H, DK]
  const void* k;            // contiguous [B, Hkv, max_len, DK-DROT] or pool [nb, Hkv, bs, DK]
  const void* v;            // contiguous [B, Hkv, max_len, DV] or pool [nb, Hkv, bs, DV]
  const void* k_rot;        // contiguous only: [B, max_len, DROT]
  void* out;                // [B, seq_q, H, DV]
  float* partial;           // [B*seq_q*H, max_splits, DV+2] when max_splits > 1
  int* sched;               // split-K plan: [0] ticket counter, [1] units listed; NULL without a workspace
  int2* units;              // split-K plan: the listed (item, split) units
  const int32_t* kv_len;    // [B] keys present (decode), or NULL: offsets[b] + seq_q
  const int32_t* offsets;   // [B] or NULL (prefill)
  const int32_t* tables;    // paged: [B, mbps]
  unsigned* err;            // device error word
  int paged;
  int B, seq_q, H, Hkv, G;  // G = H / Hkv
  int GH, QR;               // query heads and query rows per work item (GH*QR = NV)
  int n_hchunks, n_rblocks; // G / GH, ceil(seq_q / QR)
  int max_len;              // contiguous rows per (b, kvh); 0 when paged
  int capacity;             // largest valid key count of one sequence
  int mbps, bs, num_blocks; // paged
  int split_rows;           // rows per split (kLeastSplitRows .. kSplitRows, or >= capacity for no split)
  int max_splits;
  float qscale;             // attention_scale * log2(e)
  int debug_withhold;       // test hook: withhold the first tile of every CTA
  // The arms of the attention row (all off when zero / NULL): a row at
  // position p sees keys first_visible_key(p, window)..p; scores s (natural
  // units) become softcap * tanh(s / softcap), then s + alibi[h] * (j - p); the
  // sink logit sinks[h] joins the softmax denominator only.
  int window;               // > 0: the last `window` positions; <= 0: no window
  float softcap2;           // softcap * log2(e) (the kernels score in the log2 domain); 0: none
  const float* sinks;       // [H] device, natural units, or NULL
  const float* alibi;       // [H] device, natural units, or NULL
  // No causal rule (attn_cross): every row sees all keys of its sequence, which may
  // hold none (its rows are zeros); kv_len NULL stands for `capacity` keys.
  int full;
};

// Keys present in sequence b, and whether the call takes that many.
__host__ __device__ inline int rows_kv_len(const RowsParams& p, int b) {
  return p.kv_len ? p.kv_len[b] : p.full ? p.capacity : (p.offsets ? p.offsets[b] : 0) + p.seq_q;
}
__host__ __device__ inline bool rows_len_ok(const RowsParams& p, int kv_len) {
  return (p.full || kv_len >= p.seq_q) && kv_len >= 1 && kv_len <= p.capacity;
}
// Keys that query row i sees (the row's own limit; window apart).
__host__ __device__ inline int rows_limit(const RowsParams& p, int kv_len, int i) {
  return p.full ? kv_len : kv_len - p.seq_q + i + 1;
}

constexpr float kLog2e = 1.4426950408889634f;

// First key a row at position p sees: p - window + 1 (not below 0) with a
// window, else 0.
__host__ __device__ inline int first_visible_key(int p, int window) {
  return (window > 0 && p - window + 1 > 0) ? p - window + 1 : 0;
}

// Dispatch of the SIMT kernel by element type and head widths; NV = GH * QR.
// Returns cudaErrorNotSupported when there is no instantiation.
cudaError_t launch_attn_rows_f32(const RowsParams& p, int dk, int dv, int drot, int nv, cudaStream_t st);
cudaError_t launch_attn_rows_bf16(const RowsParams& p, int dk, int dv, int drot, int nv, cudaStream_t st);
// Largest NV the instantiation set offers for these widths (0 = unsupported).
int rows_max_nv(int bf16, int dk, int dv, int drot);

cudaError_t launch_split_combine(const RowsParams& p, int dv, int bf16, cudaStream_t st);

// The split-K plan: lists the units with keys into p.units and resets the
// ticket counter (p.sched must be set).
cudaError_t launch_plan_units(const RowsParams& p, cudaStream_t st);

// Split-K workspace layout: the plan (ticket counter and total, then the unit
// list), then the partial results.
constexpr size_t kPlanHeaderBytes = 256;
inline size_t round_up256(size_t n) { return (n + 255) / 256 * 256; }
inline size_t plan_bytes(size_t units_max) { return kPlanHeaderBytes + round_up256(units_max * 8); }

// x2 != NULL: a second tensor of the same tokens (heads2 heads, its own layout)
// turned by the same angles in the same launch.
cudaError_t launch_rope(void* x, const int32_t* positions, int B, int T, int heads, int d, int heads_outer,
                        int rot_offset, int rot_dim, double theta, int bf16, cudaStream_t st, void* x2 = nullptr,
                        int heads2 = 0, int heads_outer2 = 0);

cudaError_t launch_append(void* q, const void* k_new, const void* v_new, void* k_pool, void* v_pool,
                          const int32_t* tables, const int32_t* lens_in, int32_t* lens_out, int B, int mbps,
                          int num_blocks, int bs, int H, int Hkv, int dk, int dv, double theta, int rot_offset,
                          int rot_dim, int bf16, unsigned* err, cudaStream_t st);

// A tensor [batch, tokens, heads, d] with its last axis dense; strides in elements.
struct HeadsView {
  void* data;
  int64_t batch_stride, token_stride, head_stride;
};

// Parameters of the q/k row kernel (norm, rotation, paged write).
struct QkParams {
  HeadsView q, k, q_out, k_out;  // PAGED: k_out.data is the key pool, no batch axis
  HeadsView v;                   // PAGED
  void* v_pool;
  const void* q_weight;          // [d] of the element type, or NULL: no norm
  const void* k_weight;
  const int32_t* positions;      // [B, T] (not PAGED), [N] with slots
  const float* freqs;            // [rot_dim / 2] float pairs (high, low part) of the frequencies
  const int32_t* tables;         // PAGED, from here on: as kv_append_paged_rows
  const int32_t* row_starts;
  const int32_t* lens_in;
  int32_t* lens_out;
  unsigned* err;
  int N, T, B;                   // N token rows (= B * T when not PAGED)
  int H, Hk, Hkv;                // query heads, key heads turned (0 without keys), KV heads of the pool
  int d, dv;
  int layout, rot_offset, rot_dim;  // layout 1: half pairs; rot_dim 0: no rotation
  float magnitude, eps;
  int parts, part_rows, first_part, lens_part;  // items per token, rows of one (set by the launcher)
  int mbps, bs, num_blocks;
  const int64_t* slots;          // [N] pool slots (block * bs + row; below 0: none), instead of tables,
                                 // row_starts and lengths; NULL: those
  int run_rows;                  // 0: only the lengths
  int lens_items;                // sequences whose length this launch advances (0 or B)
};
cudaError_t launch_qk_rows(const QkParams& p, int bf16, int paged, cudaStream_t st);

// ---- a step's index arrays and accepted rows (plan_rows.cu, commit_rows.cu) ------
// Parameters of kv_plan_rows (include/gqa_attn.h has the meaning of the arrays).
struct PlanRows {
  const int32_t *lens, *new_rows, *keep, *parents;
  int32_t* tables;
  const int32_t* held_in;
  int32_t* held_out;
  int32_t* free_list;
  const int32_t* free_in;
  int32_t *free_out, *row_starts, *positions;
  int64_t* slots;
  unsigned long long* mask;
  unsigned* err;
  int N, B, words, mbps, num_blocks, bs;
  // set by the launcher
  int per, lanes;                       // sequences of a CTA, threads of a sequence
  int write_rows, write_state, report;  // what this launch writes (see there)
};
// Sequences of a call: their prefix sums stay in shared memory.
constexpr int kPlanRowsMaxB = 16384;
cudaError_t launch_plan_rows(PlanRows p, cudaStream_t st);

// Parameters of kv_commit_rows, of up to kCommitLayers layers a launch.
constexpr int kCommitLayers = 64;
struct CommitRows {
  void* k_pools[kCommitLayers];
  void* v_pools[kCommitLayers];  // NULL: none
  const int32_t *tables, *lens_in, *row_starts, *path, *n_path;
  int32_t* lens_out;
  unsigned* err;
  int n_layers, B, max_path, mbps, num_blocks, bs, Hkv;
  int k_bytes, v_bytes;          // of a row
  int lens_only, lens_later;     // this launch writes the lengths alone; another launch does
};
cudaError_t launch_commit_rows(const CommitRows& p, cudaStream_t st);

// The arms for the tensor-core prefill: window (<= 0: none), softcap * log2 e
// (0: none), sink logits and ALiBi slopes ([H] fp32 on the device, natural
// units, or NULL).
struct TcArms {
  int window;
  float softcap2;
  const float* sinks;
  const float* alibi;
};

// tcgen05 causal prefill (bf16, d_k = d_v = 64). Returns cudaErrorNotSupported
// for other shapes. Contiguous k, v [B, Hkv, seq_kv_max, 64] (tables NULL), or
// paged pools [num_blocks, Hkv, bs, 64] with block tables [B, mbps] and
// seq_kv_max = mbps * bs.
cudaError_t launch_prefill_tc(const void* q, const void* k, const void* v, void* out, int B, int seq_q,
                              int seq_kv_max, const int32_t* offsets, int H, int Hkv, int dk, int dv,
                              float qscale, unsigned* err, cudaStream_t st, const int32_t* tables = nullptr,
                              int mbps = 0, int bs = 0, int num_blocks = 0, const TcArms* arms = nullptr,
                              int debug_withhold = 0);
// bs = 0: contiguous K/V; else the pool's block size and max blocks per sequence.
bool prefill_tc_supported(int bf16, int dk, int dv, int bs = 0, int mbps = 0);

// ---- attention without a causal rule on tcgen05 (dense_tc.cu) -----------------
// How the attention of drafted rows is cut into work (tree_part.cuh).
constexpr int kTreeSeqs = 500;  // sequences of a launch: their table stays in shared memory
struct alignas(16) TreeRec {    // what the join reads of a row tile
  int row, n, hc, b;            // its first packed row, its drafted rows; KV head and head chunk; sequence
  int part, parts, stride, hist;  // its partial results: part, part + stride, .. (0: written whole); the sequence's history
  int row0, rows, pad[2];         // and its rows
};
struct TreeWork {
  const int32_t *row_starts, *offsets;
  const unsigned long long* mask;  // [N, words], or NULL: every row sees those up to its own
  int N, B, max_rows, words;
  int heads, GH, RPT, R;           // KV heads times head chunks; heads and rows of a tile; rows of a partial result
  int capacity, bs, window;
  int step_log2;                   // keys of a tile
  int keys_once;                   // no key is read for a second row tile
  int whole;                       // a unit of all of an item's keys writes its rows' outputs itself
  int slots, pair_slots;           // pieces of the line of single tiles, and of pairs (0: no pairs)
  TreeRec* rec;                    // of each row tile
  uint8_t* odd;                    // [row tiles][4]: of those written whole, a quarter's rows hold a value that is not finite
  int* line;                       // [0] the row tiles
  unsigned* err;
};

// One unit of work: rows i0 .. i0 + n_i - 1 of heads head0 .. head0 + GH - 1 against keys
// key0 .. key1 - 1 of sequence seq (key0 a multiple of the pool's block size). part: where
// the partial result goes, in 16-byte steps from DenseParams::partial (-1: final results);
// batch: attn_cross, the sequence's place in q and out; own: shared prefix, a unit of one
// sequence's own keys, with a partial result of own_rows rows instead of 128.
struct alignas(16) DenseUnit {
  int i0, n_i, head0, seq;
  int key0, key1, part, batch_or_own;
};

// A partial result of R rows: o [d_v / 4][R][4], then m [R] (log2 units) and l [R].
__host__ __device__ inline size_t dense_part_floats(int R, int dv) { return (size_t)R * (size_t)(dv + 2); }

struct DenseParams {
  int H, G;
  int GH, RPT, n_hchunks;  // rows of a tile: RPT rows i x GH heads (dense_rows)
  int n_i;                 // rows i of a sequence (attn_cross: seq_q; shared prefix: B)
  int S_kv;                // keys a sequence can hold
  // attn_cross: units from their index, key ranges of split_tiles tiles
  int Hkv, n_units;
  const int32_t* kv_lens;  // [B] or NULL: S_kv
  int n_tiles, n_splits, split_tiles;
  // shared prefix: units from the plan, a length per row
  const DenseUnit* units;
  const int* units_listed;
  int* ticket;             // 0 at the launch
  const int32_t* seq_lens;
  int own_rows;
  const int32_t* tables;   // paged pools (NULL: contiguous)
  int mbps, bs, num_blocks;
  float* partial;
  __nv_bfloat16* out;
  float qscale;
  unsigned* err;
  int debug_withhold;
  int window;              // the arms, as for the tensor-core prefill
  float cap_in, cap_out;
  const float* alibi;
  // drafted rows: units from the line, a mask per row; q and out [N, H, d]
  TreeWork tree;
};

// Heads of a group per row tile (the largest divisor of G that is at most 128) and
// rows i per tile.
void dense_rows(int G, int* GH, int* RPT);
bool dense_tc_supported(int bf16, int dk, int dv, int bs = 0);
bool tree_tc_supported(int bf16, int dk, int dv, int bs = 0);  // of drafted rows: (256, 256) too
// Units that the SMs work on at a time.
int dense_tc_slots(int dk);
cudaError_t launch_dense_tc(const void* q, const void* k, const void* v, const DenseParams& p, int n_b, int dk, int dv,
                            bool arms, cudaStream_t st);

// A group of sequences with a shared prefix (the planner's record).
struct alignas(16) DenseGroup {
  int first, members, tiles, n_splits;  // row tiles, key ranges (key tiles until they are chosen)
  int unit0, key_lo, prefix;            // its first unit; the keys [key_lo, prefix) that the members who share all see
  int sharers, source;                  // how many do, and the first of them, whose table entries are read
  int pad[3];
};

// One sequence of a shared-prefix step, for the combine: n_pre key ranges, for head chunk c
// in units pre_unit0 + c * pre_stride on, its row row0 + (head within the chunk); n_own
// parts of its own keys, for head chunk c in own parts own_part0 + c * n_own on.
struct alignas(16) SeqPlan {
  int n_pre, pre_unit0, pre_stride, row0;
  int n_own, own_part0, full0, pad;  // full0: the first of its full own units (the planner's)
};

struct DenseCombine {
  int n_b, n_i, H;         // output rows [n_b, n_i, H] of dv (64 or 128) columns
  int GH, RPT, dv;
  int n_tiles, n_splits;   // attn_cross
  const float* partial;
  const SeqPlan* seq;      // shared prefix
  const float* own_partial;
  int own_rows;
  const float* sinks;
  __nv_bfloat16* out;
};
cudaError_t launch_dense_combine(const DenseCombine& p, cudaStream_t st);

// A plan's cost is counted in key tiles: what a unit takes beside its tiles (the first
// tile's latency, the epilogue and its share of the join).
constexpr int kDenseUnitTiles = 1;
constexpr int kDenseSms = 152;

// Parts of own keys beyond two per item (sequence, KV head, head chunk) that a plan may make.
constexpr int kOwnExtra = 4 * kDenseSms;

// The plan of a shared-prefix step: the units of the prefixes and of the own keys, and what
// each sequence has.
struct SharedPlan {
  const int32_t* seq_lens;
  const int32_t* group_starts;   // [n_groups + 1]
  const int32_t* shared_blocks;  // [n_groups]
  int B, Hkv, capacity, bs, mbps, window, dv;
  int n_groups, max_prefix_units, slots;
  int GH, RPT, n_hchunks, own_rows;
  int own_part_at;               // where the own parts begin, in 16-byte steps from the partial results
  DenseGroup* groups;            // scratch [n_groups], used where they do not fit shared memory
  SeqPlan* seq;                  // [B]
  DenseUnit* units;
  int* units_listed;
  unsigned* err;
};
cudaError_t launch_shared_plan(const SharedPlan& s, cudaStream_t st);

// ---- attention of drafted rows (attn_tree_paged) ---------------------------------
// On the tensor cores (dense_tc.cu; launch_dense_tc with p.tree.row_starts set), or on the SIMT kernel
// (tree_rows.cu) for every other type, width and block size; both leave partial results of R rows, which
// launch_tree_combine joins.
struct TreeParams {
  TreeWork w;
  const void *q, *k, *v;           // [N, H, d_k], pools
  void* out;                       // [N, H, d_v]
  const int32_t* tables;
  float* partial;
  int H, G, Hkv, mbps, num_blocks, dk, dv;
  float qscale;                    // attention_scale * log2(e)
  float softcap2;                  // softcap * log2(e), 0: none
  const float *sinks, *alibi;
  int check;                       // the join looks for values that rows do not see but the products mixed in
  int tiles;                       // row tiles, at most
};
int tree_rows_ctas(int bf16, int dk, int dv);  // of the SIMT kernel an SM (0: width not taken)
int tree_rows_tile();                          // rows (times heads) of its tile
cudaError_t launch_tree_rows(const TreeParams& p, int bf16, cudaStream_t st);
cudaError_t launch_tree_combine(const TreeParams& p, int bf16, cudaStream_t st);

// Absorbed MLA decode on tcgen05 (bf16, d_c = 512, d_r = 64): attention of
// q_abs [B, H, d_c + d_r] over the latent rows [B, max_len, d_c + d_r] (value =
// the first d_c columns) into out_lat [B, H, d_c]; splits of `chunk` rows write
// (m, l, o) into partial [B * H, ceil(max_len / chunk), d_c + 2] when a sequence
// has more than one, and the split combine merges them.
bool mla_absorbed_tc_supported(int bf16, int d_c, int d_r);
// Paged (tables != NULL): latent is a pool [num_blocks, bs, d_c + d_r], max_len
// is ignored (mbps * bs rows per sequence), bs one of 8, 16, 32, 64.
cudaError_t launch_mla_absorbed_tc(const void* q_abs, const void* latent, const int32_t* seq_lens, void* out_lat,
                                   float* partial, int B, int max_len, int H, int d_c, int d_r, int chunk,
                                   float qscale, unsigned* err, cudaStream_t st, const int32_t* tables = nullptr,
                                   int mbps = 0, int bs = 0, int num_blocks = 0, int debug_withhold = 0);
bool mla_absorbed_paged_block_ok(int bs);
// Rows of one split of the absorbed MLA decode: 1024, doubled (up to 8192) while
// the (sequence, head tile, split) clusters of a call at its capacity would still
// number at least 64 (one wave of the GPU's 76 two-CTA cluster slots, nearly
// filled), so that a batch fills the GPU with as few partial results to merge
// as it can. A function of B, H and the capacity alone: a sequence's result does
// not depend on the lengths of the others, and two calls with the same three
// values split alike.
constexpr int kMlaChunk = 1024;
inline int mla_chunk_rows(int B, int H, int capacity) {
  const long long clusters_per_split = (long long)B * ((H + 127) / 128);
  int chunk = kMlaChunk;
  while (chunk < 8192 && clusters_per_split * (((long long)capacity + 2 * chunk - 1) / (2 * chunk)) >= 64) chunk *= 2;
  return chunk;
}

// y[b, h, :M] = W[h] x[b, h, :K] (bf16, fp32 accumulation), W [H, M, K]; the
// `tail` columns of x after K are copied to y after M.
cudaError_t launch_head_matvec(const void* W, const void* x, int x_stride, void* y, int y_stride, int B, int H, int M,
                               int K, int tail, cudaStream_t st);

// The same product on tcgen05 (bf16): W's rows in tiles of 128 (M % 128 == 0),
// K % 64 == 0 and K <= 512; cudaErrorNotSupported otherwise.
bool head_proj_tc_supported(int M, int K);
cudaError_t launch_head_proj_tc(const void* W, const void* x, int x_stride, void* y, int y_stride, int B, int H, int M,
                                int K, int tail, unsigned* err, cudaStream_t st);

}  // namespace gqa
