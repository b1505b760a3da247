// Internal interface between the C-ABI layer (gw_abi.cu) and the kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/gw.h"

namespace gw {

// ---- split-KV plan constants ------------------------------------------------
// A local decode work unit is (sequence, KV head, chunk of kLocalChunkPages
// logical pages of that sequence's window); a global unit is (sequence, chunk
// of global_chunk_pages(L) pages).  Chunks depend only on the sequence's own
// length, so a row's arithmetic never depends on the rest of the batch.
constexpr int kLocalChunkPagesBf16 = 8;
constexpr int kLocalChunkPagesE4m3 = 8;
// Global chunks start at 32 pages and double until a sequence has at most
// kGlobalMaxChunks of them (long contexts get long chunks, so the partials
// stay a small fraction of the KV bytes).
constexpr int kGlobalChunkPagesMin = 32;
constexpr int kGlobalMaxChunks = 128;

// The decode kernels keep the batch's split plan in shared memory.
constexpr int kMaxBatch = 4096;


__host__ __device__ __forceinline__ int local_chunks(int L, int window, int chunk) {
  const int first = L > window ? L - window : 0;
  const int p0 = first / 16, p1 = (L - 1) / 16;
  return (p1 - p0 + chunk) / chunk;
}

// An upper bound on local_chunks(L, window, chunk) over L <= 16 * max_pages.
__host__ __device__ __forceinline__ int local_max_chunks(int max_pages, int window, int chunk) {
  const int span = (window - 1) / 16 + 1;  // p1 - p0 once L > window
  const int d = max_pages - 1 < span ? max_pages - 1 : span;
  return (d + chunk) / chunk;
}

// An upper bound on global_chunks(L) over L <= 16 * max_pages.
__host__ __device__ __forceinline__ int global_max_chunks(int max_pages) {
  const int c = (max_pages + kGlobalChunkPagesMin - 1) / kGlobalChunkPagesMin;
  return c < kGlobalMaxChunks ? c : kGlobalMaxChunks;
}

__host__ __device__ __forceinline__ int global_chunk_pages(int L) {
  const int pages = (L + 15) / 16;
  int cpg = kGlobalChunkPagesMin;
  while ((pages + cpg - 1) / cpg > kGlobalMaxChunks) cpg *= 2;
  return cpg;
}

__host__ __device__ __forceinline__ int global_chunks(int L) {
  const int cpg = global_chunk_pages(L);
  return ((L + 15) / 16 + cpg - 1) / cpg;
}

// ---- drafted trees (gw_tree_attn_*) ------------------------------------------
// A work unit is (sequence, KV head or half of the output dims, block of rows
// with the heads that share their K and V, chunk of tiles); a tile is 64 tokens,
// aligned to 64.  Chunks depend on the sequence's own length, rows and window
// only (and the call's bound on rows), as the decode's.
constexpr int kMaxTreeRows = 64;    // rows of a sequence: the bits of a mask word
constexpr int kMaxTreeBatch = 256;  // sequences of a call: their plan is in shared memory
constexpr int kTreeTile = 64;
constexpr int kTreeRows = 128;    // rows x heads of a block
// Rows x heads up to which a call's rows lie along N: what the accumulators of all
// dims leave room for, three terms of P wide on e4m3 pools.
__host__ __device__ constexpr int tree_few_rows(int layout) {
  return layout == GW_LAYOUT_GLOBAL_FOLDED || layout == GW_LAYOUT_GLOBAL_FULL ? 64 : 32;
}
constexpr int kTreeMaxChunks = 76;

// How a call is cut: `per` rows in a block, chunks of at most `aim` tiles, at most
// `most` of them unless a block has one.
struct TreeRule {
  int per, aim, most;
};

// Local layers: a window of 1024 is one chunk (in two, 16 sequences with 16 drafts
// take 61 us instead of 50, one sequence 18 instead of 21).
__host__ __device__ constexpr TreeRule tree_rule_local(int group) { return {kTreeRows / group, 18, 38}; }
// Global layers, rows along M: units (two a chunk and block) enough for the GPU's
// 152 SMs, few enough that their parts, 128 KB a unit, stay small beside the cache
// (8 x 131072 tokens, one block: 367 us with up to 38 chunks, 404 with 76; 344 with
// 19, which would leave a lone sequence a fourth of the SMs).  Short chunks serve
// few sequences, long ones many: over 124 calls of 1 to 32 sequences of 2048 to 32768
// tokens (some with lengths 1 : 16 apart), 1, 2 and 4 blocks, all layouts, chunks of
// 8, 16, 24, 32 and 40 tiles took 1.14, 1.16, 1.23, 1.31 and 1.34 times the best of
// the five in the geometric mean and 1.81, 1.55, 1.82, 2.46 and 2.45 times at worst.
// One sequence of 8192 tokens, four blocks, 32, 41, 49, 61 and 61 us; 16 of 512 to
// 8192, one block 52, 45, 53, 62 and 72, four 182, 139, 131, 130 and 121; 32 of
// 8192, four blocks 579, 458, 443, 395 and 395.
__host__ __device__ constexpr TreeRule tree_rule_global(int heads) { return {kTreeRows / heads, 16, 38}; }
// Global layers, rows along N: one unit of 64 or 128 KB of parts a chunk (8 x 131072
// tokens, 4 drafts of 8 heads: 224 us with up to 38 chunks instead of 231, but a lone
// sequence has as many SMs as chunks).  One sequence of 8192 tokens: chunks of 8
// tiles 23 us, of 6 20, of 12 26; 16 of 512 to 8192: 30, 40 and 35.
__host__ __device__ constexpr TreeRule tree_rule_few(int heads) { return {kTreeRows / heads, 8, kTreeMaxChunks}; }

__host__ __device__ __forceinline__ int tree_most_chunks(const TreeRule& rule, int blocks) {
  const int shared = kTreeMaxChunks / blocks;
  const int most = shared < rule.most ? shared : rule.most;
  return most > 1 ? most : 1;
}

struct TreeSpan {
  int first;   // first tile
  int tiles;   // tiles [first, first + tiles)
  int blocks;  // blocks of rows
  int ct;      // tiles of a chunk: even chunks
  __host__ __device__ int chunks() const { return (tiles - 1) / ct + 1; }
};

// Of n rows over L >= n >= 1 tokens.  Rows sit at tokens L - n and later, so the
// first key of any is L - n - window + 1.
__host__ __device__ __forceinline__ TreeSpan tree_span(int L, int n, int window, const TreeRule& rule) {
  TreeSpan s;
  const int lo = L - n - window + 1;
  s.first = lo > 0 ? lo / kTreeTile : 0;
  s.tiles = (L - 1) / kTreeTile - s.first + 1;
  s.blocks = (n + rule.per - 1) / rule.per;
  const int most = tree_most_chunks(rule, s.blocks);
  const int want = (s.tiles - 1) / rule.aim + 1, chunks = want < most ? want : most;
  s.ct = (s.tiles - 1) / chunks + 1;
  return s;
}
// A bound on a sequence's chunks over L <= 16 * max_pages and n <= max_rows.
__host__ __device__ __forceinline__ int tree_max_chunks(int max_pages, int max_rows, int window, const TreeRule& rule) {
  // tokens in sight: all, or window - 1 cached ones and the drafts, in tiles they need not begin
  const int64_t all = (static_cast<int64_t>(max_pages) * 16 + kTreeTile - 1) / kTreeTile;
  const int64_t seen = (static_cast<int64_t>(window) + max_rows + kTreeTile - 3) / kTreeTile + 1;
  const int64_t c = ((all < seen ? all : seen) + rule.aim - 1) / rule.aim;
  return static_cast<int>(c < rule.most ? c : rule.most);
}

// Workspace layout (offsets from the 256-byte aligned workspace base):
//   [0, 256)          reserved
//   [256, ub_end)     int32 unit_base[batch + 1], rounded up to 256 bytes
//   [ub_end, ml_end)  float2 (m, l) per (unit, head of the unit)
//   [ml_end, o_end)   float  o[unit][head of the unit][head_dim]
//   [o_end, ...)      int32 prompt_base[batch + 1] (prompt-row tile offsets)
struct WsLayout {
  size_t reserved, unit_base, ml, o, prompt_base, total;
  int64_t max_units;
  int heads_per_unit;
};

WsLayout ws_layout(int layout, int dtype, int kv_heads, int num_q_heads, int batch, int max_seq_len,
                   int window);

struct LocalArgs {
  const uint8_t* pool;
  int64_t num_pages;
  int32_t kv_heads;
  int32_t num_q_heads;
  const uint16_t* q;  // bf16 bits
  uint16_t* out;      // bf16 bits
  int32_t batch;
  const int32_t* cu_q_rows;
  const int32_t* seq_lens;
  const int32_t* block_table;
  int32_t max_pages;
  int32_t window;  // local; ignored for global
  float scale_log2;  // softmax scale * log2(e)
  int32_t* unit_base;
  float2* part_ml;
  float* part_o;
  int64_t max_units;
  int32_t* status;
  int32_t* prompt_base;  // tile offsets of the prompt-row kernels
  float* lse;            // optional: natural-log log-sum-exp per (decode row, q head)
  // Fused append (gw_append_decode_attn_*): the K/V row of each decode row,
  // at position seq_len - 1, written by the decode kernel; k_new null: none.
  const uint16_t* k_new;
  const uint16_t* v_new;
  const float* rope_cs;
  int32_t max_pos;
  int32_t early_inputs;  // gw_set_early_inputs: plan before the wait on the previous kernel
  // Attention weights (gw_decode_attn_global_acc); score null: none.
  float* score;    // [batch][max_pages * 16][num_q_heads], logits in base-2 units
  float* acc;      // [batch][acc_stride]
  int64_t acc_stride;
  float decay;
  // Drafted trees (gw_tree_attn_*); tree_mask null: none.
  const uint64_t* tree_mask;  // [total_rows]: visible drafts of each row
  const int32_t* tree_pos;    // [total_rows], local only
  int32_t max_q_rows;         // bound on a sequence's rows
  int32_t part_rows;          // rows of a unit's partials
};

struct AppendArgs {
  uint8_t* pool;
  int64_t num_pages;
  int32_t kv_heads;
  const uint16_t* k;
  const uint16_t* v;
  int32_t num_rows;
  const int32_t* slot;
  const int32_t* pos;
  const float* rope_cs;
  int32_t max_pos;
  int32_t* status;
  int32_t early_inputs;  // gw_set_early_inputs: slot, pos and RoPE rows read before the wait
};

int num_sms();
// CTAs of a persistent attention kernel: one per SM, or the calling thread's
// gw_set_max_ctas cap if smaller.
int grid_ctas();
// Whether this thread's launches may start before their predecessor in the
// stream has finished (programmatic dependent launch); gw_set_early_launch.
bool early_launch();
// Whether the calling thread's calls may read their index inputs before the
// previous kernel of their stream has finished; gw_set_early_inputs.
bool early_inputs();

// Every host-side check of gw_decode_attn_local, workspace size included,
// with errors reported under the name `fn`; launches nothing.
gw_status validate_local_call(const char* fn, const gw_kv_pool* pool, const void* q, void* out, int32_t num_q_heads,
                              int32_t batch, const int32_t* cu_q_rows, const int32_t* seq_lens,
                              const int32_t* block_table, int32_t max_pages_per_seq, int32_t max_q_rows,
                              int32_t window, float scale, size_t workspace_bytes, int32_t* dev_status);

// Records `fmt` (printf-style) as the calling thread's gw_last_error message,
// prefixed by `fn`, and returns `code`.
gw_status set_error(gw_status code, const char* fn, const char* fmt, ...);

// Log-sum-exp merge of each decode row's partials into bf16 `out`; units of
// heads_per_unit q heads, planned as in a.unit_base, at most max_chunks
// chunks per sequence; with `discard`, the merged partials' L2 lines are
// dropped unwritten.  With a.score, also the weights pass of
// gw_decode_attn_global_acc.
cudaError_t launch_combine(const LocalArgs& a, int heads_per_unit, int head_dim, int max_chunks, bool discard,
                           cudaStream_t st);

cudaError_t launch_append(int layout, int dtype, const AppendArgs& a, cudaStream_t st);

// Up to kMaxMergeParts attention results of the same rows over disjoint key
// sets, merged by their log-sum-exp (gw_merge_lse).
constexpr int kMaxMergeParts = 16;
struct MergeArgs {
  const uint16_t* o[kMaxMergeParts];  // bf16 [rows][heads][head_dim]
  const float* lse[kMaxMergeParts];   // [rows][heads], natural log
  int32_t n_parts, rows, heads, head_dim;
  uint16_t* out;
  float* lse_out;
};
cudaError_t launch_merge_lse(const MergeArgs& m, cudaStream_t st);
// (cos, sin) table of gw_rope_cs: float32 [max_pos][rot_dim / 2][2].
cudaError_t launch_rope_cs(float* out, double theta, int rot_dim, int head_dim, int max_pos, cudaStream_t st);
// gw_rope_rows: strides in elements; `inplace` rows keep their unrotated dims.
struct RopeRowsArgs {
  const void* x;
  void* y;
  int64_t x_row, x_head, y_row, y_head;
  int32_t num_rows, num_heads, head_dim, rot_dim;
  int32_t pairs, inverse, inplace;
  const int32_t* pos;
  const float* rope_cs;
  int32_t max_pos;
  int32_t* status;
  int32_t early_inputs;  // gw_set_early_inputs: pos and RoPE rows read before the wait
};
cudaError_t launch_rope_rows(int elem, const RopeRowsArgs& a, cudaStream_t st);
// The pairs' frequencies of gw_rope_cs_scaled, computed on the host in float64:
// turns per position modulo 1, as a 96-bit binary fraction.
constexpr int kMaxRopePairs = 256;
struct RopeFreqs {
  uint64_t hi[kMaxRopePairs];
  uint32_t lo[kMaxRopePairs];
};
cudaError_t launch_rope_cs_scaled(float* out, const RopeFreqs& freqs, double amplitude, int half, int max_pos,
                                  cudaStream_t st);
// gw_kv_evict_select
struct SelectArgs {
  const float* acc;
  int64_t acc_stride;
  int32_t batch;
  const int32_t* seq_lens;
  int32_t budget, sinks, recent;
  int32_t* keep_idx;
  int64_t keep_stride;
  int32_t* keep_lens;
  int32_t* status;
};
cudaError_t launch_evict_select(const SelectArgs& a, cudaStream_t st);
// gw_kv_evict_compact
struct CompactArgs {
  uint8_t* pool;
  int64_t num_pages;
  int32_t batch;
  const int32_t* block_table;
  int32_t max_pages;
  const int32_t* seq_lens;
  const int32_t* keep_idx;
  int64_t keep_stride;
  const int32_t* keep_lens;
  const int32_t* dst_table;  // == block_table in place
  int32_t dst_max_pages;
  float* acc;
  int64_t acc_stride;
  int32_t* status;
};
cudaError_t launch_evict_compact(int layout, const CompactArgs& a, cudaStream_t st);
// gw_norm_rope_append: strides in elements; `tied`: v is k's projection (one
// global KV head); `run`: heads per warp, set by the launch.
struct NormRopeArgs {
  uint8_t* pool;
  int64_t num_pages;
  int32_t kv_heads;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head;
  int32_t num_rows, num_q_heads;
  const float* q_weight;
  const float* k_weight;
  float eps;
  int32_t v_norm, tied, run;
  const int32_t* slot;
  const int32_t* pos;
  const float* rope_cs;
  int32_t max_pos;
  uint16_t* out;
  int32_t* status;
  int32_t early_inputs;  // gw_set_early_inputs: slot, pos and RoPE rows read before the wait
};
cudaError_t launch_norm_rope(int layout, int dtype, const NormRopeArgs& a, cudaStream_t st);

constexpr int kMaxTreePools = 64;  // pools of a gw_kv_tree_move call
// gw_tree_accept
struct TreeAcceptArgs {
  int32_t batch;
  int32_t max_q_rows;
  const int32_t* cu_q_rows;
  const int32_t* seq_lens;
  const int32_t* parent;
  const int32_t* draft;
  const int32_t* target;
  int32_t* path;
  int64_t path_stride;
  int32_t* path_lens;
  int32_t* next_tokens;  // or null
  int32_t* new_lens;     // or null
  int32_t* status;
};
// gw_tree_attn_*: the attention kernel, then the merge of the chunks of the
// sequences that have several
cudaError_t launch_local_tree(int dtype, int group, const LocalArgs& a, cudaStream_t st);
cudaError_t launch_global_tree(int layout, const LocalArgs& a, cudaStream_t st);
cudaError_t launch_local_tree_few(int dtype, int group, const LocalArgs& a, cudaStream_t st);
cudaError_t launch_local_tree_rows(int dtype, int group, const LocalArgs& a, cudaStream_t st);
cudaError_t launch_global_tree_few(int layout, const LocalArgs& a, cudaStream_t st);
cudaError_t launch_global_tree_rows(int layout, const LocalArgs& a, cudaStream_t st);
cudaError_t launch_tree_accept(const TreeAcceptArgs& a, cudaStream_t st);
// gw_kv_tree_move
struct TreeMoveArgs {
  uint8_t* pools[kMaxTreePools];
  int64_t num_pages[kMaxTreePools];
  int64_t page_bytes;
  int32_t pieces;  // 16-byte pieces of a token
  int32_t batch;
  const int32_t* cu_q_rows;
  const int32_t* seq_lens;
  const int32_t* block_table;
  int32_t max_pages;
  const int32_t* path;
  int64_t path_stride;
  const int32_t* path_lens;
  int32_t* status;
};
cudaError_t launch_tree_move(int layout, int dtype, int n_pools, const TreeMoveArgs& a, cudaStream_t st);
cudaError_t launch_bw_probe(const void* buf, int64_t chunks, int32_t* status, cudaStream_t st);
cudaError_t launch_bw_probe_tma(const void* buf, int64_t pages, int32_t* status, cudaStream_t st);
cudaError_t launch_wait_selftest(int32_t* status, int32_t* result, int64_t limit_ns, cudaStream_t st);
// TMA descriptor of a LOCAL pool: rows of 256 elements in 128-byte chunks
// (4 chunks of 64 bf16, or 2 chunks of 128 e4m3); row = ((page * kv_heads +
// head) * 2 + {K, V}) * 16 + token; box {one chunk, 1, 16 rows}, 128-byte
// swizzle.
constexpr int kPageTokens = 16;
// Tensor map of a LOCAL pool: boxes of one 128-byte chunk of `box_rows` rows
// (16: a page head's K or V; 32: its K and V together), 128-byte swizzled.
cudaError_t make_local_kv_map(const LocalArgs& a, CUtensorMap* map, int dtype = GW_KV_BF16, int box_rows = 16);
cudaError_t launch_local_decode(int dtype, int group, const LocalArgs& a, cudaStream_t st);
// tcgen05 decode kernel (kind::f8f6f4) for e4m3 LOCAL pools, plus the combine
cudaError_t launch_local_decode_e4m3_tc(int group, const LocalArgs& a, cudaStream_t st);
cudaError_t launch_global_decode(int layout, const LocalArgs& a, cudaStream_t st);
cudaError_t launch_local_prompt(int dtype, int group, const LocalArgs& a, int max_q_rows, cudaStream_t st);
// tcgen05 prompt-row kernel for local layers (bf16 or e4m3 pools); expects
// a.prompt_base planned with 128 / group queries per tile
cudaError_t launch_local_prompt_tc(int dtype, int group, const LocalArgs& a, cudaStream_t st);
// tcgen05 prompt-row kernel for global layers; expects a.prompt_base planned
// with 2 tiles (output-dim halves) per block of 128 / num_q_heads queries
cudaError_t launch_global_prompt_tc(int layout, const LocalArgs& a, cudaStream_t st);
cudaError_t launch_global_prompt(int layout, const LocalArgs& a, int max_q_rows, cudaStream_t st);

}  // namespace gw
