// The split-KV plan of a decode call, computed inside the decode kernels.
//
// Every CTA scans the batch's lengths into its own shared memory (a few
// hundred nanoseconds for serving batches), so no plan kernel and no work
// counter sit in front of the decode.  Units are dealt round-robin over the
// CTAs (or warps), so the plan is all a CTA needs to find its own work.
#pragma once

#include "common.cuh"

namespace gw {

__device__ __forceinline__ bool plan_len_ok(const LocalArgs& a, int L) {
  return L >= 1 && static_cast<int64_t>(L) <= static_cast<int64_t>(a.max_pages) * kPage;
}

// ub[s] = units of the sequences before s (ub[batch] = total), with count(s)
// the units of sequence s.  Must be called by every thread of the block;
// scratch holds 32 ints.
template <class CountOf>
__device__ __forceinline__ void plan_scan(int batch, int32_t* ub, int32_t* scratch, CountOf count) {
  const int nt = blockDim.x, t = threadIdx.x;
  const int per = (batch + nt - 1) / nt;
  const int s0 = min(batch, t * per), s1 = min(batch, s0 + per);
  int mine = 0;
  for (int s = s0; s < s1; ++s) {
    const int units = count(s);
    ub[s] = units;  // per-sequence count for now
    mine += units;
  }
  // exclusive scan of the per-thread sums
  const int lane = t & 31, w = t >> 5;
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[w] = x;
  __syncthreads();
  if (w == 0) {
    int v = lane < (nt >> 5) ? scratch[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane < (nt >> 5)) scratch[lane] = v;
  }
  __syncthreads();
  int run = (w > 0 ? scratch[w - 1] : 0) + x - mine;
  for (int s = s0; s < s1; ++s) {
    const int c = ub[s];
    ub[s] = run;
    run += c;
  }
  if (t == nt - 1) ub[batch] = run;
  __syncthreads();
}

// The plan of a decode call: plan_scan over the decode-row sequences, with
// units_of(L) the units of one decode row of length L.  Rows of invalid length
// (L < 1 or beyond the block table) get no units.  With `publish`, CTA 0
// also stores the plan to the workspace for the combine kernel and raises
// GW_DEV_LEN_RANGE for invalid rows; without it (a plan made before the wait
// on the previous kernel) nothing is written to global memory, and
// publish_plan does both once the wait is over.
template <class UnitsOf>
__device__ void plan_in_smem(const LocalArgs& a, int32_t* ub, int32_t* scratch, UnitsOf units_of,
                             bool publish = true) {
  plan_scan(a.batch, ub, scratch, [&](int s) {
    const int n = a.cu_q_rows[s + 1] - a.cu_q_rows[s];
    const int L = a.seq_lens[s];
    if (n != 1) return 0;
    if (plan_len_ok(a, L)) return units_of(L);
    if (blockIdx.x == 0 && publish) set_status(a.status, GW_DEV_LEN_RANGE);
    return 0;
  });
  if (blockIdx.x == 0 && publish)
    for (int s = threadIdx.x; s <= a.batch; s += blockDim.x) a.unit_base[s] = ub[s];
}

// The plan of a gw_tree_attn_* call.
struct TreePlan {
  int32_t ub[kMaxTreeBatch + 1];  // units of the sequences before place p
  int32_t scratch[32];
  int16_t seq[kMaxTreeBatch];  // the sequence at place p
};

// A sequence's units are `copies` (KV heads, or halves of the output dims) x blocks
// of rows x chunks.  Sequences stand in the order of their chunks' lengths, the
// longest first, and units are dealt in rounds that run to and fro (tree_unit), so
// that CTAs get about the same (16 sequences of 512 to 8192 tokens, 16 drafts, a
// global layer: 138 -> 126 us).  Sequences without rows have no units; nor have
// those with more rows than max_q_rows, a length below their rows or beyond the
// block table (GW_DEV_LEN_RANGE), whose output rows become zeros here.  CTA 0
// stores each sequence's first unit (-1: none) for the merge.
__device__ __forceinline__ void plan_tree(const LocalArgs& a, TreePlan& plan, int copies, const TreeRule& rule,
                                          int head_dim) {
  constexpr int kPer = 2;  // sequences of a thread: at least 128 threads
  const int t = threadIdx.x, nt = blockDim.x;
  int tiles[kPer], units[kPer], rank[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = t + i * nt;
    tiles[i] = units[i] = 0;
    if (s >= a.batch) continue;
    const int n = a.cu_q_rows[s + 1] - a.cu_q_rows[s], L = a.seq_lens[s];
    if (n >= 1 && n <= a.max_q_rows && L >= n && plan_len_ok(a, L)) {
      const TreeSpan sp = tree_span(L, n, a.window, rule);
      tiles[i] = sp.ct;
      units[i] = copies * sp.blocks * sp.chunks();
    }
    plan.ub[s] = tiles[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = t + i * nt;
    rank[i] = 0;
    if (s < a.batch)
      for (int o = 0; o < a.batch; ++o) {
        const int k = plan.ub[o];
        rank[i] += k > tiles[i] || (k == tiles[i] && o < s);
      }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = t + i * nt;
    if (s >= a.batch) continue;
    plan.seq[rank[i]] = static_cast<int16_t>(s);
    plan.ub[rank[i]] = units[i];
  }
  __syncthreads();
  plan_scan(a.batch, plan.ub, plan.scratch, [&](int p) { return plan.ub[p]; });
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = t + i * nt;
    if (s < a.batch && blockIdx.x == 0) a.unit_base[s] = units[i] ? plan.ub[rank[i]] : -1;
  }
  // places without units are the last ones
  for (int p = a.batch - 1 - blockIdx.x; p >= 0 && plan.ub[p + 1] == plan.ub[p]; p -= gridDim.x) {
    const int s = plan.seq[p], n = a.cu_q_rows[s + 1] - a.cu_q_rows[s];
    if (n == 0) continue;
    if (t == 0) set_status(a.status, GW_DEV_LEN_RANGE);
    uint4* row = reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(a.cu_q_rows[s]) * a.num_q_heads * head_dim);
    const int64_t pieces = static_cast<int64_t>(n) * a.num_q_heads * head_dim / 8;
    for (int64_t i = t; i < pieces; i += nt) row[i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// The unit that this CTA takes in round k: rounds run to and fro over the CTAs.
__device__ __forceinline__ int tree_unit(int k) {
  const int b = blockIdx.x, g = gridDim.x;
  return k * g + (k & 1 ? g - 1 - b : b);
}

// The keys of a tree's row: cached tokens [kmin, base) and the drafts of
// `drafts`, bit i of which is token base + i; and what its logits are scaled by
// (q's scaling undone, on e4m3 pools).
struct TreeRow {
  uint64_t drafts;
  int kmin;
  float scale;
};

// Row r of sequence s (n rows at tokens [base, base + n), first row row0); one
// at a position before the drafts' first sees nothing (GW_DEV_POS_RANGE).
// `windowed`: tokens at positions up to pos - window are not seen, drafts by
// their own positions.
__device__ __forceinline__ TreeRow tree_row(const LocalArgs& a, int row0, int r, int n, int base, bool windowed) {
  TreeRow t;
  t.kmin = 0;
  t.scale = 1.f;
  t.drafts = a.tree_mask[row0 + r] & (n < 64 ? (1ull << n) - 1 : ~0ull);
  if (windowed) {
    const int pos = a.tree_pos[row0 + r];
    if (pos < base) {
      set_status(a.status, GW_DEV_POS_RANGE);
      t.kmin = 0x7fffffff;
      t.drafts = 0;
      return t;
    }
    t.kmin = max(0, pos - a.window + 1);
    if (t.kmin > base)  // else no draft is as far back
      for (int i = 0; i < n; ++i)
        if (a.tree_pos[row0 + i] < t.kmin) t.drafts &= ~(1ull << i);
  }
  return t;
}

// The keys of tile [key0, key0 + 64) that the row sees, a bit each.
__device__ __forceinline__ uint64_t tree_tile_mask(const TreeRow& t, int base, int key0) {
  const int lo = t.kmin - key0, hi = min(64, base - key0);  // cached: bits [lo, hi)
  uint64_t m = 0;
  if (hi > 0 && lo < hi) m = (hi < 64 ? (1ull << hi) - 1 : ~0ull) & (lo > 0 ? ~0ull << lo : ~0ull);
  const int d = base - key0;  // the first draft's bit
  if (d >= 0 && d < 64) m |= t.drafts << d;
  if (d < 0 && d > -64) m |= t.drafts >> -d;
  return m;
}

// The global half of a plan made with publish = false, once the previous
// kernel has finished: CTA 0's threads t of nt store the plan and raise
// GW_DEV_LEN_RANGE for invalid decode rows.
__device__ __forceinline__ void publish_plan(const LocalArgs& a, const int32_t* ub, int t, int nt) {
  if (blockIdx.x != 0) return;
  for (int s = t; s <= a.batch; s += nt) {
    a.unit_base[s] = ub[s];
    if (s < a.batch && a.cu_q_rows[s + 1] - a.cu_q_rows[s] == 1 && !plan_len_ok(a, a.seq_lens[s]))
      set_status(a.status, GW_DEV_LEN_RANGE);
  }
}

// The sequence that owns unit u (0 <= u < ub[batch]): the largest s with
// ub[s] <= u, which skips sequences without units.
__device__ __forceinline__ int plan_seq(const int32_t* ub, int batch, int u) {
  int lo = 0, hi = batch;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (ub[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

}  // namespace gw
