// Attention of drafted trees: launchers, and the merge of the chunks of long
// sequences.  The attention kernels are attn_tree_local.cu and
// attn_tree_local_rows.cu (local layers), attn_tree_global.cu and
// attn_tree_global_rows.cu (global layers); all write the rows of single-chunk
// sequences themselves.
//
// The rows of a sequence (n <= 64) times its heads are a matrix product's rows,
// but the cache is long, so the work is split along it: a unit's result is the
// unnormalised row and its (m, l), base 2, and
//   o = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c,  M = max_c m_c.
#include "common.cuh"

namespace gw {
namespace {

// A warp merges 8 of the 256 dims of 32 rows of a unit, a lane a row: parts lie as
// [unit][8-column block 32][row][8], so that what a warp stores or reads at a time
// is 1 KB in one piece.  The rows' weights are put in shared memory first.  Every
// fourth chunk has a sum of its own and the four are added in a fixed order, so that
// a row depends neither on its companions nor on kSplit: 4, a warp to each sum, where
// the warps of kSplit = 1 would be few.  kLocal: units are (KV head, chunk, row
// block), else (chunk, row block, half of the dims).
//
// 8 x 131072 tokens, 8 heads, 4 drafts (512 warps with kSplit = 1, 76 chunks): the
// call 221 us with 4 and 237 with 1 (254 at a step when 262 with (m, l) read chunk by
// chunk); 4 x 131072, full layout, 167 and 174.  16 sequences of 512 to 8192 tokens,
// 16 drafts, 32 heads (16384 warps, up to 8 chunks): 194 and 140.
template <int kSplit>
struct Merge {
  static constexpr int kWarps = kSplit == 1 ? 4 : 8;
  static constexpr int kCols = kWarps / kSplit;  // 8-column blocks of a block
};

__device__ __forceinline__ void load_f32x8(const float* p, float (&x)[8]) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
               : "l"(p));
}

template <bool kLocal, int kSplit>
__global__ void __launch_bounds__(Merge<kSplit>::kWarps * 32, kSplit == 1 ? 1 : 2)
    tree_merge_kernel(const LocalArgs a, int group, int copies, int blocks, const TreeRule rule, int scale) {
  constexpr int kMergeWarps = Merge<kSplit>::kWarps, kMergeCols = Merge<kSplit>::kCols;
  __shared__ float w[kTreeMaxChunks][32], wl[kTreeMaxChunks][32];
  __shared__ float top[kMergeWarps][32], sums[kSplit == 1 ? 1 : kMergeWarps][8][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = (a.part_rows + 31) / 32;  // of 32 rows, in a unit
  int task = blockIdx.x;
  const int c8 = task % (32 / kMergeCols) * kMergeCols + warp / kSplit;
  task /= 32 / kMergeCols;
  const int pg = task % groups;
  task /= groups;
  const int qb = task % blocks;
  task /= blocks;
  const int copy = task % copies;  // KV head or half
  const int s = task / copies;
  const int row0 = a.cu_q_rows[s], n = a.cu_q_rows[s + 1] - row0, L = a.seq_lens[s];
  const int64_t ub = static_cast<int64_t>(a.unit_base[s]) * scale;  // `scale` parts a unit
  if (ub < 0) return;
  const TreeSpan sp = tree_span(L, n, a.window, rule);
  const int nc = sp.chunks();
  if (nc == 1 || qb >= sp.blocks) return;  // the attention kernel has written it
  const int place = pg * 32 + lane, q = qb * rule.per + place / group;
  const bool ok = place < a.part_rows && q < n;
  const int64_t u0 = ub + (kLocal ? copy * nc * sp.blocks + qb : qb * 2 + copy);
  const int64_t step = (kLocal ? sp.blocks : 2 * sp.blocks) * static_cast<int64_t>(a.part_rows);
  const float2* ml = a.part_ml + u0 * a.part_rows + place;
  // a warp takes every kMergeWarps-th chunk's (m, l), all its loads in flight at once
  constexpr int kMine = (kTreeMaxChunks + kMergeWarps - 1) / kMergeWarps;
  float2 mine[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int c = warp + kMergeWarps * i;
    if (kMergeWarps * i >= nc) break;
    mine[i] = ok && c < nc ? ml[c * step] : make_float2(-INFINITY, 0.f);
  }
  float M = -INFINITY;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    if (kMergeWarps * i >= nc) break;
    M = fmaxf(M, mine[i].x);
  }
  top[warp][lane] = M;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kMergeWarps; ++k) M = fmaxf(M, top[k][lane]);
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int c = warp + kMergeWarps * i;
    if (c >= nc) break;
    const float x = M == -INFINITY ? 0.f : ex2(mine[i].x - M);
    w[c][lane] = x;
    wl[c][lane] = x * mine[i].y;
  }
  __syncthreads();
  float den = 0.f;
#pragma unroll 4
  for (int c = 0; c < nc; ++c) den += wl[c][lane];
  const float inv = den == 0.f ? 0.f : 1.f / den;  // NaN where a chunk's sum is
  constexpr int kMine4 = 4 / kSplit;  // of the four sums
  float acc[kMine4][8];
#pragma unroll
  for (int i = 0; i < kMine4; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[i][k] = 0.f;
  if (ok) {
    const float* po = a.part_o + ((u0 * 32 + c8) * a.part_rows + place) * 8;
    auto add = [&](int c, float (&to)[8]) {
      float x[8];
      load_f32x8(po + c * step * 256, x);
#pragma unroll
      for (int k = 0; k < 8; ++k) to[k] = fmaf(w[c][lane], x[k], to[k]);
    };
    if constexpr (kSplit == 1) {
      int c = 0;
#pragma unroll 4
      for (; c + 4 <= nc; c += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) add(c + i, acc[i]);
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (c + i < nc) add(c + i, acc[i]);
    } else {
#pragma unroll 8
      for (int c = warp % 4; c < nc; c += 4) add(c, acc[0]);
    }
  }
  float sum[8];
  if constexpr (kSplit == 1) {
    if (!ok) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] = (acc[0][k] + acc[1][k]) + (acc[2][k] + acc[3][k]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) sums[warp][k][lane] = acc[0][k];
    __syncthreads();
    if (!ok || warp % 4) return;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      sum[k] = (acc[0][k] + sums[warp + 1][k][lane]) + (sums[warp + 2][k][lane] + sums[warp + 3][k][lane]);
  }
  const int head = kLocal ? copy * group + place % group : place % group;
  uint16_t* dst = a.out + ((static_cast<int64_t>(row0) + q) * a.num_q_heads + head) * (kLocal ? 256 : 512) +
                  (kLocal ? 0 : 256 * copy);
  uint32_t pk[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    __nv_bfloat162 b = __floats2bfloat162_rn(sum[2 * k] * inv, sum[2 * k + 1] * inv);
    pk[k] = *reinterpret_cast<uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(dst + 8 * c8) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
}

template <bool kLocal, int kSplit>
cudaError_t launch_merge_split(const LocalArgs& a, int group, int copies, int blocks, int64_t columns,
                               const TreeRule& rule, int scale, cudaStream_t st) {
  using M = Merge<kSplit>;
  return launch_pdl(tree_merge_kernel<kLocal, kSplit>, dim3(static_cast<unsigned>(columns / M::kCols)),
                    dim3(M::kWarps * 32), 0, st, a, group, copies, blocks, rule, scale);
}

template <bool kLocal>
cudaError_t launch_merge(const LocalArgs& a, int group, const TreeRule& rule, int scale, cudaStream_t st) {
  const int copies = kLocal ? a.kv_heads : 2, blocks = (a.max_q_rows + rule.per - 1) / rule.per;
  // column blocks of 32 rows in the call: split where they are fewer than about 27 an SM
  const int64_t columns = static_cast<int64_t>(a.batch) * copies * blocks * ((a.part_rows + 31) / 32) * 32;
  return columns < 4096 ? launch_merge_split<kLocal, 4>(a, group, copies, blocks, columns, rule, scale, st)
                        : launch_merge_split<kLocal, 1>(a, group, copies, blocks, columns, rule, scale, st);
}

}  // namespace

// Up to 32 rows x heads (64 on bf16 global layers) lie along the products' N, more
// along M.  Local, 16 sequences of 512 to 8192 tokens, 16 KV heads of 2 heads, bf16:
// 16 drafts 49 us (along M 55), 33 drafts 55.0 (along N, in blocks of 32 rows,
// 100.6); 61 e4m3 sequences, 7 drafts 91 us (177).  Global, 8 x 131072 tokens, 8
// heads: 4 drafts 222 us (along M 389), 8 drafts 314 (381); 1 x 8192, 8 drafts 32
// (36); 2 sequences of 37 and 100 tokens, full layout, 5 drafts 11.8 (11.0).  The
// rule is the call's bound, so that a captured call stays what it is.
//
// The merge is left out where the block table's width allows one chunk only.
cudaError_t launch_local_tree(int dtype, int group, const LocalArgs& a, cudaStream_t st) {
  const TreeRule rule = tree_rule_local(group);
  cudaError_t e = a.max_q_rows * group <= tree_few_rows(GW_LAYOUT_LOCAL) ? launch_local_tree_few(dtype, group, a, st)
                                                       : launch_local_tree_rows(dtype, group, a, st);
  if (e != cudaSuccess || tree_max_chunks(a.max_pages, a.max_q_rows, a.window, rule) == 1) return e;
  return launch_merge<true>(a, group, rule, 1, st);
}

cudaError_t launch_global_tree(int layout, const LocalArgs& a, cudaStream_t st) {
  const bool few = a.max_q_rows * a.num_q_heads <= tree_few_rows(layout);
  const TreeRule rule = few ? tree_rule_few(a.num_q_heads) : tree_rule_global(a.num_q_heads);
  cudaError_t e = few ? launch_global_tree_few(layout, a, st) : launch_global_tree_rows(layout, a, st);
  if (e != cudaSuccess || tree_max_chunks(a.max_pages, a.max_q_rows, a.window, rule) == 1) return e;
  return launch_merge<false>(a, a.num_q_heads, rule, few ? 2 : 1, st);
}

}  // namespace gw
