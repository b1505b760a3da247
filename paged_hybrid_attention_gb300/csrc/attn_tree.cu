// Attention of drafted trees: launchers, and the merge of the chunks of long
// sequences.  The attention kernels are attn_prompt_tc.cu (local layers) and
// attn_tree_global.cu (global layers); both write rows of single-chunk
// sequences themselves.
//
// The rows of a sequence (n <= 64) times its heads are a matrix product's rows,
// but the cache is long, so the work is split along it: a unit's result is the
// unnormalised row and its (m, l), base 2, and
//   o = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c,  M = max_c m_c.
#include "common.cuh"

namespace gw {
namespace {

// A warp merges 256 dims of one (row, head); a lane owns 8 dims, and lanes
// fetch the chunks' (m, l) two each (kTreeMaxChunks).  Chunks are added in
// order, so a row does not depend on its companions.  kLocal: units are (KV
// head, chunk, row block), else (chunk, row block, half of the dims).
template <bool kLocal>
__global__ void __launch_bounds__(256) tree_merge_kernel(const LocalArgs a, int group) {
  constexpr int kSlices = kLocal ? 1 : 2;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int slice = static_cast<int>(task % kSlices);
  const int h = static_cast<int>(task / kSlices % a.num_q_heads);
  const int64_t sr = task / kSlices / a.num_q_heads;
  const int r = static_cast<int>(sr % a.max_q_rows);
  const int s = static_cast<int>(sr / a.max_q_rows);
  if (s >= a.batch) return;
  const int row0 = a.cu_q_rows[s], n = a.cu_q_rows[s + 1] - row0, L = a.seq_lens[s];
  const int ub = a.unit_base[s], units = a.unit_base[s + 1] - ub;
  if (r >= n || units == 0) return;
  const TreeSpan sp = tree_span(L, n, a.window, group, kLocal ? kTreeLocalTiles : kTreeGlobalTiles);
  const int nc = sp.chunks();
  if (nc == 1) return;  // the attention kernel has written it
  const int per = 128 / group, cap = min(per, a.max_q_rows);
  const int qb = r / per, q = r - qb * per;
  // unit of chunk c: u0 + c * ustep; the row's place in a unit
  const int64_t u0 = ub + (kLocal ? h / group * nc * sp.blocks + qb : qb * 2 + slice);
  const int ustep = kLocal ? sp.blocks : 2 * sp.blocks;
  const int place = kLocal ? h % group * cap + q : q * group + h;
  const int64_t first = u0 * a.part_rows + place, step = static_cast<int64_t>(ustep) * a.part_rows;
  float2 ml[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = lane + 32 * k;
    ml[k] = c < nc ? a.part_ml[first + c * step] : make_float2(-INFINITY, 0.f);
  }
  float M = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float w[2], den = 0.f;
#pragma unroll
  for (int k = 0; k < 2; ++k) w[k] = M == -INFINITY ? 0.f : ex2(ml[k].x - M);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const float* po = a.part_o + first * 256 + lane * 8;
#pragma unroll 8
  for (int c = 0; c < nc; ++c) {
    const float4 x = *reinterpret_cast<const float4*>(po + c * step * 256);
    const float4 y = *reinterpret_cast<const float4*>(po + c * step * 256 + 4);
    const float wc = __shfl_sync(0xffffffffu, c < 32 ? w[0] : w[1], c & 31);
    const float lc = __shfl_sync(0xffffffffu, c < 32 ? ml[0].y : ml[1].y, c & 31);
    den = fmaf(wc, lc, den);
    acc[0] = fmaf(wc, x.x, acc[0]);
    acc[1] = fmaf(wc, x.y, acc[1]);
    acc[2] = fmaf(wc, x.z, acc[2]);
    acc[3] = fmaf(wc, x.w, acc[3]);
    acc[4] = fmaf(wc, y.x, acc[4]);
    acc[5] = fmaf(wc, y.y, acc[5]);
    acc[6] = fmaf(wc, y.z, acc[6]);
    acc[7] = fmaf(wc, y.w, acc[7]);
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  uint32_t pk[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 b = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    pk[i] = *reinterpret_cast<uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(a.out + ((static_cast<int64_t>(row0) + r) * a.num_q_heads + h) * (256 * kSlices) +
                            256 * slice + 8 * lane) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
}

template <bool kLocal>
cudaError_t launch_merge(const LocalArgs& a, int group, cudaStream_t st) {
  const int64_t warps = static_cast<int64_t>(a.batch) * a.max_q_rows * a.num_q_heads * (kLocal ? 1 : 2);
  return launch_pdl(tree_merge_kernel<kLocal>, dim3(static_cast<unsigned>((warps + 7) / 8)), dim3(256), 0, st, a, group);
}

}  // namespace

// The merge is left out where the block table's width allows one chunk only.
cudaError_t launch_local_tree(int dtype, int group, const LocalArgs& a, cudaStream_t st) {
  cudaError_t e = launch_local_tree_tc(dtype, group, a, st);
  if (e != cudaSuccess || tree_max_chunks(a.max_pages, a.max_q_rows, a.window, kTreeLocalTiles) == 1) return e;
  return launch_merge<true>(a, group, st);
}

cudaError_t launch_global_tree(int layout, const LocalArgs& a, cudaStream_t st) {
  cudaError_t e = launch_global_tree_tc(layout, a, st);
  if (e != cudaSuccess || tree_max_chunks(a.max_pages, a.max_q_rows, a.window, kTreeGlobalTiles) == 1) return e;
  return launch_merge<false>(a, a.num_q_heads, st);
}

}  // namespace gw
