// gw_tree_accept and gw_kv_tree_move: the path of drafted tokens that the
// target has chosen, and the move of its rows to the front of the drafts.
#include "common.cuh"

namespace gw {
namespace {

// One warp per sequence, two rows of its tree per lane.  From the root on, the
// next row of the path is the lowest child whose draft is what the target chose
// after the present one: a ballot over the lanes' rows finds it.  At most 64
// steps of two ballots and a shuffle; a call is one launch and the latency of
// three dependent loads.
constexpr int kAcceptWarps = 4;

__global__ void __launch_bounds__(kAcceptWarps * 32) tree_accept_kernel(const TreeAcceptArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x * kAcceptWarps + (threadIdx.x >> 5);
  if (b >= a.batch) return;
  const int row0 = a.cu_q_rows[b], n = a.cu_q_rows[b + 1] - row0, L = a.seq_lens[b];
  if (n <= 0 || n > a.max_q_rows || L < n) {
    if (lane == 0) {
      if (n != 0 || L < 0) set_status(a.status, GW_DEV_LEN_RANGE);
      a.path_lens[b] = 0;
      if (a.new_lens) a.new_lens[b] = L;
    }
    return;
  }
  int parent[2], draft[2], target[2];
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    parent[k] = -1;
    draft[k] = target[k] = 0;
    if (i < n) {
      draft[k] = a.draft[row0 + i];
      target[k] = a.target[row0 + i];
      if (i > 0) {  // the root's own entry is not read
        parent[k] = a.parent[row0 + i];
        if (parent[k] < 0 || parent[k] >= i) {
          parent[k] = -1;
          bad = true;
        }
      }
    }
  }
  if (bad) set_status(a.status, GW_DEV_TREE_RANGE);
  int32_t* path = a.path + b * a.path_stride;
  int at = 0, steps = 0, want;
  while (true) {
    if (lane == 0) path[steps] = at;
    ++steps;
    want = __shfl_sync(0xffffffffu, at < 32 ? target[0] : target[1], at & 31);
    const uint32_t lo = __ballot_sync(0xffffffffu, parent[0] == at && draft[0] == want);
    const uint32_t hi = __ballot_sync(0xffffffffu, parent[1] == at && draft[1] == want);
    if (!(lo | hi)) break;
    at = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);  // above its parent, so the walk ends
  }
  if (lane == 0) {
    a.path_lens[b] = steps;
    if (a.next_tokens) a.next_tokens[b] = want;
    if (a.new_lens) a.new_lens[b] = L - n + steps;
  }
}

// Where the 16-byte piece `u` of token o of a page lies, in bytes of the page.
//   local   [kv head][K, V][16][256]: kPieces per (head, K or V) row
//   global  [token block 2][column block][8][16 bytes]
template <int LAYOUT, int DT>
__device__ __forceinline__ int64_t piece_at(int u, int o) {
  if constexpr (LAYOUT == GW_LAYOUT_LOCAL) {
    constexpr int kPieces = DT == GW_KV_BF16 ? 32 : 16;
    return (static_cast<int64_t>(u / kPieces) * kPage + o) * (kPieces * 16) + (u % kPieces) * 16;
  } else {
    constexpr int kBlk = LAYOUT == GW_LAYOUT_GLOBAL_FOLDED ? 80 : LAYOUT == GW_LAYOUT_GLOBAL_FULL ? 128 : 40;
    return ((static_cast<int64_t>(o / 8) * kBlk + u) * 8 + o % 8) * 16;
  }
}

// Block (x, y, z): 256 pieces of the rows of sequence y in pool z.  The path's
// places are looked up once per block; then a thread takes its piece of up to
// kMoveRows rows into registers and writes them, from the path's front.  Row i
// comes from a draft at or behind i, so what a thread has yet to read lies
// behind what it has written, and no two threads share a piece.  40 pools of 16 KV
// heads, 16 sequences, paths of 5: 13 us in a graph with the acceptance before it,
// the rows' bytes 12.
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 8;

template <int LAYOUT, int DT>
__global__ void __launch_bounds__(kMoveThreads) tree_move_kernel(const TreeMoveArgs a) {
  __shared__ int32_t src_page[kMaxTreeRows], dst_page[kMaxTreeRows];
  __shared__ uint8_t src_off[kMaxTreeRows], dst_off[kMaxTreeRows];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, b = blockIdx.y;
  const bool report = blockIdx.x == 0 && blockIdx.z == 0;
  const int n = a.cu_q_rows[b + 1] - a.cu_q_rows[b], L = a.seq_lens[b], m = a.path_lens[b];
  if (n < 0 || n > kMaxTreeRows || L < n || L > static_cast<int64_t>(a.max_pages) * kPage) {
    if (report && tid == 0) set_status(a.status, GW_DEV_LEN_RANGE);
    return;
  }
  if (m < 0 || m > n || m > a.path_stride) {
    if (report && tid == 0) set_status(a.status, GW_DEV_TREE_RANGE);
    return;
  }
  const int64_t pages = a.num_pages[blockIdx.z];
  if (tid < m) {
    const int32_t* path = a.path + b * a.path_stride;
    const int at = path[tid], before = tid > 0 ? path[tid - 1] : -1;
    int32_t sp = -1, dp = -1;
    if (at < tid || at >= n || at <= before) {
      if (report) set_status(a.status, GW_DEV_TREE_RANGE);
    } else if (at != tid) {
      const int s = L - n + at, d = L - n + tid;
      const int32_t* table = a.block_table + static_cast<int64_t>(b) * a.max_pages;
      sp = table[s / kPage];
      dp = table[d / kPage];
      src_off[tid] = s % kPage;
      dst_off[tid] = d % kPage;
      if (sp < 0 || sp >= pages || dp < 0 || dp >= pages) {
        if (blockIdx.x == 0) set_status(a.status, GW_DEV_PAGE_RANGE);
        sp = -1;
      }
    }
    src_page[tid] = sp;
    dst_page[tid] = dp;
  }
  __syncthreads();
  const int u = blockIdx.x * kMoveThreads + tid;
  if (u >= a.pieces) return;
  uint8_t* pool = a.pools[blockIdx.z];
  for (int i0 = 0; i0 < m; i0 += kMoveRows) {
    uint4 x[kMoveRows];
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i)
      if (i0 + i < m && src_page[i0 + i] >= 0)
        x[i] = *reinterpret_cast<const uint4*>(pool + src_page[i0 + i] * a.page_bytes +
                                               piece_at<LAYOUT, DT>(u, src_off[i0 + i]));
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i)
      if (i0 + i < m && src_page[i0 + i] >= 0)
        *reinterpret_cast<uint4*>(pool + dst_page[i0 + i] * a.page_bytes + piece_at<LAYOUT, DT>(u, dst_off[i0 + i])) =
            x[i];
  }
}

}  // namespace

cudaError_t launch_tree_accept(const TreeAcceptArgs& a, cudaStream_t st) {
  return launch_pdl(tree_accept_kernel, dim3((a.batch + kAcceptWarps - 1) / kAcceptWarps), dim3(kAcceptWarps * 32), 0,
                    st, a);
}

cudaError_t launch_tree_move(int layout, int dtype, int n_pools, const TreeMoveArgs& a, cudaStream_t st) {
  const dim3 grid((a.pieces + kMoveThreads - 1) / kMoveThreads, a.batch, n_pools), block(kMoveThreads);
  if (layout == GW_LAYOUT_LOCAL)
    return dtype == GW_KV_BF16 ? launch_pdl(tree_move_kernel<GW_LAYOUT_LOCAL, GW_KV_BF16>, grid, block, 0, st, a)
                               : launch_pdl(tree_move_kernel<GW_LAYOUT_LOCAL, GW_KV_E4M3>, grid, block, 0, st, a);
  if (layout == GW_LAYOUT_GLOBAL_FOLDED)
    return launch_pdl(tree_move_kernel<GW_LAYOUT_GLOBAL_FOLDED, GW_KV_BF16>, grid, block, 0, st, a);
  if (layout == GW_LAYOUT_GLOBAL_FULL)
    return launch_pdl(tree_move_kernel<GW_LAYOUT_GLOBAL_FULL, GW_KV_BF16>, grid, block, 0, st, a);
  return launch_pdl(tree_move_kernel<GW_LAYOUT_GLOBAL_FOLDED_E4M3, GW_KV_E4M3>, grid, block, 0, st, a);
}

}  // namespace gw
