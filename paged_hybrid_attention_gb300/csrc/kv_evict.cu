// gw_kv_evict_select and gw_kv_evict_compact: a sequence of the global cache
// cut to the tokens that have drawn the most attention.
#include "common.cuh"

namespace gw {
namespace {

// ---- select -------------------------------------------------------------------
// The weights' order as unsigned integers: larger weight, larger key; -0 and
// 0 share a key, and every NaN has key 0, below -inf.
__device__ __forceinline__ uint32_t order_key(float w) {
  uint32_t u = __float_as_uint(w);
  if (w != w) return 0;
  if (w == 0.f) u = 0;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr int kSelThreads = 1024;

// Exclusive sum of v over the block's threads in thread order; `total`
// receives the sum.  `scratch`: 33 values.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* scratch, uint64_t& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the previous call's reads of scratch are done
  if (lane == 31) scratch[w] = x;
  __syncthreads();
  if (w == 0) {
    uint64_t s = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    scratch[lane] = s;
  }
  __syncthreads();
  total = scratch[31];
  return (w > 0 ? scratch[w - 1] : 0) + x - v;
}

// One block per sequence.  The k-th largest key of the middle is found digit
// by digit from the top (four passes of 8 bits), then one pass in token order
// writes the kept indices.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const SelectArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint64_t scratch[32];
  __shared__ uint32_t found[2];  // digit, keys above it within the prefix
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, tid = threadIdx.x;
  const int L = a.seq_lens[b];
  int32_t* keep = a.keep_idx + b * a.keep_stride;
  if (L < 0 || L > a.acc_stride) {
    if (tid == 0) {
      set_status(a.status, GW_DEV_LEN_RANGE);
      a.keep_lens[b] = 0;
    }
    return;
  }
  if (tid == 0) a.keep_lens[b] = min(L, a.budget);
  if (L <= a.budget) {
    for (int j = tid; j < L; j += kSelThreads) keep[j] = j;
    return;
  }
  const float* acc = a.acc + b * a.acc_stride;
  const int lo = a.sinks, hi = L - a.recent;
  uint32_t need = a.budget - a.sinks - a.recent;  // of the middle
  const bool any = need > 0;
  uint32_t prefix = 0, mask = 0;
  for (int shift = 24; any && shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int j = lo + tid; j < hi; j += kSelThreads) {
      const uint32_t key = order_key(acc[j]);
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1u);
    }
    __syncthreads();
    // thread t < 256: keys of digit 255 - t and above
    uint64_t total;
    const uint32_t mine = tid < 256 ? hist[255 - tid] : 0;
    const uint32_t above = static_cast<uint32_t>(block_scan(mine, scratch, total));
    if (tid < 256 && above < need && above + mine >= need) {
      found[0] = 255 - tid;
      found[1] = above;
    }
    __syncthreads();
    prefix |= found[0] << shift;
    mask |= 255u << shift;
    need -= found[1];
    __syncthreads();
  }
  // keep all above `prefix`, and the first `need` equal to it
  uint32_t sure = 0, ties = 0;  // so far
  for (int j0 = 0; j0 < L; j0 += kSelThreads) {
    const int j = j0 + tid;
    uint32_t is_sure = 0, is_tie = 0;
    if (j < L) {
      if (j < lo || j >= hi) {
        is_sure = 1;
      } else if (any) {
        const uint32_t key = order_key(acc[j]);
        is_sure = key > prefix;
        is_tie = key == prefix;
      }
    }
    uint64_t total;
    const uint64_t before = block_scan((static_cast<uint64_t>(is_sure) << 32) | is_tie, scratch, total);
    const uint32_t ties_before = ties + static_cast<uint32_t>(before);
    if (is_sure || (is_tie && ties_before < need))
      keep[sure + static_cast<uint32_t>(before >> 32) + min(ties_before, need)] = j;
    sure += static_cast<uint32_t>(total >> 32);
    ties += static_cast<uint32_t>(total);
  }
}

// ---- compact ------------------------------------------------------------------
// Token i's row takes token keep[i]'s place, keep[i] >= i.  A block walks one
// 16-byte column block of the sequence's rows in token order, in steps of
// kMoveThreads rows: a step reads its rows, all of them before it writes any
// (the barrier), and no later step reads what it writes, since later steps'
// sources lie at or behind their own first token.  So the move is exact in
// place, and column blocks need no order among themselves.
constexpr int kMoveThreads = 256;

template <int LAYOUT>
struct RowShape {
  static constexpr int kBlk = LAYOUT == GW_LAYOUT_GLOBAL_FOLDED ? 80 : LAYOUT == GW_LAYOUT_GLOBAL_FULL ? 128 : 40;
  static constexpr int kPageBytes = kPage * kBlk * 16;
};

// The source token of kept token i, or -1 if keep_idx does not ascend there.
__device__ __forceinline__ int source_of(const int32_t* keep, int i, int L) {
  const int j = keep[i];
  const int before = i > 0 ? keep[i - 1] : -1;
  return j > before && j >= i && j < L ? j : -1;
}

template <int LAYOUT>
__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const CompactArgs a) {
  using R = RowShape<LAYOUT>;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y, col = blockIdx.x, tid = threadIdx.x;
  const int L = a.seq_lens[b], n = a.keep_lens[b];
  const bool reports = col == 0;
  if (L < 0 || L > a.max_pages * kPage) {
    if (reports && tid == 0) set_status(a.status, GW_DEV_LEN_RANGE);
    return;
  }
  if (n < 0 || n > L || n > a.keep_stride || n > static_cast<int64_t>(a.dst_max_pages) * kPage) {
    if (reports && tid == 0) set_status(a.status, GW_DEV_KEEP_RANGE);
    return;
  }
  const int32_t* keep = a.keep_idx + b * a.keep_stride;
  if (col == R::kBlk) {  // the weights
    float* acc = a.acc + b * a.acc_stride;
    for (int i0 = 0; i0 < n; i0 += kMoveThreads) {
      const int i = i0 + tid;
      const int j = i < n ? source_of(keep, i, L) : -1;
      const float w = j >= 0 ? acc[j] : 0.f;
      __syncthreads();
      if (j >= 0) acc[i] = w;
    }
    __syncthreads();
    for (int i = n + tid; i < L; i += kMoveThreads) acc[i] = 0.f;
    return;
  }
  const int32_t* src_table = a.block_table + static_cast<int64_t>(b) * a.max_pages;
  const int32_t* dst_table = a.dst_table + static_cast<int64_t>(b) * a.dst_max_pages;
  for (int i0 = 0; i0 < n; i0 += kMoveThreads) {
    const int i = i0 + tid;
    const int j = i < n ? source_of(keep, i, L) : -1;
    bool move = false;
    uint8_t* to = nullptr;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (j >= 0) {
      const int32_t sp = src_table[j / kPage], dp = dst_table[i / kPage];
      move = sp >= 0 && sp < a.num_pages && dp >= 0 && dp < a.num_pages;
      if (!move && reports) set_status(a.status, GW_DEV_PAGE_RANGE);
      if (move && sp == dp && i == j) move = false;
      if (move) {
        v = *reinterpret_cast<const uint4*>(a.pool + static_cast<int64_t>(sp) * R::kPageBytes +
                                            ((j % kPage / 8) * R::kBlk + col) * 128 + (j % 8) * 16);
        to = a.pool + static_cast<int64_t>(dp) * R::kPageBytes + ((i % kPage / 8) * R::kBlk + col) * 128 + (i % 8) * 16;
      }
    } else if (i < n && reports) {
      set_status(a.status, GW_DEV_KEEP_RANGE);
    }
    __syncthreads();
    if (move) *reinterpret_cast<uint4*>(to) = v;
  }
}

template <int LAYOUT>
cudaError_t launch_compact_layout(const CompactArgs& a, cudaStream_t st) {
  const dim3 grid(RowShape<LAYOUT>::kBlk + (a.acc ? 1 : 0), a.batch);
  return launch_pdl(evict_compact_kernel<LAYOUT>, grid, dim3(kMoveThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_evict_select(const SelectArgs& a, cudaStream_t st) {
  return launch_pdl(evict_select_kernel, dim3(a.batch), dim3(kSelThreads), 0, st, a);
}

cudaError_t launch_evict_compact(int layout, const CompactArgs& a, cudaStream_t st) {
  if (layout == GW_LAYOUT_GLOBAL_FOLDED) return launch_compact_layout<GW_LAYOUT_GLOBAL_FOLDED>(a, st);
  if (layout == GW_LAYOUT_GLOBAL_FULL) return launch_compact_layout<GW_LAYOUT_GLOBAL_FULL>(a, st);
  return launch_compact_layout<GW_LAYOUT_GLOBAL_FOLDED_E4M3>(a, st);
}

}  // namespace gw
