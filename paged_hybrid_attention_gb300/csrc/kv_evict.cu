// gw_kv_evict_select and gw_kv_evict_compact: a sequence of the global cache
// cut to the tokens that have drawn the most attention.
#include "common.cuh"

namespace gw {
namespace {

// A launch in clusters of `ctas` blocks along x, early under the same terms as
// launch_pdl's.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, int ctas, cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = early_launch() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// ---- select -------------------------------------------------------------------
// The weights' order as unsigned integers: larger weight, larger key; -0 and
// 0 share a key, and every NaN has key 1, below -inf (0x007fffff).
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = 0
  const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  return w != w ? 1u : k;
}
// Keys of no weight: a token behind the slice's end, and one at either end of
// the sequence that is kept in any case (inf has 0xff800000).
constexpr uint32_t kNoToken = 0, kProtected = 0xffffffffu;

// A cluster of 1 to kMaxSelCtas blocks takes a sequence, each block a
// contiguous slice of its tokens, each warp a contiguous piece of the slice, up
// to kSelKeys tokens per thread in registers (longer slices are read again in
// rounds).  The k-th largest key of the middle is found digit by digit from
// the top, 8 bits at a time: each block counts its keys of the current prefix
// by digit in shared memory, and after a cluster barrier every block adds up
// all blocks' counts and finds the same digit.  (Digits of 11 bits save a pass
// but make each block read eight times as many counts of the others.)  It
// ends with the first digit all of whose keys are kept.  Then the blocks
// exchange how many of their tokens are kept or tied, and write their indices
// in order.  8 x 131072 tokens take 15 to 16 us, 4.2 MB of weights read once: short
// passes between barriers bound it (a pass over 16 keys a thread is 1.2 us, its
// barrier and sums 1.5 us).
constexpr int kSelThreads = 1024;
constexpr int kSelKeys = 16;
constexpr int kMaxSelCtas = 8;

// The 32-bit word that block `rank` of the cluster has at this shared address.
__device__ __forceinline__ uint32_t ld_cluster(const uint32_t* p, int rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const SelectArgs a, int ctas) {
  __shared__ uint32_t hist[4][256];
  __shared__ uint32_t found[3];  // digit, keys of the prefix above it, keys of it
  __shared__ uint32_t kept[2];   // this block's tokens: kept for sure, tied
  __shared__ uint2 warp_kept[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  pdl_wait();
  pdl_trigger();
  const int L = a.seq_lens[b];
  int32_t* keep = a.keep_idx + b * a.keep_stride;
  if (L < 0 || L > a.acc_stride) {  // the same for the whole cluster
    if (rank == 0 && tid == 0) {
      set_status(a.status, GW_DEV_LEN_RANGE);
      a.keep_lens[b] = 0;
    }
    return;
  }
  if (rank == 0 && tid == 0) a.keep_lens[b] = min(L, a.budget);
  if (L <= a.budget) {
    for (int64_t j = rank * kSelThreads + tid; j < L; j += ctas * kSelThreads) keep[j] = static_cast<int32_t>(j);
    return;
  }
  // tokens by their place in the block's slice [t0, t0 + n): a slice has fewer
  // than 2^29, since a long row has kMaxSelCtas of them
  const int per = (L - 1) / ctas + 1;
  const int t0 = static_cast<int>(min(static_cast<int64_t>(rank) * per, static_cast<int64_t>(L)));
  const int n = min(per, L - t0);
  const int lo = a.sinks - t0, hi = L - a.recent - t0;  // the middle
  const float* acc = a.acc + b * a.acc_stride + t0;
  uint32_t need = a.budget - a.sinks - a.recent;  // of the middle
  const int rounds = (per - 1) / (kSelThreads * kSelKeys) + 1;
  const int keys = rounds > 1 ? kSelKeys : (per - 1) / kSelThreads + 1;  // of a thread, per round
  uint32_t key[kSelKeys];
  int first = 0;  // the token of r = 0; the next lie 32 apart
  auto load = [&](int round) {
    first = (round * 32 + warp) * keys * 32 + lane;
#pragma unroll
    for (int r = 0; r < kSelKeys; ++r) {
      if (r < keys) {
        const int j = first + r * 32;
        key[r] = j < n ? __float_as_uint(acc[j]) : 0;
      }
    }
#pragma unroll
    for (int r = 0; r < kSelKeys; ++r) {
      if (r < keys) {
        const int j = first + r * 32;
        key[r] = j >= n ? kNoToken : j < lo || j >= hi ? kProtected : order_key(__uint_as_float(key[r]));
      }
    }
  };
  load(0);
  (&hist[0][0])[tid] = 0;
  if (tid < 2) kept[tid] = 0;
  __syncthreads();
  uint32_t prefix = 0, mask = 0;
  const bool middle = need > 0;  // the same for the whole cluster
#pragma unroll 1
  for (int shift = 24; middle && shift >= 0; shift -= 8) {
    uint32_t* h = hist[shift / 8];
    for (int round = 0; round < rounds; ++round) {
      if (rounds > 1) load(round);
#pragma unroll
      for (int r = 0; r < kSelKeys; ++r) {
        // key + 1 is 1 and 0 for the keys of no weight
        if (r < keys && ((key[r] ^ prefix) & mask) == 0 && key[r] + 1 > 1) atomicAdd(&h[(key[r] >> shift) & 255], 1u);
      }
    }
    cluster_arrive();
    cluster_wait();
    if (warp < 8) {  // thread t: digit 255 - t, counted over the cluster
      uint32_t from[kMaxSelCtas], count = 0;
#pragma unroll
      for (int c = 0; c < kMaxSelCtas; ++c) from[c] = c < ctas ? ld_cluster(&h[255 - tid], c) : 0;
#pragma unroll
      for (int c = 0; c < kMaxSelCtas; ++c) count += from[c];
      uint32_t x = count;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) warp_kept[warp].x = x;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      uint32_t above = x - count;
      for (int w = 0; w < warp; ++w) above += warp_kept[w].x;
      if (above < need && above + count >= need) {
        found[0] = 255 - tid;
        found[1] = above;
        found[2] = count;
      }
    }
    __syncthreads();
    prefix |= found[0] << shift;
    mask |= 255u << shift;
    need -= found[1];
    const bool done = found[2] == need;  // all of the digit's keys are kept, whatever their lower bits
    __syncthreads();                     // found and warp_kept are written again
    if (done) break;
  }
  // Kept for sure: the ends, and in the middle what lies above `prefix`; of the
  // keys that match it the first `need`.  If nothing of the middle is kept, no
  // key but the ends' is above `last`.
  const uint32_t last = middle ? prefix | ~mask : kProtected;
  auto is_sure = [&](int r) { return key[r] > last || key[r] == kProtected; };
  auto is_tie = [&](int r) { return middle && key[r] >= prefix && key[r] <= last && key[r] + 1 > 1; };
  auto count_warp = [&]() {  // the round's counts of this warp
    uint2 n = make_uint2(0, 0);
#pragma unroll
    for (int r = 0; r < kSelKeys; ++r) {
      if (r < keys) {
        n.x += is_sure(r);
        n.y += is_tie(r);
      }
    }
    return make_uint2(__reduce_add_sync(0xffffffffu, n.x), __reduce_add_sync(0xffffffffu, n.y));
  };
  uint2 mine = make_uint2(0, 0);
  for (int round = 0; round < rounds; ++round) {
    if (rounds > 1) load(round);
    const uint2 w = count_warp();
    mine.x += w.x;
    mine.y += w.y;
  }
  if (lane == 0) {
    atomicAdd(&kept[0], mine.x);
    atomicAdd(&kept[1], mine.y);
    warp_kept[warp] = mine;
  }
  cluster_arrive();
  cluster_wait();
  // of the blocks before this one: lane c adds up block c
  uint32_t base_sure = lane < rank ? ld_cluster(&kept[0], lane) : 0, base_ties = lane < rank ? ld_cluster(&kept[1], lane) : 0;
  base_sure = __reduce_add_sync(0xffffffffu, base_sure);
  base_ties = __reduce_add_sync(0xffffffffu, base_ties);
  cluster_arrive();  // waited for at the end: no block leaves while others read its shared memory
  for (int round = 0; round < rounds; ++round) {
    if (rounds > 1) {
      load(round);
      mine = count_warp();
      __syncthreads();  // the previous round's reads of warp_kept are done
      if (lane == 0) warp_kept[warp] = mine;
      __syncthreads();
    }
    const uint2 w = warp_kept[lane];
    uint32_t sure = base_sure + __reduce_add_sync(0xffffffffu, lane < warp ? w.x : 0);
    uint32_t ties = base_ties + __reduce_add_sync(0xffffffffu, lane < warp ? w.y : 0);
    base_sure += __reduce_add_sync(0xffffffffu, w.x);
    base_ties += __reduce_add_sync(0xffffffffu, w.y);
    const uint32_t low = (1u << lane) - 1;
    if (mine.y == 0) {  // no ties in this warp, as in nearly all
      sure += min(ties, need);
#pragma unroll
      for (int r = 0; r < kSelKeys; ++r) {
        if (r < keys) {
          const uint32_t s = __ballot_sync(0xffffffffu, is_sure(r));
          if (is_sure(r)) keep[sure + __popc(s & low)] = t0 + first + r * 32;
          sure += __popc(s);
        }
      }
      continue;
    }
#pragma unroll
    for (int r = 0; r < kSelKeys; ++r) {
      if (r < keys) {
        const uint32_t s = __ballot_sync(0xffffffffu, is_sure(r)), e = __ballot_sync(0xffffffffu, is_tie(r));
        const uint32_t ties_before = ties + __popc(e & low);
        if ((s >> lane & 1) || ((e >> lane & 1) && ties_before < need))
          keep[sure + __popc(s & low) + min(ties_before, need)] = t0 + first + r * 32;
        sure += __popc(s);
        ties += __popc(e);
      }
    }
  }
  cluster_wait();
}

// ---- compact ------------------------------------------------------------------
// Token i's row takes token keep[i]'s place, keep[i] >= i.  A walk takes
// kWalkCols adjacent 16-byte column blocks of the sequence's rows in token
// order, a step of kMoveThreads rows per block at a time: all of a step's rows
// are read before any is written (the barrier, of the block or of the walk's
// cluster), and no later step reads what it writes, since later steps' sources
// lie at or behind their own first token.  So the move is exact in place, walks
// need no order among themselves, and the next step's rows may be on their way
// while this one's are written.
// 8 x 131072 folded rows to 32768 take 190 to 200 us: 924 MB read (the 64-byte
// pieces that hold a kept row) and 316 MB written, 0.92 to 0.96 of a copy's rate;
// to 122880, 470 us (384 at a copy's rate).  Few sequences are bound by a step's
// round trip, about 1.4 us: their walks get more blocks.  512 rows per block and
// step are the best: 256 took 284 us, 1024 278 us; four column blocks a walk are
// no faster, one takes 264 us.
constexpr int kMoveThreads = 512;
constexpr int kWalkCols = 2;     // column blocks of a walk
constexpr int kMaxMoveCtas = 8;  // blocks of a walk

template <int LAYOUT>
struct RowShape {
  static constexpr int kBlk = LAYOUT == GW_LAYOUT_GLOBAL_FOLDED ? 80 : LAYOUT == GW_LAYOUT_GLOBAL_FULL ? 128 : 40;
  static constexpr int kPageBytes = kPage * kBlk * 16;
};

// The source token of kept token i, or -1 if keep_idx does not ascend there or
// has fallen below i, where a row would move backwards.
__device__ __forceinline__ int source_of(const int32_t* keep, int i, int L) {
  const int j = keep[i];
  const int before = i > 0 ? keep[i - 1] : -1;
  return j > before && j >= i && j < L ? j : -1;
}

// Kept rows are scattered 16-byte pieces: fetching them 64 bytes at a time
// instead of the default 128 saves a quarter of the DRAM reads when one row in
// four is kept (199 against 242 us for 8 x 131072 rows cut to 32768).
__device__ __forceinline__ uint4 ld_piece(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L2::64B.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p)
               : "memory");
  return v;
}

// All of a walk's threads have read a step: the block's, or those of the `ctas`
// blocks of its cluster.
__device__ __forceinline__ void step_bar(int ctas) {
  if (ctas == 1) {
    __syncthreads();
  } else {
    cluster_arrive();
    cluster_wait();
  }
}

// The weights of one sequence: the same walk, kAccRows tokens per thread and step.
__device__ __forceinline__ void move_weights(float* acc, const int32_t* keep, int n, int L, int rank, int ctas) {
  constexpr int kAccRows = 8;
  const int tid = threadIdx.x;
  const int64_t step = static_cast<int64_t>(ctas) * kMoveThreads * kAccRows;
  for (int64_t i0 = static_cast<int64_t>(rank) * kMoveThreads * kAccRows, s0 = 0; s0 < n; i0 += step, s0 += step) {
    int j[kAccRows];
    float w[kAccRows];
#pragma unroll
    for (int r = 0; r < kAccRows; ++r) {
      const int64_t i = i0 + r * kMoveThreads + tid;
      j[r] = i < n ? source_of(keep, static_cast<int>(i), L) : -1;
    }
#pragma unroll
    for (int r = 0; r < kAccRows; ++r) w[r] = j[r] >= 0 ? acc[j[r]] : 0.f;
    step_bar(ctas);
#pragma unroll
    for (int r = 0; r < kAccRows; ++r)
      if (j[r] >= 0) acc[i0 + r * kMoveThreads + tid] = w[r];
  }
  step_bar(ctas);
  for (int64_t i = static_cast<int64_t>(n) + rank * kMoveThreads + tid; i < L; i += ctas * kMoveThreads) acc[i] = 0.f;
}

// One walk: column block pair `col` of sequence b, or its weights (-1).  It may
// begin before the blocks' last one has ended: no two walks share a byte.
template <int LAYOUT>
__device__ __forceinline__ void compact_walk(const CompactArgs& a, int b, int col, int rank, int ctas) {
  using R = RowShape<LAYOUT>;
  constexpr int W = kWalkCols;
  const int tid = threadIdx.x;
  const int L = a.seq_lens[b], n = a.keep_lens[b];
  const bool reports = col == 0;
  if (L < 0 || L > a.max_pages * kPage) {  // as below, the same for all of a cluster
    if (reports && rank == 0 && tid == 0) set_status(a.status, GW_DEV_LEN_RANGE);
    return;
  }
  if (n < 0 || n > L || n > a.keep_stride || n > static_cast<int64_t>(a.dst_max_pages) * kPage) {
    if (reports && rank == 0 && tid == 0) set_status(a.status, GW_DEV_KEEP_RANGE);
    return;
  }
  const int32_t* keep = a.keep_idx + b * a.keep_stride;
  if (col < 0) {
    move_weights(a.acc + b * a.acc_stride, keep, n, L, rank, ctas);
    return;
  }
  const int32_t* src_table = a.block_table + static_cast<int64_t>(b) * a.max_pages;
  const int32_t* dst_table = a.dst_table + static_cast<int64_t>(b) * a.dst_max_pages;
  uint8_t* base = a.pool + col * W * 128;
  struct Rows {
    uint4 v[W];
    uint8_t* to;  // null: nothing to move
  };
  const int64_t step = static_cast<int64_t>(ctas) * kMoveThreads;
  const int mine = rank * kMoveThreads + tid;  // this thread's row of a step
  // the source token of the thread's row of the step at i0; -1: none
  auto index = [&](int64_t i0) {
    const int64_t i = i0 + mine;
    if (i >= n) return -1;
    const int j = source_of(keep, static_cast<int>(i), L);
    if (j < 0 && reports) set_status(a.status, GW_DEV_KEEP_RANGE);
    return j;
  };
  auto fetch = [&](int64_t i0, int j, Rows& x) {
    x.to = nullptr;
    if (j < 0) return;
    const int i = static_cast<int>(i0) + mine;
    const int32_t sp = src_table[j / kPage], dp = dst_table[i / kPage];
    if (sp < 0 || sp >= a.num_pages || dp < 0 || dp >= a.num_pages) {
      if (reports) set_status(a.status, GW_DEV_PAGE_RANGE);
      return;
    }
    if (sp == dp && i == j) return;
    const uint8_t* from = base + static_cast<int64_t>(sp) * R::kPageBytes + (j % kPage / 8) * (R::kBlk * 128) + (j % 8) * 16;
    x.to = base + static_cast<int64_t>(dp) * R::kPageBytes + (i % kPage / 8) * (R::kBlk * 128) + (i % 8) * 16;
#pragma unroll
    for (int k = 0; k < W; ++k) x.v[k] = ld_piece(from + k * 128);
  };
  Rows now, next;
  int j = index(0), j1 = index(step);
  fetch(0, j, now);
  for (int64_t i0 = 0; i0 < n; i0 += step) {
    const int j2 = index(i0 + 2 * step);
    fetch(i0 + step, j1, next);
    step_bar(ctas);
    if (now.to) {
#pragma unroll
      for (int k = 0; k < W; ++k) *reinterpret_cast<uint4*>(now.to + k * 128) = now.v[k];
    }
    now = next;
    j1 = j2;
  }
}

// A cluster of `ctas` blocks per walk, sequences along y; kTurns: fewer
// clusters than walks, which take them in turn (a kernel of its own: the loop
// takes 54 registers instead of 40, and held to 40 it spilled and cost every
// move 2 to 3%).
template <int LAYOUT, bool kTurns>
__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const CompactArgs a, int ctas) {
  pdl_wait();
  pdl_trigger();
  const int rank = static_cast<int>(blockIdx.x) % ctas, first = static_cast<int>(blockIdx.x) / ctas;
  if constexpr (kTurns) {
    const int per_seq = RowShape<LAYOUT>::kBlk / kWalkCols + (a.acc ? 1 : 0);
    for (int walk = first; walk < per_seq * a.batch; walk += static_cast<int>(gridDim.x) / ctas)
      compact_walk<LAYOUT>(a, walk / per_seq, walk % per_seq - (a.acc ? 1 : 0), rank, ctas);
  } else {
    compact_walk<LAYOUT>(a, blockIdx.y, first - (a.acc ? 1 : 0), rank, ctas);
  }
}

template <int LAYOUT>
cudaError_t launch_compact_layout(const CompactArgs& a, cudaStream_t st) {
  // As many blocks to a walk as leave the blocks of all walks on the GPU at
  // once, three per SM less a twelfth that clusters leave unused.  1 x 131072
  // folded rows to a quarter: eight 34 us, four 50, one 91; 3 x 131072: three
  // 85, two 102, one 115; 8 x 131072: one 191, two 233.  Under a CTA cap there
  // are as many blocks as SMs are allowed, since three do not keep to one SM.
  const int per_seq = RowShape<LAYOUT>::kBlk / kWalkCols + (a.acc ? 1 : 0);
  const int64_t walks = static_cast<int64_t>(per_seq) * a.batch;
  const bool capped = grid_ctas() < num_sms();
  const int64_t room = capped ? grid_ctas() / walks : 11 * static_cast<int64_t>(grid_ctas()) / (4 * walks);
  const int ctas = static_cast<int>(room < 1 ? 1 : room > kMaxMoveCtas ? kMaxMoveCtas : room);
  const int clusters = grid_ctas() / ctas;
  if (capped && clusters < walks)
    return launch_cluster(evict_compact_kernel<LAYOUT, true>, dim3(clusters * ctas), dim3(kMoveThreads), ctas, st, a, ctas);
  return launch_cluster(evict_compact_kernel<LAYOUT, false>, dim3(per_seq * ctas, a.batch), dim3(kMoveThreads), ctas, st, a,
                        ctas);
}

}  // namespace

cudaError_t launch_evict_select(const SelectArgs& a, cudaStream_t st) {
  // Lengths are device values: the row stride bounds them.  More blocks per
  // sequence while each would still have more than 4096 tokens.  With 1024 |
  // 2048 | 4096 | 8192 | 16384 instead, 16 x 8192 tokens take 11.8 | 10.9 | 10.7 |
  // 10.6 | 10.7 us, 16 x 16384 18.9 | 18.9 | 10.2 | 10.9 | 13.1, 1 x 8192 9.7 |
  // 9.4 | 9.7 | 10.5 | 10.5, 8 x 131072 16.1 with any.  (128 x 16384, which fill
  // the GPU with one block each: 84 | 84 | 37 | 21 | 14.)
  int ctas = 1;
  while (ctas < kMaxSelCtas && a.acc_stride > static_cast<int64_t>(4096) * ctas) ctas *= 2;
  return launch_cluster(evict_select_kernel, dim3(static_cast<unsigned>(a.batch) * ctas), dim3(kSelThreads), ctas, st, a, ctas);
}

cudaError_t launch_evict_compact(int layout, const CompactArgs& a, cudaStream_t st) {
  if (layout == GW_LAYOUT_GLOBAL_FOLDED) return launch_compact_layout<GW_LAYOUT_GLOBAL_FOLDED>(a, st);
  if (layout == GW_LAYOUT_GLOBAL_FULL) return launch_compact_layout<GW_LAYOUT_GLOBAL_FULL>(a, st);
  return launch_compact_layout<GW_LAYOUT_GLOBAL_FOLDED_E4M3>(a, st);
}

}  // namespace gw
