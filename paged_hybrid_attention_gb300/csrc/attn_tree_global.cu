// Attention of drafted trees on GLOBAL layers (gw_tree_attn_global), on the
// tensor cores (tcgen05): head dim 512, one KV head, all three pool layouts, calls
// of up to 64 rows x heads (e4m3 pool: 32; attn_tree_global_rows.cu has the others).
//
// Row r of a sequence's n rows sees the cached tokens [0, L - n) and the drafts of
// its mask word.  A unit is (sequence, chunk of tiles).  The cached tokens are the
// products' long side and the rows x heads their NR columns, 32 or 64:
//   S^T[T x NR]    = K_tile[T x 512] . Q^T       (UMMA M = 64, e4m3 128)
//   O^T[512 x NR] += V_tile^T[512 x T] . P^T     (UMMA M = 128, four times)
// so that the cache is read once and no logit computed twice (rows along M fill 128
// of them and make each half of the output dims compute all logits).  T is 48 tokens
// on folded pools, three tiles in shared memory beside 32 rows of Q (8 x 131072
// tokens, 8 heads, 4 drafts: 222 us, two tiles of 64 tokens 231) and two beside 64
// (309 us with 8 drafts at that step, three of 32 tokens 316); on the full layout 64; on the e4m3
// pool, whose MMAs bound a call, 128 (203 us with tiles of 64 and 193 with 128 at
// that step).
//
// 8 x 131072 tokens, 8 heads, 4 drafts: folded 222 us with the merge (0.89 of the copy
// rate), e4m3 148 (0.67); full layout, 4 x 131072, 167 (0.94).  8 drafts: folded 314
// us (0.63, bound by the MMAs' and the softmax's chain over two tiles; in
// attn_tree_global_rows.cu 381), full 176 (0.90; 247).
//
// A tile is whole pages of 8-token x 16-byte blocks, which are UMMA core matrices:
// the K-major A operand of Q.K^T, whose K-steps point at k_rot and V on folded
// pools, and the MN-major A operand of P.V.  (With T = 48 the last quarter of A's
// 64 rows is whatever lies behind the tile; nothing reads those rows of S.)  On the
// full layout, whose tile is 128 KB, there is room for one, and K and V are copied
// and released apart.
// On the e4m3 pool q is two e4m3 terms after an exact power-of-two scaling per row,
// side by side along N, and P three e5m2 terms (tcgen05.cuh), side by side too:
// S and O have a column per row and term, which the softmax and the epilogue add.
//
// Warp roles (384 threads, 512 with 64 rows): 0-3 softmax (a thread per token) and
// epilogue (a thread per dim) of rows 0-31, 12-15 of the others, 4 copies (of K on
// the full layout, whose V warp 5 copies), 6 issues Q.K^T (and owns tensor memory), 7
// issues P.V, 8-11 Q rows and what they see (with one warp a sequence of 8192 tokens
// took 4 us more at 8 drafts, 3 at 4).  Every wait is bounded (GW_DEV_TIMEOUT).
#include "attn_tree.cuh"

namespace gw {
namespace {

constexpr float kUnset = -1e38f;  // reference of a row that has seen no key

template <int LAYOUT, int NR>
struct FT;
template <int NR>
struct FT<GW_LAYOUT_GLOBAL_FOLDED, NR> {
  static constexpr bool kE4 = false, kApart = false;
  static constexpr int kPages = 3;  // of a tile
  static constexpr int kPageBytes = 20480, kBlk = 80, kVcb = 0, kBufs = NR == 32 ? 3 : 2, kSteps = 32;
  __device__ static constexpr int k_cb(int ks) { return ks < 8 ? 64 + 2 * ks : 2 * ks; }
};
template <int NR>
struct FT<GW_LAYOUT_GLOBAL_FULL, NR> {
  static constexpr bool kE4 = false, kApart = true;
  static constexpr int kPages = 4;
  static constexpr int kPageBytes = 32768, kBlk = 128, kVcb = 64, kBufs = 1, kSteps = 32;
  __device__ static constexpr int k_cb(int ks) { return 2 * ks; }
};
template <>
struct FT<GW_LAYOUT_GLOBAL_FOLDED_E4M3, 32> {
  static constexpr bool kE4 = true, kApart = false;
  static constexpr int kPages = 8;
  static constexpr int kPageBytes = 10240, kBlk = 40, kVcb = 0, kBufs = 2, kSteps = 16;
  __device__ static constexpr int k_cb(int ks) { return ks < 4 ? 32 + 2 * ks : 2 * ks; }
};

template <int LAYOUT, int NR>
struct FL : FT<LAYOUT, NR> {
  using B = FT<LAYOUT, NR>;
  static constexpr int kGroups = NR / 32;              // of softmax warps, 32 rows each
  static constexpr int kThreads = 256 + 128 * kGroups;
  static constexpr int kTok = B::kPages * kPage;       // tokens of a tile
  static constexpr int kTerms = B::kE4 ? 3 : 1;        // of P
  static constexpr int kNT = NR * kTerms;              // N of P.V
  static constexpr int kSCols = B::kE4 ? 2 * NR : NR;  // N of Q.K^T
  static constexpr int kOBase = 2 * kSCols;            // O's columns, behind the buffers of S
  static constexpr int kRowsPerBlk = B::kE4 ? 16 : 8;  // rows in 16 bytes of P
  static constexpr int kQBlk = B::kE4 ? 32 : 64;       // 16-byte blocks of a row of Q (of a term)
};

template <int LAYOUT, int NR>
struct FSmem {
  using T = FL<LAYOUT, NR>;
  uint8_t tiles[T::kBufs][T::kPages * T::kPageBytes];
  uint8_t q[NR * 1024];  // bf16 [NR / 8][64][8][16 B]; e4m3 [hi, lo][NR / 8][32][8][16 B]
  uint8_t p[T::kTok * T::kNT * (T::kE4 ? 1 : 2)];  // P^T [8 tokens][16-byte block of rows][8][16 B]
  TreeRow rows[kRowRing][NR];
  float m[NR], alpha[NR], inv[NR], red[T::kGroups][4][32];
  uint64_t kfull[T::kBufs], kempty[T::kBufs], vfull[T::kBufs], vempty[T::kBufs];
  uint64_t s_ready[2], s_free[2], p_ready, p_free, o_done, q_full, q_free;
  int32_t mask[T::kBufs], vmask[T::kBufs];  // pages of the tile (K, V apart) that were loaded
  // by tile parity: index + 1 of the last tile that asked for a new reference
  int32_t flag[T::kGroups][2];
  uint32_t tmem_base;
  TreePlan plan;
};
static_assert(sizeof(FSmem<GW_LAYOUT_GLOBAL_FOLDED, 32>) <= 232448, "shared memory of one CTA");
static_assert(sizeof(FSmem<GW_LAYOUT_GLOBAL_FOLDED, 64>) <= 232448, "shared memory of one CTA");
static_assert(sizeof(FSmem<GW_LAYOUT_GLOBAL_FULL, 32>) <= 232448, "shared memory of one CTA");
static_assert(sizeof(FSmem<GW_LAYOUT_GLOBAL_FULL, 64>) <= 232448, "shared memory of one CTA");
static_assert(sizeof(FSmem<GW_LAYOUT_GLOBAL_FOLDED_E4M3, 32>) <= 232448, "shared memory of one CTA");

// of a group of softmax warps
__device__ __forceinline__ void softmax_bar(int group) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
}

struct Unit {
  int s, n, nc, base, hi, t0, nt, row0;
};

template <int LAYOUT, int HQ, int NR>
__device__ __forceinline__ Unit unit_of(const LocalArgs& a, const TreePlan& plan, int u) {
  Unit w;
  const int at = plan_seq(plan.ub, a.batch, u);
  w.s = plan.seq[at];
  w.row0 = a.cu_q_rows[w.s];
  w.n = a.cu_q_rows[w.s + 1] - w.row0;
  const int L = a.seq_lens[w.s];
  w.base = L - w.n;
  const TreeSpan sp = tree_span(L, w.n, a.window, tree_rule_few(HQ));
  w.nc = sp.chunks();
  const int c = u - plan.ub[at];
  w.t0 = c * sp.ct * kTreeTile;
  const int tiles = min(sp.ct, sp.tiles - c * sp.ct);
  w.hi = min(L, (c * sp.ct + tiles) * kTreeTile) - 1;
  w.nt = (w.hi - w.t0) / FL<LAYOUT, NR>::kTok + 1;
  return w;
}

template <int LAYOUT, int HQ, int NR>
__global__ void __launch_bounds__(FL<LAYOUT, NR>::kThreads, 1) global_tree_kernel(const LocalArgs a) {
  using T = FL<LAYOUT, NR>;
  using SM = FSmem<LAYOUT, NR>;
  constexpr bool kE4 = T::kE4;
  constexpr int NB = T::kBufs, kTok = T::kTok, kPages = T::kPages;
  constexpr float kBelow = Reference<kE4>::kBelow, kRaise = Reference<kE4>::kRaise;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  SM& sm = *reinterpret_cast<SM*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  int32_t* st = a.status;

  if (tid == 0) {
    for (int b = 0; b < NB; ++b) {
      mbar_init(&sm.kfull[b], 1);
      mbar_init(&sm.kempty[b], 1);
      mbar_init(&sm.vfull[b], 1);
      mbar_init(&sm.vempty[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.s_ready[b], 1);
      mbar_init(&sm.s_free[b], 128 * T::kGroups);
      for (int g = 0; g < T::kGroups; ++g) sm.flag[g][b] = 0;
    }
    mbar_init(&sm.p_ready, 128 * T::kGroups);
    mbar_init(&sm.p_free, 1);
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.q_full, 4);
    mbar_init(&sm.q_free, 1);
    fence_mbar_init();
  }
  if (warp == 6) {
    tc::alloc(&sm.tmem_base, 512);
    tc::relinquish();
  }
  pdl_wait();
  pdl_trigger();
  plan_tree(a, sm.plan, 1, tree_rule_few(HQ), 512);
  const int total = sm.plan.ub[a.batch];
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp == 4 || (T::kApart && warp == 5)) {
    // --------------------------------------------------------- page copies
    // lane j copies page j of a tile, or its K or V: per 8-token block
    const bool is_v = warp == 5;
    uint64_t* const fulls = is_v ? sm.vfull : sm.kfull;
    uint64_t* const empties = is_v ? sm.vempty : sm.kempty;
    const uint64_t pol = policy_evict_first();
    uint32_t gi = 0;
    int wt = 0;
    bool ok = true;
    for (int u = tree_unit(0); u < total && ok; u = tree_unit(++wt)) {
      const Unit w = unit_of<LAYOUT, HQ, NR>(a, sm.plan, u);
      const int32_t* bt = a.block_table + static_cast<int64_t>(w.s) * a.max_pages;
      for (int t = 0; t < w.nt; ++t, ++gi) {
        const int b = gi % NB;
        const uint32_t use = gi / NB;
        const int k = w.t0 + t * kTok + lane * kPage;
        int32_t pg = -1;
        if (lane < kPages && k <= w.hi) {
          pg = bt[k / kPage];
          if (pg < 0 || pg >= a.num_pages) {
            if (!is_v) set_status(st, GW_DEV_PAGE_RANGE);
            pg = -1;
          }
        }
        const uint32_t loaded = __ballot_sync(0xffffffffu, pg >= 0);
        if (use > 0 && !warp_wait(&empties[b], (use - 1) & 1, st)) { ok = false; break; }
        constexpr uint32_t kBytes = T::kApart ? T::kPageBytes / 2 : T::kPageBytes;
        if (lane == 0) {
          (is_v ? sm.vmask : sm.mask)[b] = static_cast<int32_t>(loaded);
          mbar_arrive_expect_tx(&fulls[b], static_cast<uint32_t>(__popc(loaded)) * kBytes);
        }
        __syncwarp();
        if (pg >= 0) {
          uint8_t* dst = sm.tiles[b] + lane * T::kPageBytes;
          const uint8_t* src = a.pool + static_cast<int64_t>(pg) * T::kPageBytes;
          if constexpr (T::kApart) {
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
              const int o = (tb * T::kBlk + (is_v ? T::kVcb : 0)) * 128;
              bulk_g2s(dst + o, src + o, T::kVcb * 128, &fulls[b], pol);
            }
          } else {
            bulk_g2s(dst, src, T::kPageBytes, &fulls[b], pol);
          }
        }
      }
    }
    drain<NB>(fulls, gi);
  } else if (warp == 6) {
    // ---------------------------------------------------- Q.K^T issue
    const uint32_t id_s =
        kE4 ? tc::idesc_e4m3(128, T::kSCols, false, false) : tc::idesc_bf16(64, T::kSCols, false, false);
    // Q: 16-byte blocks 128 B apart, then the next 8 rows (of a term, then of the next)
    const uint64_t dq = tc::smem_desc(smem_u32(sm.q), 128, T::kQBlk * 128);
    uint32_t gi = 0;
    int wt = 0;
    bool ok = true;
    for (int u = tree_unit(0); u < total && ok; u = tree_unit(++wt)) {
      const Unit w = unit_of<LAYOUT, HQ, NR>(a, sm.plan, u);
      if (!warp_wait(&sm.q_full, wt & 1, st)) break;
      for (int j = 0; j < w.nt; ++j, ++gi) {
        const int b = gi % NB, sb = gi & 1;
        if (!warp_wait(&sm.kfull[b], (gi / NB) & 1, st)) { ok = false; break; }
        if (gi >= 2 && !warp_wait(&sm.s_free[sb], ((gi >> 1) - 1) & 1, st)) { ok = false; break; }
        const uint32_t ta = smem_u32(sm.tiles[b]);
        const int mask = sm.mask[b];
        if (mask != (1 << kPages) - 1) {  // pages not loaded: zeros, no stale bytes
          constexpr int kCols = T::kApart ? T::kVcb : T::kBlk;  // of K, or of the page
          for (int blk = 0; blk < 2 * kPages; ++blk) {          // 8-token blocks
            if ((mask >> (blk >> 1)) & 1) continue;
            for (int o = lane * 16; o < kCols * 128; o += 32 * 16) zero16(ta + blk * T::kBlk * 128 + o);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc::fence_after();
        const uint64_t dk = tc::smem_desc(ta, 128, T::kBlk * 128);
#pragma unroll
        for (int ks = 0; ks < T::kSteps; ++ks) {
          const uint64_t ad = dk + ((T::k_cb(ks) * 128) >> 4), bd = dq + ((2 * ks * 128) >> 4);
          if constexpr (kE4)
            tc::mma_e4m3_warp(tmem + T::kSCols * sb, ad, bd, id_s, ks > 0);
          else
            tc::mma_bf16_warp(tmem + T::kSCols * sb, ad, bd, id_s, ks > 0);
        }
        if (T::kApart) tc::commit_warp(&sm.kempty[b]);
        tc::commit_warp(&sm.s_ready[sb]);
        if (j == w.nt - 1) tc::commit_warp(&sm.q_free);
      }
    }
    drain<2>(sm.s_ready, gi);
  } else if (warp == 7) {
    // ------------------------------------------------------- P.V issue
    const uint32_t id_o =
        kE4 ? tc::idesc_e4m3_e5m2(128, T::kNT, true, true) : tc::idesc_bf16(128, T::kNT, true, true);
    // P^T: 8-token groups of kNT / kRowsPerBlk blocks of 128 bytes
    constexpr uint32_t kGroup = T::kNT / T::kRowsPerBlk * 128;
    constexpr int kDimBlks = kE4 ? 8 : 16;  // 16-byte column blocks of 128 dims
    const uint64_t dp = tc::smem_desc(smem_u32(sm.p), kGroup, 128);
    uint32_t gi = 0;
    int wt = 0;
    bool ok = true;
    for (int u = tree_unit(0); u < total && ok; u = tree_unit(++wt)) {
      const Unit w = unit_of<LAYOUT, HQ, NR>(a, sm.plan, u);
      const uint32_t o = tmem + T::kOBase;
      for (int j = 0; j < w.nt; ++j, ++gi) {
        const int b = gi % NB;
        if (T::kApart && !warp_wait(&sm.vfull[b], (gi / NB) & 1, st)) { ok = false; break; }
        // (a unit's first P comes after the last unit's O has been read)
        if (!warp_wait(&sm.p_ready, gi & 1, st)) { ok = false; break; }
        const uint32_t ta = smem_u32(sm.tiles[b]);
        const int key0 = w.t0 + j * kTok;
        const int vmask = T::kApart ? sm.vmask[b] : (1 << kPages) - 1;
        if (key0 + kTok - 1 > w.hi || vmask != (1 << kPages) - 1) {
          // V rows behind the last key (K rows there only made logits that were
          // masked) or of pages not loaded: zero weights must meet finite values
          // (8-token blocks from their 16-byte pieces' start: a row's pieces share banks)
          const int k = lane & 7;
          for (int blk = 0; blk < kTok / 8; ++blk) {
            const bool page_ok = (vmask >> (blk / 2)) & 1;
            if (page_ok && key0 + 8 * blk + 7 <= w.hi) continue;
            if (!page_ok || key0 + 8 * blk + k > w.hi)
#pragma unroll
              for (int cb = 0; cb < 4 * kDimBlks; cb += 4)
                zero16(ta + (blk * T::kBlk + T::kVcb + cb + (lane >> 3)) * 128 + k * 16);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc::fence_after();
#pragma unroll
        for (int kk = 0; kk < kTok / (kE4 ? 32 : 16); ++kk) {
          const uint64_t bd = dp + ((kk * (kE4 ? 4 : 2) * kGroup) >> 4);
#pragma unroll
          for (int blk = 0; blk < 4; ++blk) {
            const uint64_t ad = tc::smem_desc(
                ta + (T::kVcb + kDimBlks * blk) * 128 + kk * (kE4 ? 4 : 2) * T::kBlk * 128, T::kBlk * 128, 128);
            if constexpr (kE4)
              tc::mma_e4m3_warp(o + T::kNT * blk, ad, bd, id_o, !(j == 0 && kk == 0));
            else
              tc::mma_bf16_warp(o + T::kNT * blk, ad, bd, id_o, !(j == 0 && kk == 0));
          }
        }
        tc::commit_warp(T::kApart ? &sm.vempty[b] : &sm.kempty[b]);
        tc::commit_warp(&sm.p_free);
        if (j == w.nt - 1) tc::commit_warp(&sm.o_done);
      }
    }
    drain<1>(&sm.p_free, gi);
  } else if (warp >= 8 && warp < 12) {
    // -------------------------------------------------------------- Q rows
    // a warp copies 8 rows of every 32: lane l row l % 8, every fourth 16-byte block
    // from l / 8 on; a sequence's rows x heads lie one after the other
    int wt = 0;
    for (int u = tree_unit(0); u < total; u = tree_unit(++wt)) {
      const Unit w = unit_of<LAYOUT, HQ, NR>(a, sm.plan, u);
      const uint16_t* src = a.q + static_cast<int64_t>(w.row0) * HQ * 512;
      const int count = w.n * HQ, first = 8 * (warp - 8);
      float scale = 1.f;
      if constexpr (kE4) {
        // each row's largest |q|
#pragma unroll 4
        for (int k = 0; k < 8; ++k) {
          const int r = first + k;
          if (r >= count) break;
          const uint4 x = *reinterpret_cast<const uint4*>(src + r * 512 + 8 * lane);
          const uint4 y = *reinterpret_cast<const uint4*>(src + r * 512 + 256 + 8 * lane);
          const uint32_t u8[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
          float mq = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            mq = fmaxf(mq, fmaxf(fabsf(__uint_as_float(u8[i] << 16)), fabsf(__uint_as_float(u8[i] & 0xFFFF0000u))));
          mq = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mq)));  // not negative: ordered as bits
          const int ex = mq > 0.f ? static_cast<int>((__float_as_uint(mq) >> 23) & 0xFF) - 127 : 7;
          const int e = min(125, max(-125, 7 - ex));
          // (an infinity, which the terms cannot hold, makes the row's logits NaN)
          if ((lane & 7) == k)
            scale = mq < INFINITY ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : NAN;
        }
      } else {
        // into L2 while the unit before is at work
#pragma unroll
        for (int g = 0; g < T::kGroups; ++g)
          if (wt > 0 && lane < 8 && 32 * g + first + lane < count) prefetch_l2(src + (32 * g + first + lane) * 512, 1024);
      }
      if (wt > 0 && !warp_wait(&sm.q_free, (wt - 1) & 1, st)) break;
#pragma unroll
      for (int g = 0; g < T::kGroups; ++g) {
        const int r = 32 * g + first + (lane & 7), rb = r / 8;
        const bool ok_row = r < count;
        const uint16_t* from = src + (ok_row ? r : 0) * 512;
        if constexpr (kE4) {
          const float up = 1.f / scale;  // a power of two: exact
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int cb = (lane >> 3) + 4 * j;
            uint32_t h[8], l[8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint4 x =
                  ok_row ? *reinterpret_cast<const uint4*>(from + 16 * cb + 8 * k) : make_uint4(0u, 0u, 0u, 0u);
              const uint32_t u4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                split_e4m3(__uint_as_float(u4[i] << 16) * up, __uint_as_float(u4[i] & 0xFFFF0000u) * up, h[4 * k + i],
                           l[4 * k + i]);
            }
            uint8_t* dst = sm.q + (rb * T::kQBlk + cb) * 128 + (lane & 7) * 16;
            *reinterpret_cast<uint4*>(dst) =
                make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
            *reinterpret_cast<uint4*>(dst + NR * 512) =
                make_uint4(l[0] | (l[1] << 16), l[2] | (l[3] << 16), l[4] | (l[5] << 16), l[6] | (l[7] << 16));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int cb = (lane >> 3) + 4 * j;
            const uint32_t at = smem_u32(sm.q + (rb * T::kQBlk + cb) * 128 + (lane & 7) * 16);
            if (ok_row)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from + 8 * cb) : "memory");
            else
              zero16(at);
          }
        }
      }
      // what the rows see, its load beside those of Q; rows behind the last see
      // everything, which costs no masks: nobody reads them
      if (lane < 8)
#pragma unroll
        for (int g = 0; g < T::kGroups; ++g) {
          const int r = 32 * g + first + lane;
          TreeRow row{~0ull, 0, 1.f};
          if (r < count) row = tree_row(a, w.row0, r / HQ, w.n, w.base, false);
          row.scale = scale;
          sm.rows[wt % kRowRing][r] = row;
        }
      if constexpr (!kE4) {
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full);
    }
  } else if (warp < 4 || warp >= 12) {  // (warp 5 has nothing to do on the folded layouts)
    // ------------------------------------------------- softmax and epilogue
    // warps 0-3 rows 0 to 31, 12-15 the others; a warp reaches quadrant warp % 4
    const int grp = warp >= 12, quad = warp & 3, row0 = 32 * grp, gtid = 32 * quad + lane;
    // M = 64 uses lanes 0..15 of a quadrant
    const int tok = kE4 ? gtid : 16 * quad + (lane & 15);
    const bool active = (kE4 || lane < 16) && tok < kTok;
    const uint32_t lane_base = static_cast<uint32_t>(32 * quad) << 16;
    uint32_t gi = 0;
    int wt = 0;
    bool ok = true, all = true;  // this warp's waits; those of the four, as last voted
    for (int u = tree_unit(0); u < total && all; u = tree_unit(++wt)) {
      const Unit w = unit_of<LAYOUT, HQ, NR>(a, sm.plan, u);
      const TreeRow* rows = sm.rows[wt % kRowRing] + row0;
      const uint32_t o_addr = tmem + lane_base + T::kOBase + row0;
      float l_acc[32];
#pragma unroll
      for (int r = 0; r < 32; ++r) l_acc[r] = 0.f;
      for (int j = 0; j < w.nt; ++j, ++gi) {
        const int sb = gi & 1;
        ok = ok && warp_wait(&sm.s_ready[sb], (gi >> 1) & 1, st);
        tc::fence_after();
        float x[32];
        {
          const uint32_t s_addr = tmem + lane_base + T::kSCols * sb + row0;
          uint32_t y[32];
          tc::ld32(s_addr, y);
          if constexpr (kE4) {
            uint32_t z[32];
            tc::ld32(s_addr + NR, z);
            tc::wait_ld();
#pragma unroll
            for (int r = 0; r < 32; ++r) x[r] = (__uint_as_float(y[r]) + __uint_as_float(z[r])) * rows[r].scale;
          } else {
            tc::wait_ld();
#pragma unroll
            for (int r = 0; r < 32; ++r) x[r] = __uint_as_float(y[r]);
          }
        }
        tc::fence_before();
        mbar_arrive(&sm.s_free[sb]);
        // rows that see this thread's token
        const int key0 = w.t0 + j * kTok;
        uint32_t vis = active ? ~0u : 0u;
        if (key0 + kTok - 1 > min(w.hi, w.base - 1)) {
          const int t = key0 + tok;
          vis = 0;
          if (active && t <= w.hi) {
            if (t < w.base) {
              vis = ~0u;
            } else {
              const int d = t - w.base;  // a draft's heads see the same
              constexpr uint32_t kHeads = HQ == 32 ? ~0u : (1u << (HQ % 32)) - 1;
#pragma unroll
              for (int r = 0; r < 32; r += HQ) vis |= ((rows[r].drafts >> d) & 1 ? kHeads : 0u) << r;
            }
          }
        }
        if (vis != ~0u) {
#pragma unroll
          for (int r = 0; r < 32; ++r)
            if (!((vis >> r) & 1)) x[r] = -INFINITY;
        }
        // A thread that asks for a new reference tags the flag of this tile's
        // parity; the other parity's may meanwhile be written for the next tile.
        bool need = false;
        const bool first = j == 0;
        if (!first) {
#pragma unroll
          for (int r = 0; r < 32; ++r) need |= fmaf(x[r], a.scale_log2, -sm.m[row0 + r]) > kRaise;
        }
        if (need) sm.flag[grp][sb] = static_cast<int32_t>(gi + 1);
        all = group_all(1 + grp, ok);
        if (!all) break;
        bool waited = false;
        if (first || sm.flag[grp][sb] == static_cast<int32_t>(gi + 1)) {
          float y[32];
#pragma unroll
          for (int r = 0; r < 32; ++r) y[r] = x[r];
          row_fold<32, true>(y, lane);
          sm.red[grp][quad][lane] = y[0];
          softmax_bar(grp);
          if (gtid < 32) {
            const float mx =
                fmaxf(fmaxf(sm.red[grp][0][gtid], sm.red[grp][1][gtid]), fmaxf(sm.red[grp][2][gtid], sm.red[grp][3][gtid])) * a.scale_log2;
            const float mo = first ? kUnset : sm.m[row0 + gtid];
            const float mn = mx != -INFINITY && mx > mo + kRaise ? mx - kBelow : mo;
            sm.m[row0 + gtid] = mn;
            sm.alpha[row0 + gtid] = ex2(mo - mn);
          }
          softmax_bar(grp);
          if (!first) {
            bool rescale = false;
#pragma unroll
            for (int r = 0; r < 32; ++r) {
              const float al = sm.alpha[row0 + r];
              l_acc[r] *= al;
              rescale |= al != 1.f;
            }
            if (rescale) {
              // O^T *= alpha per row, once P.V of the tile before is done
              ok = ok && warp_wait(&sm.p_free, (gi - 1) & 1, st);
              waited = true;
              tc::fence_after();
#pragma unroll 1
              for (int c = 0; c < 4 * T::kTerms; ++c) {
                uint32_t o[32];
                tc::ld32(o_addr + NR * c, o);
                tc::wait_ld();
#pragma unroll
                for (int r = 0; r < 32; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * sm.alpha[row0 + r]);
                tc::st_cols(o_addr + NR * c, o);
              }
              tc::wait_st();
            }
          }
        }
        // p = 2^(s scale - m), rounded for the product; l sums it as rounded, so
        // that numerator and denominator round alike
        constexpr int kRB = 32 / T::kRowsPerBlk;
        uint32_t words[T::kTerms][kRB][4];
#pragma unroll
        for (int rb = 0; rb < kRB; ++rb) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (kE4) {
              const int r = 16 * rb + 4 * k;
              float p[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) p[i] = ex2(fmaf(x[r + i], a.scale_log2, -sm.m[row0 + r + i]));
              uint32_t w3[3];
              float used[4];
              tc::split_e5m2(p[0], p[1], p[2], p[3], w3, used);
#pragma unroll
              for (int i = 0; i < 4; ++i) l_acc[r + i] += used[i];
#pragma unroll
              for (int t = 0; t < 3; ++t) words[t][rb][k] = w3[t];
            } else {
              const int r = 8 * rb + 2 * k;
              const float p0 = ex2(fmaf(x[r], a.scale_log2, -sm.m[row0 + r]));
              const float p1 = ex2(fmaf(x[r + 1], a.scale_log2, -sm.m[row0 + r + 1]));
              __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
              l_acc[r] += __low2float(pb);
              l_acc[r + 1] += __high2float(pb);
              words[0][rb][k] = *reinterpret_cast<uint32_t*>(&pb);
            }
          }
        }
        // into shared memory once P.V of the tile before has read its P
        if (gi >= 1 && !waited) ok = ok && warp_wait(&sm.p_free, (gi - 1) & 1, st);
        uint8_t* dst = sm.p + (tok >> 3) * (T::kNT / T::kRowsPerBlk * 128) + (tok & 7) * 16;
        if (active) {
#pragma unroll
          for (int t = 0; t < T::kTerms; ++t)
#pragma unroll
            for (int rb = 0; rb < kRB; ++rb)
              *reinterpret_cast<uint4*>(dst + (t * kRB + rb + kRB * grp) * 128) =
                  make_uint4(words[t][rb][0], words[t][rb][1], words[t][rb][2], words[t][rb][3]);
        }
        fence_proxy_async_smem();
        tc::fence_before();
        mbar_arrive(&sm.p_ready);
      }
      if (!all) break;
      // ---- epilogue: l over the threads, then O^T by dims
      row_fold<32, false>(l_acc, lane);
      sm.red[grp][quad][lane] = l_acc[0];
      all = group_all(1 + grp, ok);
      if (!all) break;
      if (gtid < 32) {
        const float l = ((sm.red[grp][0][gtid] + sm.red[grp][1][gtid]) + sm.red[grp][2][gtid]) + sm.red[grp][3][gtid];
        sm.inv[row0 + gtid] = w.nc > 1 ? 1.f : l > 0.f ? 1.f / l : 0.f;
        if (w.nc > 1 && row0 + gtid < w.n * HQ)  // once per half of the dims: their parts are apart
#pragma unroll
          for (int half = 0; half < 2; ++half)
            a.part_ml[(2 * static_cast<int64_t>(u) + half) * a.part_rows + row0 + gtid] =
                make_float2(sm.m[row0 + gtid] == kUnset ? -INFINITY : sm.m[row0 + gtid], l);
      }
      softmax_bar(grp);
      ok = warp_wait(&sm.o_done, wt & 1, st);
      if (!ok) continue;  // to the next unit's vote
      tc::fence_after();
#pragma unroll 1
      for (int blk = 0; blk < 4; ++blk) {
        float o[32];
        {
          uint32_t y[T::kTerms][32];
#pragma unroll
          for (int t = 0; t < T::kTerms; ++t) tc::ld32(o_addr + T::kNT * blk + NR * t, y[t]);
          tc::wait_ld();
#pragma unroll
          for (int r = 0; r < 32; ++r) {
            o[r] = __uint_as_float(y[0][r]);
#pragma unroll
            for (int t = 1; t < T::kTerms; ++t) o[r] += __uint_as_float(y[t][r]);
            o[r] *= sm.inv[row0 + r];
          }
        }
        const int dim = 128 * blk + gtid, count = w.n * HQ;
        if (w.nc > 1) {
          // a part's columns by eights, [8-column block 32][row][8]
          float* part =
              a.part_o + ((2 * static_cast<int64_t>(u) + dim / 256) * 32 + dim % 256 / 8) * a.part_rows * 8 + dim % 8;
#pragma unroll
          for (int r = 0; r < 32; ++r)
            if (row0 + r < count) part[8 * (row0 + r)] = o[r];
        } else {
          __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + static_cast<int64_t>(w.row0) * HQ * 512 + dim;
#pragma unroll
          for (int r = 0; r < 32; ++r)
            if (row0 + r < count) out[(row0 + r) * 512] = __float2bfloat16_rn(o[r]);
        }
      }
    }
  }

  tc::fence_before();
  __syncthreads();
  if (warp == 6) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

template <int LAYOUT, int HQ, int NR>
cudaError_t launch_nr(const LocalArgs& a, cudaStream_t st) {
  auto kern = global_tree_kernel<LAYOUT, HQ, NR>;
  const size_t smem = sizeof(FSmem<LAYOUT, NR>);
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid_ctas()), dim3(FL<LAYOUT, NR>::kThreads), smem, st, a);
}

template <int LAYOUT, int HQ>
cudaError_t launch_lh(const LocalArgs& a, cudaStream_t st) {
  if constexpr (tree_few_rows(LAYOUT) == 64)
    if (a.max_q_rows * HQ > 32) return launch_nr<LAYOUT, HQ, 64>(a, st);
  return launch_nr<LAYOUT, HQ, 32>(a, st);
}

template <int LAYOUT>
cudaError_t launch_l(const LocalArgs& a, cudaStream_t st) {
  switch (a.num_q_heads) {
    case 8: return launch_lh<LAYOUT, 8>(a, st);
    case 16: return launch_lh<LAYOUT, 16>(a, st);
    case 32: return launch_lh<LAYOUT, 32>(a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_global_tree_few(int layout, const LocalArgs& a, cudaStream_t st) {
  if (layout == GW_LAYOUT_GLOBAL_FOLDED_E4M3) return launch_l<GW_LAYOUT_GLOBAL_FOLDED_E4M3>(a, st);
  return layout == GW_LAYOUT_GLOBAL_FOLDED ? launch_l<GW_LAYOUT_GLOBAL_FOLDED>(a, st)
                                           : launch_l<GW_LAYOUT_GLOBAL_FULL>(a, st);
}

}  // namespace gw
