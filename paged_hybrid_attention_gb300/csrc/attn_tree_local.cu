// Attention of drafted trees on LOCAL layers (gw_tree_attn_local), on the
// tensor cores (tcgen05): head dim 256, bf16 or e4m3 pools, trees of up to 32
// rows x heads of a KV head (attn_tree_local_rows.cu has the others).
//
// Row r of a sequence's n <= 64 rows, at position pos_r, sees the cached tokens
// j < L - n with j > pos_r - W and the drafts of its mask word whose positions
// are in the window.  A unit is (sequence, KV head, chunk of tiles).  A tree has few
// rows, so that the cached tokens are the products' long side and the rows their
// columns:
//   S^T[T x NR]    = K_tile[T x 256] . Q^T       (UMMA M = T)
//   O^T[256 x NR] += V_tile^T[256 x T] . P^T     (UMMA M = 128, twice)
// with T = 64 tokens (bf16) or 128 (e4m3) and NR = 16 or 32 rows: an MMA takes
// about as long with 16 columns as with 64, and with the rows along M instead
// (128 of them, a quarter used) a call waited on the MMAs: 61 x 14 rows on the
// e4m3 pool 177 us, 1.1 us per 64 tokens, against 0.72 us of memory.
//
// On e4m3 pools q is two e4m3 terms after an exact power-of-two scaling per row,
// side by side along N, and P three e5m2 terms (tcgen05.cuh), side by side too:
// S and O have a column per row and term, which the softmax and the epilogue add.
//
// K and V arrive by TMA, 128-byte swizzled (2 KB boxes: 16 rows of a page, one
// 128-byte chunk), three stages each, over the units' boundaries; K is the
// K-major, V^T the MN-major A operand as they lie.  At a unit's end the copies and
// the next unit's Q.K^T go on while the softmax warps store O.
// Warp roles (288 threads): 0-3 softmax (a thread per token) and epilogue (a
// thread per dim), 4 and 5 copies of K and V, 6 issues Q.K^T (and owns tensor
// memory), 7 issues P.V, 8 Q rows and what they see.  Every wait is bounded
// (GW_DEV_TIMEOUT).
//
// Bound by memory: 16 sequences of 512 to 8192 tokens, 16 drafts, 16 KV heads of 2,
// window 1024, 49 us (0.82 of the copy rate); e4m3, 61 sequences, 7 drafts 91 us
// (0.85); 64 sequences, 4 drafts 155 us (1.0).
#include "attn_tree.cuh"
#include "tma.cuh"

namespace gw {
namespace {

constexpr int kThreads = 288;
constexpr int kStages = 3;   // K and V tiles in shared memory, each
constexpr int kTileBytes = 32768;
constexpr float kUnset = -1e38f;  // reference of a row that has seen no key

template <int DT, int NR>
struct LT {
  static constexpr bool kE4 = DT == GW_KV_E4M3;
  static constexpr int kTok = kE4 ? 128 : 64;     // tokens of a tile
  static constexpr int kPages = kTok / kPage;
  static constexpr int kC = kE4 ? 2 : 4;          // 128-byte chunks of a row
  static constexpr int kPlane = kTok * 128;       // one chunk column of a tile
  static constexpr int kTerms = kE4 ? 3 : 1;      // of P
  static constexpr int kNT = NR * kTerms;         // N of P.V
  static constexpr int kSCols = kE4 ? 2 * NR : NR;  // N of Q.K^T
  static constexpr int kOBase = 2 * kSCols;       // O's columns, behind the buffers of S
  static constexpr int kRowsPerBlk = kE4 ? 16 : 8;  // rows in 16 bytes of P
};

template <int DT, int NR>
struct LSmem {
  using T = LT<DT, NR>;
  uint8_t k[kStages][kTileBytes];
  uint8_t v[kStages][kTileBytes];
  uint8_t q[NR * 512];  // bf16 [NR / 8][32][8][16 B]; e4m3 [hi, lo][NR / 8][16][8][16 B]
  uint8_t p[T::kTok * T::kNT * (T::kE4 ? 1 : 2)];  // P^T [8 tokens][16-byte block of rows][8][16 B]
  TreeRow rows[kRowRing][NR];
  float m[NR], alpha[NR], inv[NR], red[4][32];
  uint64_t kfull[kStages], kempty[kStages], vfull[kStages], vempty[kStages];
  uint64_t s_ready[2], s_free[2], p_ready, p_free, o_done, q_full, q_free;
  int32_t kmask[kStages], vmask[kStages];  // pages of the tile that were loaded
  int32_t kmax[kRowRing];                  // the first token that every row sees
  int32_t flag[2];  // by tile parity: index + 1 of the last tile that asked for a new reference
  uint32_t tmem_base;
  TreePlan plan;
};
static_assert(sizeof(LSmem<GW_KV_BF16, 32>) <= 232448, "shared memory of one CTA");
static_assert(sizeof(LSmem<GW_KV_E4M3, 32>) <= 232448, "shared memory of one CTA");

__device__ __forceinline__ void softmax_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// Zero the rows r of a K or V stage for which want(r).
template <class T, class Want>
__device__ __forceinline__ void zero_rows(uint32_t base, int lane, Want want) {
  constexpr int kU = T::kC * 8;  // 16-byte units per row
  for (int idx = lane; idx < T::kTok * kU; idx += 32) {
    const int r = idx / kU, u = idx % kU;
    if (want(r)) zero16(base + (u >> 3) * T::kPlane + r * 128 + (u & 7) * 16);
  }
}

// x[r] of row r reduced over a warp's lanes, lane l getting row l % NR's: lanes
// 16 apart first, then, each lane keeping half of its rows, 8, 4, 2 and 1, so that
// the order is the same for 16 rows and 32.  x is used up.
template <int NR, bool kMax>
__device__ __forceinline__ float row_reduce(float (&x)[NR], int lane) {
  if constexpr (NR == 16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float recv = __shfl_xor_sync(0xffffffffu, x[i], 16);
      x[i] = kMax ? fmaxf(x[i], recv) : x[i] + recv;
    }
  }
  row_fold<NR, kMax>(x, lane);
  return x[0];
}

template <int N>
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 16)
    tc::ld16(taddr, r);
  else
    tc::ld32(taddr, r);
}

struct Unit {
  int s, g, rows, n, nc, base, lo, hi, t0, nt, row0;
};

template <int DT, int G>
__device__ __forceinline__ Unit unit_of(const LocalArgs& a, const TreePlan& plan, int u) {
  constexpr int kTok = LT<DT, 32>::kTok;
  Unit w;
  const int at = plan_seq(plan.ub, a.batch, u);
  w.s = plan.seq[at];
  w.row0 = a.cu_q_rows[w.s];
  w.n = a.cu_q_rows[w.s + 1] - w.row0;
  const int L = a.seq_lens[w.s];
  w.base = L - w.n;
  const TreeSpan sp = tree_span(L, w.n, a.window, tree_rule_local(G));
  w.nc = sp.chunks();
  const int r = u - plan.ub[at], c = r % w.nc;  // one block of rows
  w.g = r / w.nc;
  w.rows = w.n * G;
  const int first = sp.first + c * sp.ct, tiles = min(sp.ct, sp.tiles - c * sp.ct);
  w.t0 = first * kTreeTile;  // the first tile's first token
  w.nt = (tiles * kTreeTile + kTok - 1) / kTok;
  w.lo = max(max(0, w.base - a.window + 1), w.t0);
  w.hi = min(L, (first + tiles) * kTreeTile) - 1;
  return w;
}

template <int DT, int G, int NR>
__global__ void __launch_bounds__(kThreads, 1)
    local_tree_kernel(const LocalArgs a, const __grid_constant__ CUtensorMap kv_map) {
  using T = LT<DT, NR>;
  using SM = LSmem<DT, NR>;
  constexpr bool kE4 = T::kE4;
  constexpr float kBelow = Reference<kE4>::kBelow, kRaise = Reference<kE4>::kRaise;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  SM& sm = *reinterpret_cast<SM*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  int32_t* st = a.status;

  if (tid == 0) {
    for (int b = 0; b < kStages; ++b) {
      mbar_init(&sm.kfull[b], 1);
      mbar_init(&sm.kempty[b], 1);
      mbar_init(&sm.vfull[b], 1);
      mbar_init(&sm.vempty[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.s_ready[b], 1);
      mbar_init(&sm.s_free[b], 128);
      sm.flag[b] = 0;
    }
    mbar_init(&sm.p_ready, 128);
    mbar_init(&sm.p_free, 1);
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_free, 1);
    fence_mbar_init();
  }
  if (warp == 6) {
    tc::alloc(&sm.tmem_base, 512);
    tc::relinquish();
  }
  pdl_wait();
  pdl_trigger();
  plan_tree(a, sm.plan, a.kv_heads, tree_rule_local(G), 256);
  const int total = sm.plan.ub[a.batch];
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp == 4 || warp == 5) {
    // ------------------------------------------------------ TMA producers
    // lane l < 16 issues the copy of page l / kC, 128-byte chunk l % kC
    const bool is_v = warp == 5;
    const uint64_t pol = policy_evict_first();
    const int j = lane / T::kC, c = lane % T::kC;
    uint32_t gi = 0;
    int wt = 0;
    bool ok = true;
    for (int u = tree_unit(0); u < total && ok; u = tree_unit(++wt)) {
      const Unit w = unit_of<DT, G>(a, sm.plan, u);
      const int32_t* bt = a.block_table + static_cast<int64_t>(w.s) * a.max_pages;
      for (int t = 0; t < w.nt; ++t, ++gi) {
        const int b = gi % kStages;
        const uint32_t use = gi / kStages;
        int32_t row = -1;
        if (j < T::kPages) {
          const int k0 = w.t0 + t * T::kTok + j * kPage;
          if (k0 + kPage - 1 >= w.lo && k0 <= w.hi) {
            const int32_t pg = bt[k0 / kPage];
            if (pg >= 0 && pg < a.num_pages)
              row = (pg * a.kv_heads + w.g) * 2 * kPage + (is_v ? kPage : 0);
            else if (c == 0)
              set_status(st, GW_DEV_PAGE_RANGE);
          }
        }
        const uint32_t loaded = __ballot_sync(0xffffffffu, row >= 0 && c == 0);  // bit kC j: page j
        int mask = 0;
#pragma unroll
        for (int q = 0; q < T::kPages; ++q) mask |= ((loaded >> (T::kC * q)) & 1) << q;
        uint64_t* full = is_v ? &sm.vfull[b] : &sm.kfull[b];
        uint64_t* empty = is_v ? &sm.vempty[b] : &sm.kempty[b];
        if (use > 0 && !warp_wait(empty, (use - 1) & 1, st)) { ok = false; break; }
        if (lane == 0) {
          if (is_v) sm.vmask[b] = mask; else sm.kmask[b] = mask;
          mbar_arrive_expect_tx(full, static_cast<uint32_t>(__popc(mask)) * T::kC * 2048);
        }
        __syncwarp();
        if (row >= 0)
          tma_rows(smem_u32(is_v ? sm.v[b] : sm.k[b]) + c * T::kPlane + j * 2048, &kv_map, c, row, full, pol);
      }
    }
    drain<kStages>(is_v ? sm.vfull : sm.kfull, gi);
  } else if (warp == 6) {
    // ---------------------------------------------------- Q.K^T issue
    const uint32_t id_s =
        kE4 ? tc::idesc_e4m3(128, 2 * NR, false, false) : tc::idesc_bf16(64, NR, false, false);
    // Q: 16-byte blocks 128 B apart, then the next 8 rows (of a term, then of the next)
    const uint64_t dq = tc::smem_desc(smem_u32(sm.q), 128, (kE4 ? 16 : 32) * 128);
    uint32_t gi = 0;
    int wt = 0;
    bool ok = true;
    for (int u = tree_unit(0); u < total && ok; u = tree_unit(++wt)) {
      const Unit w = unit_of<DT, G>(a, sm.plan, u);
      if (!warp_wait(&sm.q_full, wt & 1, st)) break;
      for (int j = 0; j < w.nt; ++j, ++gi) {
        const int b = gi % kStages, sb = gi & 1;
        if (!warp_wait(&sm.kfull[b], (gi / kStages) & 1, st)) { ok = false; break; }
        if (gi >= 2 && !warp_wait(&sm.s_free[sb], ((gi >> 1) - 1) & 1, st)) { ok = false; break; }
        const uint32_t ka = smem_u32(sm.k[b]);
        const int mask = sm.kmask[b];
        if (mask != (1 << T::kPages) - 1) {  // pages not loaded: zeros, no stale bytes
          zero_rows<T>(ka, lane, [&](int r) { return ((mask >> (r / kPage)) & 1) == 0; });
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc::fence_after();
        // a K-step is 32 bytes of each token's row: 16 bf16 or 32 e4m3 dims
#pragma unroll
        for (int ks = 0; ks < (kE4 ? 8 : 16); ++ks) {
          const uint64_t ad = tc::smem_desc_sw128(ka + (ks >> 2) * T::kPlane + (ks & 3) * 32, 16);
          const uint64_t bd = dq + ((2 * ks * 128) >> 4);
          if constexpr (kE4)
            tc::mma_e4m3_warp(tmem + T::kSCols * sb, ad, bd, id_s, ks > 0);
          else
            tc::mma_bf16_warp(tmem + T::kSCols * sb, ad, bd, id_s, ks > 0);
        }
        tc::commit_warp(&sm.kempty[b]);
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
    const uint64_t dp = tc::smem_desc(smem_u32(sm.p), kGroup, 128);
    uint32_t gi = 0;
    int wt = 0;
    bool ok = true;
    for (int u = tree_unit(0); u < total && ok; u = tree_unit(++wt)) {
      const Unit w = unit_of<DT, G>(a, sm.plan, u);
      const uint32_t o = tmem + T::kOBase;
      for (int j = 0; j < w.nt; ++j, ++gi) {
        const int b = gi % kStages;
        if (!warp_wait(&sm.vfull[b], (gi / kStages) & 1, st)) { ok = false; break; }
        // V rows of tokens outside [lo, hi] or of pages not loaded: zero weights must meet finite values
        const int key0 = w.t0 + j * T::kTok;
        const int mask = sm.vmask[b];
        if (mask != (1 << T::kPages) - 1 || key0 < w.lo || key0 + T::kTok - 1 > w.hi) {
          zero_rows<T>(smem_u32(sm.v[b]), lane, [&](int r) {
            const int key = key0 + r;
            return !(((mask >> (r / kPage)) & 1) && key >= w.lo && key <= w.hi);
          });
          fence_proxy_async_smem();
          __syncwarp();
        }
        // (a unit's first P comes after the last unit's O has been read)
        if (!warp_wait(&sm.p_ready, gi & 1, st)) { ok = false; break; }
        tc::fence_after();
        const uint32_t va = smem_u32(sm.v[b]);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {  // 16 (bf16) or 32 (e4m3) tokens
          const uint64_t bd = dp + ((kk * (kE4 ? 4 : 2) * kGroup) >> 4);
#pragma unroll
          for (int blk = 0; blk < 2; ++blk) {  // 128 dims: two chunks of 64 bf16, or one of e4m3
            const uint64_t ad =
                tc::smem_desc_sw128(va + blk * (kE4 ? 1 : 2) * T::kPlane + kk * (kE4 ? 4096 : 2048), T::kPlane);
            if constexpr (kE4)
              tc::mma_e4m3_warp(o + T::kNT * blk, ad, bd, id_o, !(j == 0 && kk == 0));
            else
              tc::mma_bf16_warp(o + T::kNT * blk, ad, bd, id_o, !(j == 0 && kk == 0));
          }
        }
        tc::commit_warp(&sm.vempty[b]);
        tc::commit_warp(&sm.p_free);
        if (j == w.nt - 1) tc::commit_warp(&sm.o_done);
      }
    }
    drain<1>(&sm.p_free, gi);
  } else if (warp == 8) {
    // -------------------------------------------------------------- Q rows
    // The next unit's rows wait in registers as Q wants them: lane l has rows
    // l % 8 + 8 rb, every fourth 16-byte block from l / 8 on.
    constexpr int kRB = NR / 8, kJ = kE4 ? 4 : 8, kW = kE4 ? 8 : 4;  // words of a block: raw, then of both terms
    uint32_t x[kRB][kJ][kW];
    TreeRow row;
    int kmax = 0;
    auto load = [&](const Unit& w) {
#pragma unroll
      for (int rb = 0; rb < kRB; ++rb) {
        const int r = 8 * rb + (lane & 7);
        const bool ok_row = r < w.rows;
        const uint16_t* src =
            a.q + (static_cast<int64_t>(w.row0 + (ok_row ? r / G : 0)) * a.num_q_heads + w.g * G + r % G) * 256;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const int cb = (lane >> 3) + 4 * j;
#pragma unroll
          for (int h = 0; h < kW / 4; ++h) {
            const uint4 y = ok_row ? *reinterpret_cast<const uint4*>(src + (kE4 ? 16 : 8) * cb + 8 * h)
                                   : make_uint4(0u, 0u, 0u, 0u);
            x[rb][j][4 * h] = y.x, x[rb][j][4 * h + 1] = y.y, x[rb][j][4 * h + 2] = y.z, x[rb][j][4 * h + 3] = y.w;
          }
        }
      }
      // rows behind the last see everything, which costs no masks; nobody reads them
      row = TreeRow{~0ull, 0, 1.f};
      if (lane < w.rows) row = tree_row(a, w.row0, lane / G, w.n, w.base, true);
      kmax = __reduce_max_sync(0xffffffffu, row.kmin);
      if constexpr (kE4) {
#pragma unroll
        for (int rb = 0; rb < kRB; ++rb) {
          float mq = 0.f;
#pragma unroll
          for (int j = 0; j < kJ; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              mq = fmaxf(mq, fmaxf(fabsf(__uint_as_float(x[rb][j][i] << 16)),
                                   fabsf(__uint_as_float(x[rb][j][i] & 0xFFFF0000u))));
          mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, 8));
          mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, 16));
          const int ex = mq > 0.f ? static_cast<int>((__float_as_uint(mq) >> 23) & 0xFF) - 127 : 7;
          const int e = min(125, max(-125, 7 - ex));
          // (an infinity, which the terms cannot hold, makes the row's logits NaN)
          const float up = mq < INFINITY ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : NAN;
          const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          const float mine = __shfl_sync(0xffffffffu, down, lane & 7);  // lanes 0..7 have rows 8 rb ..
          if (lane >> 3 == rb) row.scale = mine;
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            uint32_t h[8], l[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              split_e4m3(__uint_as_float(x[rb][j][i] << 16) * up, __uint_as_float(x[rb][j][i] & 0xFFFF0000u) * up, h[i],
                         l[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[rb][j][i] = h[2 * i] | (h[2 * i + 1] << 16);
              x[rb][j][4 + i] = l[2 * i] | (l[2 * i + 1] << 16);
            }
          }
        }
      }
    };
    auto store = [&](int wt) {
#pragma unroll
      for (int rb = 0; rb < kRB; ++rb)
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const int cb = (lane >> 3) + 4 * j;
          uint8_t* dst = sm.q + (rb * (kE4 ? 16 : 32) + cb) * 128 + (lane & 7) * 16;
#pragma unroll
          for (int h = 0; h < kW / 4; ++h)
            *reinterpret_cast<uint4*>(dst + h * (NR * 256)) =
                make_uint4(x[rb][j][4 * h], x[rb][j][4 * h + 1], x[rb][j][4 * h + 2], x[rb][j][4 * h + 3]);
        }
      if (lane < NR) sm.rows[wt % kRowRing][lane] = row;
      if (lane == 0) sm.kmax[wt % kRowRing] = kmax;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full);
    };
    int wt = 0;
    for (int u = tree_unit(0); u < total; u = tree_unit(++wt)) {
      load(unit_of<DT, G>(a, sm.plan, u));
      if (wt > 0 && !warp_wait(&sm.q_free, (wt - 1) & 1, st)) break;
      store(wt);
    }
  } else {
    // ------------------------------------------------- softmax and epilogue
    const bool active = kE4 || lane < 16;  // M = 64 uses lanes 0..15 of a quadrant
    const int tok = kE4 ? 32 * warp + lane : 16 * warp + lane;
    const uint32_t lane_base = static_cast<uint32_t>(32 * warp) << 16;
    uint32_t gi = 0;
    int wt = 0;
    bool ok = true, all = true;  // this warp's waits; those of the four, as last voted
    for (int u = tree_unit(0); u < total && all; u = tree_unit(++wt)) {
      const Unit w = unit_of<DT, G>(a, sm.plan, u);
      const TreeRow* rows = sm.rows[wt % kRowRing];
      const uint32_t o_addr = tmem + lane_base + T::kOBase;
      float l_acc[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) l_acc[r] = 0.f;
      for (int j = 0; j < w.nt; ++j, ++gi) {
        const int sb = gi & 1;
        ok = ok && warp_wait(&sm.s_ready[sb], (gi >> 1) & 1, st);
        tc::fence_after();
        float x[NR];
        {
          const uint32_t s_addr = tmem + lane_base + T::kSCols * sb;
          uint32_t y[NR];
          ld_cols<NR>(s_addr, y);
          if constexpr (kE4) {
            uint32_t z[NR];
            ld_cols<NR>(s_addr + NR, z);
            tc::wait_ld();
#pragma unroll
            for (int r = 0; r < NR; ++r) x[r] = (__uint_as_float(y[r]) + __uint_as_float(z[r])) * rows[r].scale;
          } else {
            tc::wait_ld();
#pragma unroll
            for (int r = 0; r < NR; ++r) x[r] = __uint_as_float(y[r]);
          }
        }
        tc::fence_before();
        mbar_arrive(&sm.s_free[sb]);
        // rows that see this thread's token
        const int key0 = w.t0 + j * T::kTok;
        uint32_t vis = active ? ~0u : 0u;
        if (!(key0 >= max(w.lo, sm.kmax[wt % kRowRing]) && key0 + T::kTok <= w.base && key0 + T::kTok - 1 <= w.hi)) {
          const int t = key0 + tok;
          vis = 0;
          if (active && t >= w.lo && t <= w.hi) {
            constexpr uint32_t kHeads = (1u << G) - 1;  // a draft's heads see the same
            if (t < w.base) {
#pragma unroll 8
              for (int r = 0; r < NR; r += G) vis |= (t >= rows[r].kmin ? kHeads : 0u) << r;
            } else {
              const int d = t - w.base;
#pragma unroll 8
              for (int r = 0; r < NR; r += G) vis |= ((rows[r].drafts >> d) & 1 ? kHeads : 0u) << r;
            }
          }
        }
        if (vis != ~0u) {
#pragma unroll
          for (int r = 0; r < NR; ++r)
            if (!((vis >> r) & 1)) x[r] = -INFINITY;
        }
        // A thread that asks for a new reference tags the flag of this tile's
        // parity; the other parity's may meanwhile be written for the next tile.
        bool need = false;
        const bool first = j == 0;
        if (!first) {
#pragma unroll
          for (int r = 0; r < NR; ++r) need |= fmaf(x[r], a.scale_log2, -sm.m[r]) > kRaise;
        }
        if (need) sm.flag[sb] = static_cast<int32_t>(gi + 1);
        all = group_all(1, ok);
        if (!all) break;
        bool waited = false;
        if (first || sm.flag[sb] == static_cast<int32_t>(gi + 1)) {
          float y[NR];
#pragma unroll
          for (int r = 0; r < NR; ++r) y[r] = x[r];
          const float top = row_reduce<NR, true>(y, lane);
          if (lane < NR) sm.red[warp][lane] = top;
          softmax_bar();
          if (tid < NR) {
            const float mx =
                fmaxf(fmaxf(sm.red[0][tid], sm.red[1][tid]), fmaxf(sm.red[2][tid], sm.red[3][tid])) * a.scale_log2;
            const float mo = first ? kUnset : sm.m[tid];
            const float mn = mx != -INFINITY && mx > mo + kRaise ? mx - kBelow : mo;
            sm.m[tid] = mn;
            sm.alpha[tid] = ex2(mo - mn);
          }
          softmax_bar();
          if (!first) {
            bool rescale = false;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              const float al = sm.alpha[r];
              l_acc[r] *= al;
              rescale |= al != 1.f;
            }
            if (rescale) {
              // O^T *= alpha per row, once P.V of the tile before is done
              ok = ok && warp_wait(&sm.p_free, (gi - 1) & 1, st);
              waited = true;
              tc::fence_after();
#pragma unroll 1
              for (int c = 0; c < 2 * T::kTerms; ++c) {
                uint32_t o[NR];
                ld_cols<NR>(o_addr + NR * c, o);
                tc::wait_ld();
#pragma unroll
                for (int r = 0; r < NR; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * sm.alpha[r]);
                tc::st_cols(o_addr + NR * c, o);
              }
              tc::wait_st();
            }
          }
        }
        // p = 2^(s scale - m), rounded for the product; l sums it as rounded, so
        // that numerator and denominator round alike
        constexpr int kRB = NR / T::kRowsPerBlk;
        uint32_t words[T::kTerms][kRB][4];
#pragma unroll
        for (int rb = 0; rb < kRB; ++rb) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (kE4) {
              const int r = 16 * rb + 4 * k;
              float p[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) p[i] = ex2(fmaf(x[r + i], a.scale_log2, -sm.m[r + i]));
              uint32_t w3[3];
              float used[4];
              tc::split_e5m2(p[0], p[1], p[2], p[3], w3, used);
#pragma unroll
              for (int i = 0; i < 4; ++i) l_acc[r + i] += used[i];
#pragma unroll
              for (int t = 0; t < 3; ++t) words[t][rb][k] = w3[t];
            } else {
              const int r = 8 * rb + 2 * k;
              const float p0 = ex2(fmaf(x[r], a.scale_log2, -sm.m[r]));
              const float p1 = ex2(fmaf(x[r + 1], a.scale_log2, -sm.m[r + 1]));
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
              *reinterpret_cast<uint4*>(dst + (t * kRB + rb) * 128) =
                  make_uint4(words[t][rb][0], words[t][rb][1], words[t][rb][2], words[t][rb][3]);
        }
        fence_proxy_async_smem();
        tc::fence_before();
        mbar_arrive(&sm.p_ready);
      }
      if (!all) break;
      // ---- epilogue: l over the threads, then O^T by dims
      const float sum = row_reduce<NR, false>(l_acc, lane);
      if (lane < NR) sm.red[warp][lane] = sum;
      all = group_all(1, ok);
      if (!all) break;
      if (tid < NR) {
        const float l = ((sm.red[0][tid] + sm.red[1][tid]) + sm.red[2][tid]) + sm.red[3][tid];
        sm.inv[tid] = w.nc > 1 ? 1.f : l > 0.f ? 1.f / l : 0.f;
        if (w.nc > 1 && tid < w.rows)
          a.part_ml[static_cast<int64_t>(u) * a.part_rows + tid] =
              make_float2(sm.m[tid] == kUnset ? -INFINITY : sm.m[tid], l);
      }
      softmax_bar();
      ok = warp_wait(&sm.o_done, wt & 1, st);
      if (!ok) continue;  // to the next unit's vote
      tc::fence_after();
#pragma unroll 1
      for (int blk = 0; blk < 2; ++blk) {
        float o[NR];
        {
          uint32_t y[T::kTerms][NR];
#pragma unroll
          for (int t = 0; t < T::kTerms; ++t) ld_cols<NR>(o_addr + T::kNT * blk + NR * t, y[t]);
          tc::wait_ld();
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            o[r] = __uint_as_float(y[0][r]);
#pragma unroll
            for (int t = 1; t < T::kTerms; ++t) o[r] += __uint_as_float(y[t][r]);
            o[r] *= sm.inv[r];
          }
        }
        const int dim = 128 * blk + 32 * warp + lane;
        if (w.nc > 1) {
          // a part's columns by eights, [8-column block 32][row][8]
          float* part = a.part_o + ((static_cast<int64_t>(u) * 32 + dim / 8) * a.part_rows) * 8 + dim % 8;
#pragma unroll
          for (int r = 0; r < NR; ++r)
            if (r < w.rows) part[8 * r] = o[r];
        } else {
          __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) +
                               (static_cast<int64_t>(w.row0) * a.num_q_heads + w.g * G) * 256 + dim;
#pragma unroll
          for (int r = 0; r < NR; ++r)
            if (r < w.rows) out[(static_cast<int64_t>(r / G) * a.num_q_heads + r % G) * 256] = __float2bfloat16_rn(o[r]);
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

template <int DT, int G, int NR>
cudaError_t launch_nr(const LocalArgs& a, cudaStream_t st) {
  CUtensorMap map;
  cudaError_t e = make_local_kv_map(a, &map, DT);
  if (e != cudaSuccess) return e;
  auto kern = local_tree_kernel<DT, G, NR>;
  const size_t smem = sizeof(LSmem<DT, NR>);
  e = set_smem_once(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid_ctas()), dim3(kThreads), smem, st, a, map);
}

// 16 rows where no sequence of the call has more: half the softmax of 32.
template <int DT, int G>
cudaError_t launch_g(const LocalArgs& a, cudaStream_t st) {
  return a.max_q_rows * G <= 16 ? launch_nr<DT, G, 16>(a, st) : launch_nr<DT, G, 32>(a, st);
}

template <int DT>
cudaError_t launch_dt(int group, const LocalArgs& a, cudaStream_t st) {
  switch (group) {
    case 1: return launch_g<DT, 1>(a, st);
    case 2: return launch_g<DT, 2>(a, st);
    case 4: return launch_g<DT, 4>(a, st);
    case 8: return launch_g<DT, 8>(a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_local_tree_few(int dtype, int group, const LocalArgs& a, cudaStream_t st) {
  return dtype == GW_KV_E4M3 ? launch_dt<GW_KV_E4M3>(group, a, st) : launch_dt<GW_KV_BF16>(group, a, st);
}

}  // namespace gw
