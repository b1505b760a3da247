// Attention of drafted trees on LOCAL layers (gw_tree_attn_local), on the
// tensor cores (tcgen05): head dim 256, bf16 or e4m3 pools, calls whose sequences
// may have more than 32 rows x heads of a KV head (attn_tree_local.cu has the others).
//
// Row r of a sequence's n <= 64 rows, at position pos_r, sees the cached tokens
// j < L - n with j > pos_r - W and the drafts of its mask word whose positions
// are in the window.  A unit is (sequence, KV head, block of 128 / G rows, chunk
// of 64-token tiles); per tile, with the G heads' rows together,
//   S[128 x 64]   = Q[128 x 256] . K^T      (UMMA M = 128, N = 64)
//   O[128 x 256] += P[128 x 64] . V         (UMMA M = 128, N = 256)
// The cache is read once for all rows of a KV head: 64 drafts of 2 heads are 128
// flop/B, so a call should stream at the memory's rate.  16 sequences of 512 to
// 8192 tokens, 64 drafts, 16 KV heads of 2: 58 us, 0.78 of the copy rate; e4m3 71 us
// (0.35), which waits on the MMAs of q's two terms and P's three and rescales O more
// often (Reference).  What stands in
// the way:
//
// - Softmax.  A sequence's n G rows need not fill the 128, and a warp reaches only
//   its own 32 lanes of tensor memory.  So up to 32 (64) rows are laid out four
//   times (twice), once per 32 (64) lanes, and a copy's threads take a quarter
//   (half) of a tile's keys, writing P = 0 for the others: the copies are the
//   same rows over different keys, each with its own (m, l), and are merged in
//   the epilogue.  A thread's work per tile is 16 keys instead of 64.
// - A unit's end.  Loading the next rows of Q and storing O took the softmax
//   warps 5 us per unit; here four other warps do both, so that the next unit's
//   first tiles go through Q.K^T and softmax meanwhile, and only its first P.V
//   waits until O has been read.
//
// K and V arrive by TMA, 128-byte swizzled (2 KB boxes: 16 rows of a page, one
// 128-byte chunk), three stages each, over the units' boundaries.  Q and P live
// in tensor memory: S at columns 0 and 64 (P over them), Q at 128, O at 256.
// On e4m3 pools a q row is two e4m3 terms after an exact power-of-two scaling,
// and P three e5m2 terms.
// Warp roles (384 threads): 0-3 softmax, 4-7 Q rows and epilogue, 8 and 9 copies
// of K and V, 10 issues Q.K^T (and owns tensor memory), 11 issues P.V.  Every
// wait is bounded (GW_DEV_TIMEOUT).
#include "attn_tree.cuh"
#include "tma.cuh"

namespace gw {
namespace {

constexpr int kM = 128, kN = 64;
constexpr int kThreads = 384;
constexpr uint32_t kColS = 0, kColQ = 128, kColO = 256;
constexpr uint32_t kPlane = kN * 128;  // one 128-byte chunk column of a tile
constexpr int kStages = 3;             // K and V tiles in shared memory, each

template <int DT>
struct LSmem {
  static constexpr int kC = DT == GW_KV_BF16 ? 4 : 2;  // 128-byte chunks of a row
  uint8_t k[kStages][kC * kPlane];
  uint8_t v[kStages][kC * kPlane];
  float merge[kM * 36];         // 32 columns of O, rows padded against bank conflicts
  TreeRow rows[kRowRing][kM];   // the keys each lane's row sees
  float2 stat[2][kM];           // (m, l) of each lane, by unit parity
  // e4m3: the next unit's Q rows, q_hi then q_lo, each lane's own
  static constexpr int kQRow = 528;
  uint8_t qstage[DT == GW_KV_E4M3 ? kM * kQRow : 16];
  uint64_t kfull[kStages], kempty[kStages], vfull[kStages], vempty[kStages];
  uint64_t s_ready[2], p_ready[2], pfree[2], stat_full[2], stat_free[2];
  uint64_t q_full, q_free, o_done, o_free;
  int32_t kmask[kStages], vmask[kStages];  // pages of the tile that were loaded
  uint32_t tmem_base;
  TreePlan plan;
};
static_assert(sizeof(LSmem<GW_KV_BF16>) <= 232448, "shared memory of one CTA");

// Zero the rows r of a K or V stage for which want(r).
template <int DT, class Want>
__device__ __forceinline__ void zero_rows(uint32_t base, int lane, Want want) {
  constexpr int kU = LSmem<DT>::kC * 8;  // 16-byte units per row
  for (int idx = lane; idx < kN * kU; idx += 32) {
    const int r = idx / kU, u = idx % kU;
    if (want(r)) zero16(base + (u >> 3) * kPlane + r * 128 + (u & 7) * 16);
  }
}
__device__ __forceinline__ void store_f32x8(float* dst, const float* x) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(x[0]), "f"(x[1]), "f"(x[2]),
               "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}

struct Unit {
  int s, g, q0, rows, copies, n, nc, base, lo, hi, t_lo, nt, row0;
};

// Unit u.  Row blocks of a chunk are neighbours, so that its K and V come from
// L2 for all but the first.
template <int G>
__device__ __forceinline__ Unit unit_of(const LocalArgs& a, const TreePlan& plan, int u) {
  constexpr int BQ = kM / G;
  Unit w;
  const int at = plan_seq(plan.ub, a.batch, u);
  w.s = plan.seq[at];
  w.row0 = a.cu_q_rows[w.s];
  w.n = a.cu_q_rows[w.s + 1] - w.row0;
  const int L = a.seq_lens[w.s];
  w.base = L - w.n;
  const TreeSpan sp = tree_span(L, w.n, a.window, tree_rule_local(G));
  w.nc = sp.chunks();
  const int r = u - plan.ub[at], gc = r / sp.blocks, c = gc % w.nc;
  w.g = gc / w.nc;
  w.q0 = (r - gc * sp.blocks) * BQ;
  w.rows = min(BQ, w.n - w.q0) * G;
  w.copies = w.rows <= 32 ? 4 : w.rows <= 64 ? 2 : 1;
  w.t_lo = sp.first + c * sp.ct;
  w.nt = min(sp.ct, sp.tiles - c * sp.ct);
  w.lo = max(max(0, w.base - a.window + 1), w.t_lo * kN);
  w.hi = min(L, (w.t_lo + w.nt) * kN) - 1;
  return w;
}

// Row (of the unit's rows) that a lane of tensor memory holds: row i is draft
// q0 + i / G of head g G + i % G.
__device__ __forceinline__ int row_of(const Unit& w, int lane128) { return lane128 & (kM / w.copies - 1); }

// One tile's softmax for a thread whose row's copy takes keys [KN share, KN
// (share + 1)) of it: S from tensor memory, P back over it, zeros for the other
// copies' keys.  False if a wait gave up.
template <int DT, int COPIES>
__device__ __forceinline__ bool softmax_tile(uint32_t s_addr, uint32_t o_addr, int share, uint64_t seen, bool all,
                                             float sc, float& m_ref, float (&lp)[4], uint64_t* pfree_before,
                                             uint32_t before_parity, int32_t* st) {
  constexpr bool kE4 = DT == GW_KV_E4M3;
  constexpr int KN = kN / COPIES;
  uint32_t sv[KN];
  if constexpr (KN == 16) {
    tc::ld16(s_addr + KN * share, sv);
  } else {
#pragma unroll
    for (int c = 0; c < KN; c += 32)
      tc::ld32(s_addr + KN * share + c, *reinterpret_cast<uint32_t(*)[32]>(&sv[c]));
  }
  tc::wait_ld();
  if (!all) {
    const uint64_t m = seen >> (KN * share);
    const uint32_t m0 = static_cast<uint32_t>(m), m1 = static_cast<uint32_t>(m >> 32);
#pragma unroll
    for (int c = 0; c < KN; ++c)
      if (!(((c < 32 ? m0 : m1) >> (c & 31)) & 1)) sv[c] = __float_as_uint(-INFINITY);
  }
  float mg[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    mg[i] = __uint_as_float(sv[i]);
#pragma unroll
    for (int c = 4 + i; c < KN; c += 4) mg[i] = fmaxf(mg[i], __uint_as_float(sv[c]));
  }
  const float mx = fmaxf(fmaxf(mg[0], mg[1]), fmaxf(mg[2], mg[3])) * sc;  // -inf stays -inf (sc > 0)
  constexpr float kBelow = Reference<kE4>::kBelow;
  const bool raise = mx > m_ref + Reference<kE4>::kRaise;  // false while the copy has no key
  if (__any_sync(0xffffffffu, raise)) {
    const float m_new = raise ? mx - kBelow : m_ref;
    const float alpha = m_ref == -INFINITY ? 0.f : ex2(m_ref - m_new);
    if (__any_sync(0xffffffffu, raise && m_ref != -INFINITY)) {
      // O *= alpha for this warp's rows once P.V of the tile before is done
      if (!warp_wait(pfree_before, before_parity, st)) return false;
      tc::fence_after();
#pragma unroll 1
      for (int blk = 0; blk < 8; ++blk) {
        uint32_t o[32];
        tc::ld32(o_addr + 32 * blk, o);
        tc::wait_ld();
        if (raise && m_ref != -INFINITY) {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
        }
        __syncwarp();
        tc::st32(o_addr + 32 * blk, o);
      }
      tc::wait_st();
    }
    if (raise) {
#pragma unroll
      for (int i = 0; i < 4; ++i) lp[i] *= alpha;
      m_ref = m_new;
    }
  }
  // p = 2^(s sc - m), rounded for the product; l sums it as rounded, so that
  // numerator and denominator round alike
  const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
  if constexpr (kE4) {
    // three e5m2 terms at columns 0, 16 and 32, 4 keys a column
    uint32_t pt[3][KN / 4];
#pragma unroll
    for (int u = 0; u < KN / 4; ++u) {
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = ex2(fmaf(__uint_as_float(sv[4 * u + i]), sc, neg_m));
      uint32_t w3[3];
      float held[4];
      tc::split_e5m2(p[0], p[1], p[2], p[3], w3, held);
      lp[u & 3] += (held[0] + held[1]) + (held[2] + held[3]);
#pragma unroll
      for (int t = 0; t < 3; ++t) pt[t][u] = w3[t];
    }
#pragma unroll
    for (int t = 0; t < 3; ++t)
#pragma unroll
      for (int c = 0; c < COPIES; ++c) {
        uint32_t x[KN / 4];
#pragma unroll
        for (int i = 0; i < KN / 4; ++i) x[i] = c == share ? pt[t][i] : 0u;
        tc::st_cols(s_addr + 16 * t + KN / 4 * c, x);
      }
  } else {
    uint32_t pw[KN / 2];
#pragma unroll
    for (int u = 0; u < KN / 2; ++u) {
      const float p0 = ex2(fmaf(__uint_as_float(sv[2 * u]), sc, neg_m));
      const float p1 = ex2(fmaf(__uint_as_float(sv[2 * u + 1]), sc, neg_m));
      __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
      lp[u & 3] += __low2float(pb) + __high2float(pb);
      pw[u] = *reinterpret_cast<uint32_t*>(&pb);
    }
#pragma unroll
    for (int c = 0; c < COPIES; ++c) {
      uint32_t x[KN / 2];
#pragma unroll
      for (int i = 0; i < KN / 2; ++i) x[i] = c == share ? pw[i] : 0u;
      tc::st_cols(s_addr + KN / 2 * c, x);
    }
  }
  tc::wait_st();
  return true;
}

template <int DT, int G>
__global__ void __launch_bounds__(kThreads, 1)
    local_tree_rows_kernel(const LocalArgs a, const __grid_constant__ CUtensorMap kv_map) {
  constexpr bool kE4 = DT == GW_KV_E4M3;
  using SM = LSmem<DT>;
  constexpr int kC = SM::kC;
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
      mbar_init(&sm.p_ready[b], kM);
      mbar_init(&sm.pfree[b], 1);
      mbar_init(&sm.stat_full[b], kM);
      mbar_init(&sm.stat_free[b], kM);
    }
    mbar_init(&sm.q_full, kM);
    mbar_init(&sm.q_free, 1);
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.o_free, kM);
    fence_mbar_init();
  }
  if (warp == 10) {
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
  const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;

  if (warp == 8 || warp == 9) {
    // ------------------------------------------------------ TMA producers
    // lane l < 4 kC issues the copy of page l / kC, 128-byte chunk l % kC
    const bool is_v = warp == 9;
    const uint64_t pol = policy_evict_first();
    const int j = lane / kC, c = lane % kC;
    uint32_t gi = 0;
    bool ok = true;
    int wt = 0;
    for (int u = tree_unit(0); u < total && ok; u = tree_unit(++wt)) {
      const Unit w = unit_of<G>(a, sm.plan, u);
      const int32_t* bt = a.block_table + static_cast<int64_t>(w.s) * a.max_pages;
      for (int t = 0; t < w.nt; ++t, ++gi) {
        const int b = gi % kStages;
        const uint32_t use = gi / kStages;
        int32_t row = -1;
        if (lane < 4 * kC) {
          const int k0 = (w.t_lo + t) * kN + j * kPage;
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
        for (int q = 0; q < 4; ++q) mask |= ((loaded >> (kC * q)) & 1) << q;
        uint64_t* full = is_v ? &sm.vfull[b] : &sm.kfull[b];
        uint64_t* empty = is_v ? &sm.vempty[b] : &sm.kempty[b];
        if (use > 0 && !warp_wait(empty, (use - 1) & 1, st)) { ok = false; break; }
        if (lane == 0) {
          if (is_v) sm.vmask[b] = mask; else sm.kmask[b] = mask;
          mbar_arrive_expect_tx(full, static_cast<uint32_t>(__popc(mask)) * kC * 2048);
        }
        __syncwarp();
        if (row >= 0)
          tma_rows(smem_u32(is_v ? sm.v[b] : sm.k[b]) + c * kPlane + j * 2048, &kv_map, c, row, full, pol);
      }
    }
    drain<kStages>(is_v ? sm.vfull : sm.kfull, gi);
  } else if (warp == 10) {
    // ---------------------------------------------------- Q.K^T issue
    const uint32_t id_s = kE4 ? tc::idesc_e4m3(kM, kN, false, false) : tc::idesc_bf16(kM, kN, false, false);
    uint32_t gi = 0;
    int wt = 0;
    bool ok = true;
    for (int u = tree_unit(0); u < total && ok; u = tree_unit(++wt)) {
      const Unit w = unit_of<G>(a, sm.plan, u);
      if (!warp_wait(&sm.q_full, wt & 1, st)) break;
      for (int j = 0; j < w.nt; ++j, ++gi) {
        const int b = gi % kStages, sb = gi & 1;
        if (!warp_wait(&sm.kfull[b], (gi / kStages) & 1, st)) { ok = false; break; }
        // this S buffer holds P of tile gi - 2 until its P.V is done
        if (gi >= 2 && !warp_wait(&sm.pfree[sb], ((gi >> 1) - 1) & 1, st)) { ok = false; break; }
        const uint32_t ka = smem_u32(sm.k[b]);
        const int mask = sm.kmask[b];
        if (mask != 0xF) {  // pages not loaded: finite zeros, no stale bytes
          zero_rows<DT>(ka, lane, [&](int r) { return ((mask >> (r / kPage)) & 1) == 0; });
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc::fence_after();
        // a K-step is 32 bytes of each key row: 16 bf16 or 32 e4m3 dims
#pragma unroll
        for (int ks = 0; ks < (kE4 ? 8 : 16); ++ks) {
          const uint64_t bd = tc::smem_desc_sw128(ka + (ks >> 2) * kPlane + (ks & 3) * 32, 16);
          if constexpr (kE4) {  // q_hi at Q columns 0..63, q_lo at 64..127
            tc::mma_e4m3_ts_warp(tmem + kColS + kN * sb, tmem + kColQ + 8 * ks, bd, id_s, ks > 0);
            tc::mma_e4m3_ts_warp(tmem + kColS + kN * sb, tmem + kColQ + 64 + 8 * ks, bd, id_s, true);
          } else {
            tc::mma_bf16_ts_warp(tmem + kColS + kN * sb, tmem + kColQ + 8 * ks, bd, id_s, ks > 0);
          }
        }
        tc::commit_warp(&sm.kempty[b]);
        tc::commit_warp(&sm.s_ready[sb]);
        if (j == w.nt - 1) tc::commit_warp(&sm.q_free);
      }
    }
    drain<2>(sm.s_ready, gi);
  } else if (warp == 11) {
    // ------------------------------------------------------- P.V issue
    const uint32_t id_o = kE4 ? tc::idesc_e5m2_e4m3(kM, 256, false, true) : tc::idesc_bf16(kM, 256, false, true);
    uint32_t gi = 0;
    int wt = 0;
    bool ok = true;
    for (int u = tree_unit(0); u < total && ok; u = tree_unit(++wt)) {
      const Unit w = unit_of<G>(a, sm.plan, u);
      for (int j = 0; j < w.nt; ++j, ++gi) {
        const int b = gi % kStages, sb = gi & 1;
        if (j == 0 && wt >= 1 && !warp_wait(&sm.o_free, (wt - 1) & 1, st)) { ok = false; break; }
        if (!warp_wait(&sm.vfull[b], (gi / kStages) & 1, st)) { ok = false; break; }
        // V rows of keys outside [lo, hi] or of pages not loaded: zero weights must meet finite values
        const int key0 = (w.t_lo + j) * kN;
        const int mask = sm.vmask[b];
        if (mask != 0xF || key0 < w.lo || key0 + kN - 1 > w.hi) {
          zero_rows<DT>(smem_u32(sm.v[b]), lane, [&](int kr) {
            const int key = key0 + kr;
            return !(((mask >> (kr >> 4)) & 1) && key >= w.lo && key <= w.hi);
          });
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (!warp_wait(&sm.p_ready[sb], (gi >> 1) & 1, st)) { ok = false; break; }
        tc::fence_after();
        const uint32_t va = smem_u32(sm.v[b]), p = tmem + kColS + kN * sb;
        if constexpr (kE4) {
          // K-steps of 32 keys (4 swizzle atoms of 8 rows), P's terms 16 columns apart
#pragma unroll
          for (int kk = 0; kk < kN / 32; ++kk) {
            const uint64_t bd = tc::smem_desc_sw128(va + kk * 4096, kPlane);
#pragma unroll
            for (int t = 0; t < 3; ++t)
              tc::mma_e4m3_ts_warp(tmem + kColO, p + 16 * t + 8 * kk, bd, id_o, !(j == 0 && kk == 0 && t == 0));
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < kN / 16; ++kk)
            tc::mma_bf16_ts_warp(tmem + kColO, p + 8 * kk, tc::smem_desc_sw128(va + kk * 2048, kPlane), id_o,
                                 !(j == 0 && kk == 0));
        }
        tc::commit_warp(&sm.vempty[b]);
        tc::commit_warp(&sm.pfree[sb]);
        if (j == w.nt - 1) tc::commit_warp(&sm.o_done);
      }
    }
    drain<2>(sm.pfree, gi);
  } else if (warp < 4) {
    // ------------------------------------------------------------ softmax
    uint32_t gi = 0;
    int wt = 0;
    bool ok = true;
    for (int u = tree_unit(0); u < total && ok; u = tree_unit(++wt)) {
      const Unit w = unit_of<G>(a, sm.plan, u);
      const int share = tid / (kM / w.copies);
      // a warp none of whose lanes has a row leaves P as it is: rows do not mix
      const bool idle = row_of(w, 32 * warp) >= w.rows;
      TreeRow row{};
      float sc = 0.f;
      float m_ref = -INFINITY, lp[4] = {0.f, 0.f, 0.f, 0.f};
      for (int j = 0; j < w.nt; ++j, ++gi) {
        const int sb = gi & 1;
        if (!warp_wait(&sm.s_ready[sb], (gi >> 1) & 1, st)) { ok = false; break; }
        tc::fence_after();
        if (!idle) {
          if (j == 0) {  // written before the unit's Q was handed over
            row = sm.rows[wt % kRowRing][tid];
            sc = a.scale_log2 * row.scale;
          }
          const int key0 = (w.t_lo + j) * kN;
          const bool all = key0 >= row.kmin && key0 + kN <= w.base;
          const uint64_t seen = all ? 0 : tree_tile_mask(row, w.base, key0);
          const uint32_t sa = tmem + lane_base + kColS + kN * sb, oa = tmem + lane_base + kColO;
          uint64_t* before = &sm.pfree[(gi - 1) & 1];
          const uint32_t bp = ((gi - 1) >> 1) & 1;
          ok = w.copies == 4 ? softmax_tile<DT, 4>(sa, oa, share, seen, all, sc, m_ref, lp, before, bp, st)
               : w.copies == 2 ? softmax_tile<DT, 2>(sa, oa, share, seen, all, sc, m_ref, lp, before, bp, st)
                               : softmax_tile<DT, 1>(sa, oa, share, seen, all, sc, m_ref, lp, before, bp, st);
          if (!ok) break;
        }
        tc::fence_before();
        mbar_arrive(&sm.p_ready[sb]);
      }
      if (!ok) break;
      if (wt >= 2 && !warp_wait(&sm.stat_free[wt & 1], ((wt >> 1) - 1) & 1, st)) break;
      sm.stat[wt & 1][tid] = make_float2(m_ref, (lp[0] + lp[1]) + (lp[2] + lp[3]));
      mbar_arrive(&sm.stat_full[wt & 1]);
    }
  } else {
    // ------------------------------------------------- Q rows and epilogue
    const int r = tid - kM;  // lane of tensor memory
    // The next unit's Q row of this lane: bf16 in registers as tensor memory wants
    // it; e4m3 in this lane's part of qstage
    uint32_t qv[kE4 ? 1 : 128];
    uint8_t* const stage = sm.qstage + (kE4 ? r * SM::kQRow : 0);
    TreeRow next_row;
    auto load_q = [&](const Unit& w) {
      const int i = row_of(w, r);
      const bool ok_row = i < w.rows;
      next_row = TreeRow{0, 0x7fffffff, 1.f};
      const int qi = w.q0 + i / G, hd = w.g * G + i % G;
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (static_cast<int64_t>(w.row0 + (ok_row ? qi : 0)) * a.num_q_heads + (ok_row ? hd : 0)) * 256);
      if constexpr (kE4) {
        if (ok_row) next_row = tree_row(a, w.row0, qi, w.n, w.base, true);
        float mq = 0.f;
        if (ok_row) {
#pragma unroll 16
          for (int c = 0; c < 32; ++c) {
            const uint4 x = src[c];
            const uint32_t u4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mq = fmaxf(mq, fmaxf(fabsf(__uint_as_float(u4[k] << 16)), fabsf(__uint_as_float(u4[k] & 0xFFFF0000u))));
          }
        }
        const int ex = mq > 0.f ? static_cast<int>((__float_as_uint(mq) >> 23) & 0xFF) - 127 : 7;
        const int e = min(125, max(-125, 7 - ex));
        // (an infinity, which the terms cannot hold, makes the row's logits NaN)
        const float up = mq < INFINITY ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : NAN;
        next_row.scale = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll 2
        for (int c = 0; c < 16; ++c) {  // 16 dims: 16 bytes of each term; the second reading from L1
          uint32_t h[8], l[8];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint4 x = ok_row ? src[2 * c + k] : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t u4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4)
              split_e4m3(__uint_as_float(u4[i4] << 16) * up, __uint_as_float(u4[i4] & 0xFFFF0000u) * up, h[4 * k + i4],
                         l[4 * k + i4]);
          }
          *reinterpret_cast<uint4*>(stage + 16 * c) = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16),
                                                                 h[4] | (h[5] << 16), h[6] | (h[7] << 16));
          *reinterpret_cast<uint4*>(stage + 256 + 16 * c) = make_uint4(l[0] | (l[1] << 16), l[2] | (l[3] << 16),
                                                                       l[4] | (l[5] << 16), l[6] | (l[7] << 16));
        }
      } else {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const uint4 x = ok_row ? src[c] : make_uint4(0u, 0u, 0u, 0u);
          qv[4 * c] = x.x;
          qv[4 * c + 1] = x.y;
          qv[4 * c + 2] = x.z;
          qv[4 * c + 3] = x.w;
        }
        if (ok_row) next_row = tree_row(a, w.row0, qi, w.n, w.base, true);
      }
    };
    auto store_q = [&](int wt) {
      if constexpr (kE4) {
#pragma unroll 1
        for (int blk = 0; blk < 4; ++blk) {
          uint32_t x[32];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 y = *reinterpret_cast<const uint4*>(stage + 128 * blk + 16 * c);
            x[4 * c] = y.x, x[4 * c + 1] = y.y, x[4 * c + 2] = y.z, x[4 * c + 3] = y.w;
          }
          tc::st32(tmem + lane_base + kColQ + 32 * blk, x);
        }
      } else {
#pragma unroll
        for (int blk = 0; blk < 4; ++blk)
          tc::st32(tmem + lane_base + kColQ + 32 * blk, *reinterpret_cast<uint32_t(*)[32]>(&qv[32 * blk]));
      }
      sm.rows[wt % kRowRing][r] = next_row;
      tc::wait_st();
      tc::fence_before();
      mbar_arrive(&sm.q_full);
    };
    if (static_cast<int>(blockIdx.x) < total) {
      load_q(unit_of<G>(a, sm.plan, blockIdx.x));
      store_q(0);
    }
    int wt = 0;
    for (int u = tree_unit(0); u < total; u = tree_unit(++wt)) {
      const Unit w = unit_of<G>(a, sm.plan, u);
      const int next = tree_unit(wt + 1);
      bool ok = true;
      if (next < total) {
        load_q(unit_of<G>(a, sm.plan, next));
        ok = warp_wait(&sm.q_free, wt & 1, st);
        tc::fence_after();
        if (ok) store_q(wt + 1);
      }
      // ---- epilogue: the copies' rows merged, as output rows or a chunk's part
      ok = ok && warp_wait(&sm.stat_full[wt & 1], (wt >> 1) & 1, st);
      const int stride = kM / w.copies;
      float2 ml[4];
      float M = -INFINITY, den = 0.f;
      for (int c = 0; c < w.copies; ++c) {
        ml[c & 3] = sm.stat[wt & 1][(r & (stride - 1)) + c * stride];
        M = fmaxf(M, ml[c & 3].x);
      }
      for (int c = 0; c < w.copies; ++c)  // a copy that saw no key has sum 0, one that saw only NaN logits NaN
        if (ml[c & 3].y != 0.f) den = fmaf(ex2(ml[c & 3].x - M), ml[c & 3].y, den);
      const float own = sm.stat[wt & 1][r].x;
      mbar_arrive(&sm.stat_free[wt & 1]);
      // this lane's factor; a part stays unnormalised
      const float f = own == -INFINITY && den == den ? 0.f : ex2(own - M) * (w.nc > 1 ? 1.f : 1.f / den);
      ok = ok && warp_wait(&sm.o_done, wt & 1, st);
      if (!group_all(1, ok)) break;  // before the barriers below
      tc::fence_after();
      const int64_t part0 = static_cast<int64_t>(u) * a.part_rows;
      if (w.nc > 1 && r < w.rows && r < stride) a.part_ml[part0 + r] = make_float2(M, den);
      // 8 columns `col..` of row i
      auto put = [&](int i, int col, const float (&x)[8]) {
        if (w.nc > 1) {
          store_f32x8(a.part_o + ((static_cast<int64_t>(u) * 32 + col / 8) * a.part_rows + i) * 8, x);
        } else {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            __nv_bfloat162 h2 = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            pk[e] = *reinterpret_cast<uint32_t*>(&h2);
          }
          uint16_t* dst = a.out + (static_cast<int64_t>(w.row0 + w.q0 + i / G) * a.num_q_heads + w.g * G + i % G) * 256;
          *reinterpret_cast<uint4*>(dst + col) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
      };
#pragma unroll 1
      for (int blk = 0; blk < 8; ++blk) {
        uint32_t o[32];
        tc::ld32(tmem + lane_base + kColO + 32 * blk, o);
        tc::wait_ld();
        if (blk == 7) {  // O has been read
          tc::fence_before();
          mbar_arrive(&sm.o_free);
        }
        float x[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] = f == 0.f ? 0.f : __uint_as_float(o[c]) * f;
        if (w.copies == 1) {
          if (r < w.rows)
#pragma unroll
            for (int c = 0; c < 32; c += 8) put(r, 32 * blk + c, *reinterpret_cast<float(*)[8]>(&x[c]));
        } else {
#pragma unroll
          for (int c = 0; c < 32; c += 4)
            *reinterpret_cast<float4*>(&sm.merge[r * 36 + c]) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
          asm volatile("bar.sync 1, 128;" ::: "memory");
          // thread t: 8 columns of row t / 4, and of row 32 + t / 4 if there are two copies
          for (int i = r >> 2; i < min(stride, w.rows); i += 32) {
            float y[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) y[c] = 0.f;
            for (int k = 0; k < w.copies; ++k) {
              const float* src = &sm.merge[(i + k * stride) * 36 + 8 * (r & 3)];
              const float4 p = *reinterpret_cast<const float4*>(src), q = *reinterpret_cast<const float4*>(src + 4);
              y[0] += p.x, y[1] += p.y, y[2] += p.z, y[3] += p.w;
              y[4] += q.x, y[5] += q.y, y[6] += q.z, y[7] += q.w;
            }
            put(i, 32 * blk + 8 * (r & 3), y);
          }
          asm volatile("bar.sync 1, 128;" ::: "memory");
        }
        __syncwarp();
      }
    }
  }

  tc::fence_before();
  __syncthreads();
  if (warp == 10) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

template <int DT, int G>
cudaError_t launch_g(const LocalArgs& a, cudaStream_t st) {
  CUtensorMap map;
  cudaError_t e = make_local_kv_map(a, &map, DT);
  if (e != cudaSuccess) return e;
  auto kern = local_tree_rows_kernel<DT, G>;
  const size_t smem = sizeof(LSmem<DT>);
  e = set_smem_once(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid_ctas()), dim3(kThreads), smem, st, a, map);
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

cudaError_t launch_local_tree_rows(int dtype, int group, const LocalArgs& a, cudaStream_t st) {
  return dtype == GW_KV_E4M3 ? launch_dt<GW_KV_E4M3>(group, a, st) : launch_dt<GW_KV_BF16>(group, a, st);
}

}  // namespace gw
