// Attention of drafted trees on GLOBAL layers (gw_tree_attn_global), on the
// tensor cores (tcgen05): head dim 512, one KV head, all three pool layouts,
// calls whose sequences may have more than 64 rows x heads, on the e4m3 pool more
// than 32 (attn_tree_global.cu has the others).
//
// Row r of a sequence's n <= 64 rows sees the cached tokens [0, L - n) and the
// drafts of its mask word.  All heads share the KV head, so 128 / HQ rows x HQ
// heads are the 128 rows of two products over the same cached rows:
//   S[128 x N]    = Q[128 x 512] . K^T        (UMMA M = 128)
//   O[128 x 256] += P[128 x N] . V[:, half]   (UMMA M = 128, N = 256)
// O[128 x 512] in fp32 would fill tensor memory, so a unit is (row block, chunk
// of tiles, half of the output dims), and both halves compute S.
//
// A tile is 64 tokens (full layout: 32) in pages of 8-token x 16-byte blocks,
// which are UMMA core matrices: K-major B operand of Q.K^T, MN-major B operand
// of P.V.  A unit of the upper half reads no V[0:128) of a folded page, one of
// the full layout only its half of V.
// Tensor memory: S (two buffers, P over them), half of Q, the O half; the other
// half of Q is in shared memory.
// On the e4m3 pool q (scaled by an exact power of two per row) is a sum of two
// e4m3 terms, as in the decode kernel, and P of three e5m2 ones.
//
// What bounds it: the chain copy, Q.K^T, softmax, P.V over two tile buffers, 1.40 us a
// tile of which the MMAs are 1.15 (folded); on the e4m3 pool the MMAs of q's two
// terms, 43 ns each, 1.45 us a tile.  8 x 131072 tokens, 4 rows x 32 heads: 367 us
// (one block; the cache alone 197); 33 rows x 16 heads, e4m3, 8 x 16384 to 32768: 433.
//
// Warp roles (384 threads): warps 0-3 softmax (a thread owns a row), 4-7 Q rows
// and epilogue, 8 and 11 copies, 9 issues Q.K^T and owns tensor memory, 10 issues
// P.V.
// At a unit's end the softmax warps go on with the next unit's first tiles: half
// of its Q waits in registers, the other half is copied once the last Q.K^T is
// done, and only the next P.V waits for O to be read (with the softmax warps
// loading Q and storing O themselves, 10 us between two units, 8 to 50 us long).
// Every wait is bounded (GW_DEV_TIMEOUT).
#include <type_traits>

#include "attn_tree.cuh"

namespace gw {
namespace {

constexpr int kM = 128;
constexpr int kThreads = 384;
constexpr uint32_t kColS = 0, kColQ = 128, kColO = 256;

template <int LAYOUT>
struct TL;
template <>
struct TL<GW_LAYOUT_GLOBAL_FOLDED> {
  static constexpr bool kE4 = false;
  static constexpr int kPageBytes = 20480, kBlk = 80, kVcb = 0;
  static constexpr int kPages = 4;   // pages of a tile
  static constexpr int kBufs = 2;    // tiles in shared memory
  static constexpr int kSteps = 32;  // K-steps of Q.K^T (32 bytes of a row each)
  __device__ static constexpr int k_cb(int ks) { return ks < 8 ? 64 + 2 * ks : 2 * ks; }
};
template <>
struct TL<GW_LAYOUT_GLOBAL_FULL> {
  static constexpr bool kE4 = false;
  static constexpr int kPageBytes = 32768, kBlk = 128, kVcb = 64;
  static constexpr int kPages = 2;
  static constexpr int kBufs = 2;
  static constexpr int kSteps = 32;
  __device__ static constexpr int k_cb(int ks) { return 2 * ks; }
};
template <>
struct TL<GW_LAYOUT_GLOBAL_FOLDED_E4M3> {
  static constexpr bool kE4 = true;
  static constexpr int kPageBytes = 10240, kBlk = 40, kVcb = 0;
  static constexpr int kPages = 4;
  static constexpr int kBufs = 3;
  static constexpr int kSteps = 16;
  __device__ static constexpr int k_cb(int ks) { return ks < 4 ? 32 + 2 * ks : 2 * ks; }
};

// The column blocks of a tile in two parts: V's half that the unit multiplies P
// with, and the rest of what Q.K^T reads (the folded layouts' K is partly V).
template <int LAYOUT>
struct Parts {
  using T = TL<LAYOUT>;
  static constexpr int kV = T::kE4 ? 16 : 32;  // blocks of V's half
  // Whether the parts are copied and released on their own.  The bf16 layouts have
  // room for two tiles, and a call waits on their copies (a tile 1.60 us, in parts
  // 1.40); the e4m3 one has three and waits on Q.K^T (1.45 us, in parts 1.55).
  static constexpr bool kApart = !T::kE4;
  __device__ static constexpr int v0(int half) { return T::kVcb + kV * half; }
  // runs [first, end) of the rest
  __device__ static constexpr int runs(int half) { return kApart && LAYOUT != GW_LAYOUT_GLOBAL_FULL && half ? 2 : 1; }
  __device__ static constexpr int first(int half, int i) {
    if (LAYOUT == GW_LAYOUT_GLOBAL_FULL) return 0;
    if (!kApart) return half ? kV / 2 : 0;
    return half == 0 ? kV : i == 0 ? kV / 2 : 2 * kV;
  }
  __device__ static constexpr int end(int half, int i) {
    if (LAYOUT == GW_LAYOUT_GLOBAL_FULL) return 64;
    return kApart && half == 1 && i == 0 ? kV : T::kBlk;
  }
  __device__ static constexpr int rest(int half) {  // blocks that warp 8 copies
    if (!kApart) return half ? T::kBlk - kV / 2 : T::kBlk;
    return end(half, 0) - first(half, 0) + (runs(half) > 1 ? end(half, 1) - first(half, 1) : 0);
  }
  __device__ static constexpr bool in_v(int half, int cb) { return kApart && cb >= v0(half) && cb < v0(half) + kV; }
};

template <int LAYOUT>
struct TSmem {
  using T = TL<LAYOUT>;
  uint8_t tiles[T::kBufs][T::kPages * T::kPageBytes];
  uint8_t q[kM * 512];  // Q dims [256, 512): [row block 16][16-byte block 32][8][16 B]; e4m3: hi, then lo
  uint64_t kfull[T::kBufs], kempty[T::kBufs], vfull[T::kBufs], vempty[T::kBufs], s_ready[2], p_ready[2], pfree[2], stat_full, stat_free;
  uint64_t q_full, q_free, o_done, o_free;
  int32_t mask[T::kBufs];  // pages of the tile that were loaded
  uint32_t tmem_base;
  float stat_inv[kM];  // 1 / l of each row
  float scale[T::kE4 ? kRowRing : 1][T::kE4 ? kM : 1];  // e4m3: 2^-e of each row's scaling
  TreePlan plan;
};
static_assert(sizeof(TSmem<GW_LAYOUT_GLOBAL_FOLDED>) <= 232448, "shared memory of one CTA");
static_assert(sizeof(TSmem<GW_LAYOUT_GLOBAL_FULL>) <= 232448, "shared memory of one CTA");
static_assert(sizeof(TSmem<GW_LAYOUT_GLOBAL_FOLDED_E4M3>) <= 232448, "shared memory of one CTA");

__device__ __forceinline__ uint32_t cm_off(int r, int c, int chunks) {
  return static_cast<uint32_t>(((r >> 3) * chunks + c) * 128 + (r & 7) * 16);
}
__device__ __forceinline__ void sts16(uint32_t dst, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void store_f32x8(float* dst, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(x[0]), "r"(x[1]), "r"(x[2]),
               "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

struct Unit {
  int s, half, q0, nq, n, base, row0;
  int k0, k1;  // keys [k0, k1)
  int nt;      // tiles of them
  int nc;
};

// Unit u: (chunk, row block, half), so that the units that read the same pages
// run at the same time.
template <int HQ, int KN>
__device__ __forceinline__ Unit unit_of(const LocalArgs& a, const TreePlan& plan, int u) {
  constexpr int QB = kM / HQ;
  Unit w;
  const int at = plan_seq(plan.ub, a.batch, u);
  w.s = plan.seq[at];
  w.row0 = a.cu_q_rows[w.s];
  w.n = a.cu_q_rows[w.s + 1] - w.row0;
  const int L = a.seq_lens[w.s];
  w.base = L - w.n;
  const TreeSpan sp = tree_span(L, w.n, a.window, tree_rule_global(HQ));
  w.nc = sp.chunks();
  const int r = u - plan.ub[at];
  w.half = r & 1;
  const int cb = r >> 1, c = cb / sp.blocks;
  w.q0 = (cb - c * sp.blocks) * QB;
  w.nq = min(QB, w.n - w.q0);
  w.k0 = c * sp.ct * kTreeTile;
  w.k1 = min(L, w.k0 + sp.ct * kTreeTile);
  w.nt = (w.k1 - w.k0 + KN - 1) / KN;
  return w;
}

template <int LAYOUT, int HQ>
__global__ void __launch_bounds__(kThreads, 1) global_tree_rows_kernel(const LocalArgs a) {
  using T = TL<LAYOUT>;
  using SM = TSmem<LAYOUT>;
  constexpr bool kE4 = T::kE4;
  constexpr int KN = T::kPages * kPage;  // keys of a tile
  constexpr int NB = T::kBufs;
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
      mbar_init(&sm.p_ready[b], kM);
      mbar_init(&sm.pfree[b], 1);
    }
    mbar_init(&sm.stat_full, kM);
    mbar_init(&sm.stat_free, kM);
    mbar_init(&sm.q_full, kM);
    mbar_init(&sm.q_free, 1);
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.o_free, kM);
    fence_mbar_init();
  }
  if (warp == 9) {
    tc::alloc(&sm.tmem_base, 512);
    tc::relinquish();
  }
  pdl_wait();
  pdl_trigger();
  plan_tree(a, sm.plan, 2, tree_rule_global(HQ), 512);
  const int total = sm.plan.ub[a.batch];
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp == 8 || warp == 11) {
    // --------------------------------------------------------- page copies
    // warp 11 copies V's half, warp 8 the rest; lane l takes 8-token block l % 2
    // of page l / 2 of a tile
    using PT = Parts<LAYOUT>;
    const bool is_v = warp == 11;
    uint64_t* const fulls = is_v ? sm.vfull : sm.kfull;
    uint64_t* const empties = is_v ? sm.vempty : sm.kempty;
    const uint64_t pol = policy_evict_last();  // the other half and row blocks read them too
    const int page = lane >> 1, tb = lane & 1;
    uint32_t gi = 0, halves = 0;  // bit b: the half of buffer b's last tile
    bool ok = true;
    int wt = 0;
    for (int u = tree_unit(0); u < total && ok && (PT::kApart || !is_v); u = tree_unit(++wt)) {
      const Unit w = unit_of<HQ, KN>(a, sm.plan, u);
      const int32_t* bt = a.block_table + static_cast<int64_t>(w.s) * a.max_pages;
      const uint32_t bytes = 128 * (is_v ? PT::kV : w.half ? PT::rest(1) : PT::rest(0));  // of an 8-token block
      for (int t = 0; t < w.nt; ++t, ++gi) {
        const int b = gi % NB;
        const uint32_t use = gi / NB;
        const int k = w.k0 + t * KN + page * kPage;
        int32_t pg = -1;
        if (page < T::kPages && k < w.k1) {
          pg = bt[k / kPage];
          if (pg < 0 || pg >= a.num_pages) {
            if (!is_v) set_status(st, GW_DEV_PAGE_RANGE);
            pg = -1;
          }
        }
        const uint32_t blocks = __ballot_sync(0xffffffffu, pg >= 0);  // bits 2 j, 2 j + 1: page j
        if (use > 0 && !warp_wait(&empties[b], (use - 1) & 1, st)) { ok = false; break; }
        // the rest's columns of one half are V's of the other: after a tile of the
        // other half they are free once its P.V is done (which is after its Q.K^T)
        if (PT::kApart && !is_v && use > 0 && static_cast<int>((halves >> b) & 1) != w.half &&
            !warp_wait(&sm.vempty[b], (use - 1) & 1, st)) {
          ok = false;
          break;
        }
        halves = (halves & ~(1u << b)) | (static_cast<uint32_t>(w.half) << b);
        if (lane == 0) {
          if (!is_v) {
            int mask = 0;
#pragma unroll
            for (int j = 0; j < T::kPages; ++j) mask |= ((blocks >> (2 * j)) & 1) << j;
            sm.mask[b] = mask;
          }
          mbar_arrive_expect_tx(&fulls[b], static_cast<uint32_t>(__popc(blocks)) * bytes);
        }
        __syncwarp();
        if (pg >= 0) {
          uint8_t* dst = sm.tiles[b] + page * T::kPageBytes + tb * T::kBlk * 128;
          const uint8_t* src = a.pool + static_cast<int64_t>(pg) * T::kPageBytes + tb * T::kBlk * 128;
          auto copy = [&](int cb0, int cb1) {
            bulk_g2s(dst + cb0 * 128, src + cb0 * 128, (cb1 - cb0) * 128, &fulls[b], pol);
          };
          if (is_v) {
            copy(PT::v0(w.half), PT::v0(w.half) + PT::kV);
          } else {
            for (int i = 0; i < PT::runs(w.half); ++i) copy(PT::first(w.half, i), PT::end(w.half, i));
          }
        }
      }
    }
    drain<NB>(fulls, gi);
  } else if (warp == 9) {
    // ---------------------------------------------------- Q.K^T issue
    const uint32_t id_s = kE4 ? tc::idesc_e4m3(kM, KN, false, false) : tc::idesc_bf16(kM, KN, false, false);
    // Q dims [256, 512): no-swizzle K-major, 128 B between 16-byte blocks, then
    // the next 8 rows; e4m3: 16 blocks a term, the lo term 32 KB behind
    const uint64_t dq = tc::smem_desc(smem_u32(sm.q), 128, kE4 ? 2048 : 4096);
    uint32_t i = 0;
    int wt = 0;
    bool ok = true;
    for (int u = tree_unit(0); u < total && ok; u = tree_unit(++wt)) {
      const Unit w = unit_of<HQ, KN>(a, sm.plan, u);
      if (!warp_wait(&sm.q_full, wt & 1, st)) break;
      for (int j = 0; j < w.nt; ++j, ++i) {
        const int b = i % NB, sb = i & 1;
        if (!warp_wait(&sm.kfull[b], (i / NB) & 1, st)) { ok = false; break; }
        // this S buffer holds P of tile i - 2 until its P.V is done
        if (i >= 2 && !warp_wait(&sm.pfree[sb], ((i >> 1) - 1) & 1, st)) { ok = false; break; }
        const uint32_t ta = smem_u32(sm.tiles[b]);
        const int mask = sm.mask[b];
        if (mask != (1 << T::kPages) - 1) {  // pages not loaded: zeros
          if (Parts<LAYOUT>::kApart && !warp_wait(&sm.vfull[b], (i / NB) & 1, st)) { ok = false; break; }
          for (int pgi = 0; pgi < T::kPages; ++pgi) {
            if ((mask >> pgi) & 1) continue;
            for (int o = lane * 16; o < T::kPageBytes; o += 32 * 16) zero16(ta + pgi * T::kPageBytes + o);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        tc::fence_after();
        const uint64_t dk = tc::smem_desc(ta, 128, T::kBlk * 128);
        const uint32_t ds = tmem + kColS + KN * sb;
        auto step = [&](int ks, bool more) {
          const uint64_t bd = dk + ((T::k_cb(ks) * 128) >> 4);
          if constexpr (kE4) {
            if (ks < 8) {
              tc::mma_e4m3_ts_warp(ds, tmem + kColQ + 8 * ks, bd, id_s, more);
              tc::mma_e4m3_ts_warp(ds, tmem + kColQ + 64 + 8 * ks, bd, id_s, true);
            } else {
              tc::mma_e4m3_warp(ds, dq + (((ks - 8) * 256) >> 4), bd, id_s, more);
              tc::mma_e4m3_warp(ds, dq + ((32768 + (ks - 8) * 256) >> 4), bd, id_s, true);
            }
          } else {
            if (ks < 16)
              tc::mma_bf16_ts_warp(ds, tmem + kColQ + 8 * ks, bd, id_s, more);
            else
              tc::mma_bf16_warp(ds, dq + (((ks - 16) * 256) >> 4), bd, id_s, more);
          }
        };
        // the K-steps outside V's half (the first of all is one of them), then,
        // once it is there, those in it
        auto steps = [&](auto half, bool v) {
#pragma unroll
          for (int ks = 0; ks < T::kSteps; ++ks)
            if (Parts<LAYOUT>::in_v(half, T::k_cb(ks)) == v) step(ks, ks > 0);
        };
        auto issue = [&](bool v) {
          if (w.half)
            steps(std::integral_constant<int, 1>{}, v);
          else
            steps(std::integral_constant<int, 0>{}, v);
        };
        issue(false);
        if (Parts<LAYOUT>::kApart && LAYOUT != GW_LAYOUT_GLOBAL_FULL) {
          if (!warp_wait(&sm.vfull[b], (i / NB) & 1, st)) {
            tc::commit_warp(&sm.s_ready[sb]);  // those issued above, for drain
            ++i;
            ok = false;
            break;
          }
          tc::fence_after();
          issue(true);
        }
        if (Parts<LAYOUT>::kApart) tc::commit_warp(&sm.kempty[b]);
        tc::commit_warp(&sm.s_ready[sb]);
        if (j == w.nt - 1) tc::commit_warp(&sm.q_free);
      }
    }
    drain<2>(sm.s_ready, i);
  } else if (warp == 10) {
    // ------------------------------------------------------- P.V issue
    const uint32_t id_o = kE4 ? tc::idesc_e5m2_e4m3(kM, 256, false, true) : tc::idesc_bf16(kM, 256, false, true);
    uint32_t i = 0;
    int wt = 0;
    bool ok = true;
    for (int u = tree_unit(0); u < total && ok; u = tree_unit(++wt)) {
      const Unit w = unit_of<HQ, KN>(a, sm.plan, u);
      for (int j = 0; j < w.nt; ++j, ++i) {
        const int b = i % NB, sb = i & 1;
        if (j == 0 && wt >= 1 && !warp_wait(&sm.o_free, (wt - 1) & 1, st)) { ok = false; break; }
        if (Parts<LAYOUT>::kApart && !warp_wait(&sm.vfull[b], (i / NB) & 1, st)) { ok = false; break; }
        if (!warp_wait(&sm.p_ready[sb], (i >> 1) & 1, st)) { ok = false; break; }
        const uint32_t ta = smem_u32(sm.tiles[b]);
        const int key0 = w.k0 + j * KN;
        if (key0 + KN > w.k1) {
          // V rows behind the last key (K rows there only made logits that were
          // masked): zero weights must meet finite values
          // (8-token blocks from their 16-byte pieces' start: a row's pieces share banks)
          const int k = lane & 7;
          for (int blk = max(w.k1 - key0, 0) / 8; blk < KN / 8; ++blk)
            if (key0 + 8 * blk + k >= w.k1)
#pragma unroll
              for (int cb = 0; cb < Parts<LAYOUT>::kV; cb += 4)
                zero16(ta + (blk * T::kBlk + Parts<LAYOUT>::v0(w.half) + cb + (lane >> 3)) * 128 + k * 16);
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc::fence_after();
        const uint64_t dv =
            tc::smem_desc(ta + (T::kVcb + (kE4 ? 16 : 32) * w.half) * 128, T::kBlk * 128, 128);
        const uint32_t p = tmem + kColS + KN * sb;
        if constexpr (kE4) {
          // K-steps of 32 keys; P's terms at columns 0, 16 and 32 of the S buffer
#pragma unroll
          for (int kk = 0; kk < KN / 32; ++kk) {
            const uint64_t bd = dv + ((kk * 4 * T::kBlk * 128) >> 4);
#pragma unroll
            for (int term = 0; term < 3; ++term)
              tc::mma_e4m3_ts_warp(tmem + kColO, p + 16 * term + 8 * kk, bd, id_o, !(j == 0 && kk == 0 && term == 0));
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < KN / 16; ++kk)
            tc::mma_bf16_ts_warp(tmem + kColO, p + 8 * kk, dv + ((kk * 2 * T::kBlk * 128) >> 4), id_o,
                                 !(j == 0 && kk == 0));
        }
        tc::commit_warp(Parts<LAYOUT>::kApart ? &sm.vempty[b] : &sm.kempty[b]);
        tc::commit_warp(&sm.pfree[sb]);
        if (j == w.nt - 1) tc::commit_warp(&sm.o_done);
      }
    }
    drain<2>(sm.pfree, i);
  } else if (warp < 4) {
    // ------------------------------------------------------------ softmax
    const int r = tid, qi = r / HQ;
    const uint32_t lane_base = static_cast<uint32_t>(32 * warp) << 16;
    auto row_of = [&](const Unit& w) {
      return qi < w.nq ? tree_row(a, w.row0, w.q0 + qi, w.n, w.base, false) : TreeRow{0, 0x7fffffff, 1.f};
    };
    uint32_t gi = 0;
    int wt = 0;
    TreeRow next_row{0, 0x7fffffff, 1.f};
    if (static_cast<int>(blockIdx.x) < total) next_row = row_of(unit_of<HQ, KN>(a, sm.plan, blockIdx.x));
    for (int u = tree_unit(0); u < total; u = tree_unit(++wt)) {
      const Unit w = unit_of<HQ, KN>(a, sm.plan, u);
      const bool row_ok = qi < w.nq;
      const TreeRow row = next_row;
      const int next = tree_unit(wt + 1);
      if (next < total) next_row = row_of(unit_of<HQ, KN>(a, sm.plan, next));  // in flight over this unit
      float sc = a.scale_log2;
      float m_ref = -INFINITY;
      float lp[4] = {0.f, 0.f, 0.f, 0.f};
      bool ok = true;
      for (int j = 0; j < w.nt; ++j, ++gi) {
        const int b = gi & 1;
        if (!warp_wait(&sm.s_ready[b], (gi >> 1) & 1, st)) { ok = false; break; }
        tc::fence_after();
        if (kE4 && j == 0) sc = a.scale_log2 * sm.scale[wt % kRowRing][r];  // written before Q was handed over
        uint32_t sv[KN];
#pragma unroll
        for (int c0 = 0; c0 < KN; c0 += 32)
          tc::ld32(tmem + lane_base + kColS + KN * b + c0, *reinterpret_cast<uint32_t(*)[32]>(&sv[c0]));
        tc::wait_ld();
        const int key0 = w.k0 + j * KN;
        if (!(key0 >= row.kmin && key0 + KN <= w.base)) {  // drafts, or a row without keys
          const uint64_t m = tree_tile_mask(row, w.base, key0);
          const uint32_t m0 = static_cast<uint32_t>(m), m1 = static_cast<uint32_t>(m >> 32);
#pragma unroll
          for (int c = 0; c < KN; ++c)
            if (!(((c < 32 ? m0 : m1) >> (c & 31)) & 1)) sv[c] = __float_as_uint(-INFINITY);
        }
        float mg[KN / 8];
#pragma unroll
        for (int g8 = 0; g8 < KN / 8; ++g8) {
          const float* x = reinterpret_cast<const float*>(&sv[g8 * 8]);
          mg[g8] = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
        }
        float mraw = mg[0];
#pragma unroll
        for (int g8 = 1; g8 < KN / 8; ++g8) mraw = fmaxf(mraw, mg[g8]);
        const float mx = mraw * sc;
        const bool raise = mx > m_ref + Reference<kE4>::kRaise;
        if (__any_sync(0xffffffffu, raise)) {
          const float m_new = raise ? mx - Reference<kE4>::kBelow : m_ref;
          const float alpha = m_ref == -INFINITY ? 0.f : ex2(m_ref - m_new);
          if (__any_sync(0xffffffffu, raise && m_ref != -INFINITY)) {
            // O *= alpha for this warp's rows once P.V of the tile before is done
            if (!warp_wait(&sm.pfree[(gi - 1) & 1], ((gi - 1) >> 1) & 1, st)) { ok = false; break; }
            tc::fence_after();
#pragma unroll 1
            for (int blk = 0; blk < 8; ++blk) {
              uint32_t o[32];
              const uint32_t ad = tmem + lane_base + kColO + 32 * blk;
              tc::ld32(ad, o);
              tc::wait_ld();
              if (raise && m_ref != -INFINITY) {
#pragma unroll
                for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
              }
              tc::st32(ad, o);
            }
            tc::wait_st();
          }
          if (raise) {
#pragma unroll
            for (int i = 0; i < 4; ++i) lp[i] *= alpha;
            m_ref = m_new;
          }
        }
        // p = 2^(s sc - m), rounded for the product; l sums it as rounded, so
        // that numerator and denominator round alike
        const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
        uint32_t pw[32];
        if constexpr (kE4) {
          uint32_t pl[16];
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = ex2(fmaf(__uint_as_float(sv[4 * v + i]), sc, neg_m));
            uint32_t w3[3];
            float held[4];
            tc::split_e5m2(p[0], p[1], p[2], p[3], w3, held);
            lp[v & 3] += (held[0] + held[1]) + (held[2] + held[3]);
            pw[v] = w3[0];
            pw[16 + v] = w3[1];
            pl[v] = w3[2];
          }
          tc::st16(tmem + lane_base + kColS + KN * b + 32, pl);
          tc::st32(tmem + lane_base + kColS + KN * b, pw);
        } else {
#pragma unroll
          for (int v = 0; v < KN / 2; ++v) {
            const float p0 = ex2(fmaf(__uint_as_float(sv[2 * v]), sc, neg_m));
            const float p1 = ex2(fmaf(__uint_as_float(sv[2 * v + 1]), sc, neg_m));
            __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
            lp[v & 3] += __low2float(pb) + __high2float(pb);
            pw[v] = *reinterpret_cast<uint32_t*>(&pb);
          }
          if constexpr (KN == 64)
            tc::st32(tmem + lane_base + kColS + KN * b, pw);
          else
            tc::st16(tmem + lane_base + kColS + KN * b, *reinterpret_cast<uint32_t(*)[16]>(&pw[0]));
        }
        tc::wait_st();
        tc::fence_before();
        mbar_arrive(&sm.p_ready[b]);
      }
      if (!ok) break;
      const float l = (lp[0] + lp[1]) + (lp[2] + lp[3]);
      if (w.nc > 1 && row_ok) a.part_ml[static_cast<int64_t>(u) * a.part_rows + r] = make_float2(m_ref, l);
      if (wt >= 1 && !warp_wait(&sm.stat_free, (wt - 1) & 1, st)) break;
      sm.stat_inv[r] = l > 0.f ? 1.f / l : 0.f;
      mbar_arrive(&sm.stat_full);
    }
  } else {
    // ------------------------------------------------- Q rows and epilogue
    const int r = tid - kM;
    const int qi = r / HQ, hd = r % HQ;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t qs = smem_u32(sm.q);
    auto row_src = [&](const Unit& w, int row) {  // row `row` of the unit's 128
      return a.q + (static_cast<int64_t>(w.row0 + w.q0 + row / HQ) * HQ + row % HQ) * 512;
    };
    // The next unit's dims [0, 256) of this thread's row, as tensor memory wants
    // them: bf16, or e4m3 hi (64 words) then lo.
    uint32_t qv[128];
    float up = 1.f;
    auto split16 = [&](const uint4& x, const uint4& y, uint32_t* hi, uint32_t* lo) {  // 16 dims: 4 words of each term
      const uint32_t u8[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t h0, l0, h1, l1;
        split_e4m3(__uint_as_float(u8[2 * i] << 16) * up, __uint_as_float(u8[2 * i] & 0xFFFF0000u) * up, h0, l0);
        split_e4m3(__uint_as_float(u8[2 * i + 1] << 16) * up, __uint_as_float(u8[2 * i + 1] & 0xFFFF0000u) * up, h1, l1);
        hi[i] = h0 | (h1 << 16);
        lo[i] = l0 | (l1 << 16);
      }
    };
    auto load_q = [&](const Unit& w, int wt) {
      const bool ok_row = qi < w.nq;
      const uint4* src = reinterpret_cast<const uint4*>(row_src(w, ok_row ? r : 0));
      const uint4 none = make_uint4(0u, 0u, 0u, 0u);
      if constexpr (kE4) {
        float mq = 0.f;
        if (ok_row) {
#pragma unroll 16
          for (int c = 0; c < 64; ++c) {
            const uint4 x = src[c];
            const uint32_t u4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mq = fmaxf(mq, fmaxf(fabsf(__uint_as_float(u4[i] << 16)), fabsf(__uint_as_float(u4[i] & 0xFFFF0000u))));
          }
        }
        const int ex = mq > 0.f ? static_cast<int>((__float_as_uint(mq) >> 23) & 0xFF) - 127 : 7;
        const int e = min(125, max(-125, 7 - ex));
        // (an infinity, which the terms cannot hold, makes the row's logits NaN)
        up = mq < INFINITY ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : NAN;
        sm.scale[wt % kRowRing][r] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int c = 0; c < 16; ++c)
          split16(ok_row ? src[2 * c] : none, ok_row ? src[2 * c + 1] : none, &qv[4 * c], &qv[64 + 4 * c]);
      } else {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const uint4 x = ok_row ? src[c] : none;
          qv[4 * c] = x.x;
          qv[4 * c + 1] = x.y;
          qv[4 * c + 2] = x.z;
          qv[4 * c + 3] = x.w;
        }
        // the other half is copied when its room is free: into L2 now
        if (ok_row) prefetch_l2(src + 32, 512);
      }
    };
    auto store_q = [&](const Unit& w) {
      auto store_low = [&]() {
#pragma unroll
        for (int blk = 0; blk < 4; ++blk)
          tc::st32(tmem + lane_base + kColQ + 32 * blk, *reinterpret_cast<uint32_t(*)[32]>(&qv[32 * blk]));
      };
      if constexpr (kE4) {
        store_low();
        const bool ok_row = qi < w.nq;
        const uint4* src = reinterpret_cast<const uint4*>(row_src(w, ok_row ? r : 0)) + 32;
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 2
        for (int c = 0; c < 16; ++c) {
          uint32_t hi[4], lo[4];
          split16(ok_row ? src[2 * c] : none, ok_row ? src[2 * c + 1] : none, hi, lo);
          const uint32_t at = qs + cm_off(r, c, 16);
          sts16(at, hi[0], hi[1], hi[2], hi[3]);
          sts16(at + 32768, lo[0], lo[1], lo[2], lo[3]);
        }
      } else {
        // a warp's 32 rows, 8 rows x 4 blocks of 16 bytes at a time: whole sectors
        // from memory, 512 contiguous bytes of shared memory
        const int rows = w.nq * HQ;
        const int row0 = 32 * (warp & 3) + (lane & 7);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int row = row0 + 8 * g;
          const uint16_t* src = row_src(w, row < rows ? row : 0) + 256 + 8 * (lane >> 3);
          const uint32_t at = qs + cm_off(row, lane >> 3, 32);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (row < rows)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + 512 * i), "l"(src + 32 * i)
                           : "memory");
            else
              zero16(at + 512 * i);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        store_low();
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      tc::wait_st();
      fence_proxy_async_smem();
      tc::fence_before();
      mbar_arrive(&sm.q_full);
    };
    if (static_cast<int>(blockIdx.x) < total) {
      const Unit w = unit_of<HQ, KN>(a, sm.plan, blockIdx.x);
      load_q(w, 0);
      store_q(w);
    }
    int wt = 0;
    for (int u = tree_unit(0); u < total; u = tree_unit(++wt)) {
      const Unit w = unit_of<HQ, KN>(a, sm.plan, u);
      const int next = tree_unit(wt + 1);
      if (next < total) {
        const Unit wn = unit_of<HQ, KN>(a, sm.plan, next);
        load_q(wn, wt + 1);
        if (!warp_wait(&sm.q_free, wt & 1, st)) break;
        tc::fence_after();
        store_q(wn);
      }
      // ---- epilogue: this half of O, as output rows or as a chunk's part
      if (!warp_wait(&sm.stat_full, wt & 1, st)) break;
      const float inv = sm.stat_inv[r];
      mbar_arrive(&sm.stat_free);
      if (!warp_wait(&sm.o_done, wt & 1, st)) break;
      tc::fence_after();
      const bool row_ok = qi < w.nq;
      // a part's columns by eights, [8-column block 32][row][8]: a warp's store is
      // then 1 KB in one piece (by rows, 32 lines: reading O took 3 us)
      float* const part = a.part_o + (static_cast<int64_t>(u) * 32 * a.part_rows + r) * 8;
      uint16_t* dst = a.out + (static_cast<int64_t>(w.row0 + w.q0 + qi) * HQ + hd) * 512 + 256 * w.half;
#pragma unroll 1
      for (int blk = 0; blk < 8; ++blk) {
        uint32_t o[32];
        tc::ld32(tmem + lane_base + kColO + 32 * blk, o);
        tc::wait_ld();
        if (blk == 7) {  // O has been read
          tc::fence_before();
          mbar_arrive(&sm.o_free);
        }
        if (row_ok && w.nc > 1) {
#pragma unroll
          for (int c = 0; c < 32; c += 8) store_f32x8(part + static_cast<int64_t>(blk * 4 + c / 8) * a.part_rows * 8, &o[c]);
        } else if (row_ok) {
#pragma unroll
          for (int c = 0; c < 32; c += 8) {
            uint32_t pk[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              __nv_bfloat162 h2 = __floats2bfloat162_rn(__uint_as_float(o[c + 2 * e]) * inv,
                                                        __uint_as_float(o[c + 2 * e + 1]) * inv);
              pk[e] = *reinterpret_cast<uint32_t*>(&h2);
            }
            *reinterpret_cast<uint4*>(dst + blk * 32 + c) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
        }
        __syncwarp();
      }
    }
  }

  tc::fence_before();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

template <int LAYOUT, int HQ>
cudaError_t launch_lh(const LocalArgs& a, cudaStream_t st) {
  auto kern = global_tree_rows_kernel<LAYOUT, HQ>;
  const size_t smem = sizeof(TSmem<LAYOUT>);
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid_ctas()), dim3(kThreads), smem, st, a);
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

cudaError_t launch_global_tree_rows(int layout, const LocalArgs& a, cudaStream_t st) {
  if (layout == GW_LAYOUT_GLOBAL_FOLDED_E4M3) return launch_l<GW_LAYOUT_GLOBAL_FOLDED_E4M3>(a, st);
  return layout == GW_LAYOUT_GLOBAL_FOLDED ? launch_l<GW_LAYOUT_GLOBAL_FOLDED>(a, st)
                                           : launch_l<GW_LAYOUT_GLOBAL_FULL>(a, st);
}

}  // namespace gw
