// gw_norm_rope_append: the norms of a layer's q, k and v heads, the rotation of
// q and k, the page write of k and v, and the q rows of the attention calls, in
// one pass over the projection's rows.
//
//   r(x) = 1 / sqrt(mean(x^2) + eps)
//   q' = rope(q r(q) wq),  k' = rope(k r(k) wk),  v' = v r(v)  (or v as it is)
//
// "Gemma 4" (pegainfer model page), "Architecture notes": on global layers K
// and V come from one projection, K through k_norm and RoPE on 128 of its 512
// dims, V through a scale-free norm.  So a folded pool's unrotated K dims are
// V's times wk, and wk goes into q' there.
//
// A warp takes a head, and a lane holds both elements of its pairs, so that the
// rotation needs no other lane: of 256 dims 4 l + i and 128 + 4 l + i, of 512
// dims the pairs 2 l + i and 64 + 2 l + i and 12 of the 384 others.  The mean
// square is one shuffle sum; everything stays in float32 registers until the
// one rounding of each output.  A warp walks a run of heads of one kind (q, k
// or v) and row, so that the row's (cos, sin) and the weights are loaded once
// for the run, with kBatch heads' loads in flight, a head's registers taking the
// next one's loads as soon as it is unpacked.
//
// Memory-bound, by the bytes in flight: 8192 rows of 32 + 2 x 16 heads of 256
// (e4m3 pool) 78 us, 0.90 of the copy rate; one 16-byte load a lane and the
// pairs' other halves by shuffles 220 us; 3 blocks an SM instead of 4 86 us
// (more registers, fewer heads in flight), 2 heads at a time 93 us, loads behind
// the position's 84 us, runs of 8 heads 99 us, of 32 95 us.
#include <type_traits>

#include "append_row.cuh"

namespace gw {
namespace {

constexpr int kNrThreads = 256;
constexpr int kMaxRun = 16;  // heads of a run

// A lane's pieces of a head: 2^k elements each, at consecutive dims.
template <bool kLocal>
struct Pieces;
template <>
struct Pieces<true> {
  static constexpr int kDim = 256, kHalf = 128;
  static constexpr int kPair = 4;    // pairs of a lane
  static constexpr int kElems = 8;   // [0, 4): dims 4 l + i, [4, 8): 128 + 4 l + i
  static constexpr int kBatch = 4;
};
template <>
struct Pieces<false> {
  static constexpr int kDim = 512, kHalf = 64;
  static constexpr int kPair = 2;
  static constexpr int kElems = 16;  // [0, 2): dims 2 l + i, [2, 4): 64 + 2 l + i, [4, 12): 128 + 8 l + i, [12, 16): 384 + 4 l + i
  static constexpr int kBatch = 2;
};

// N consecutive bf16 elements as 32-bit words.
template <int N>
__device__ __forceinline__ void load_words(const uint16_t* p, uint32_t* w) {
  if constexpr (N == 2) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 4) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x, w[1] = x.y;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  }
}

template <int N>
__device__ __forceinline__ void load_floats(const float* p, float* w) {
  if constexpr (N == 2) {
    const float2 x = *reinterpret_cast<const float2*>(p);
    w[0] = x.x, w[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(p + i);
      w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
    }
  }
}

// N floats as bf16 or e4m3 at dst (an address for that many elements).
template <int N, int DT>
__device__ __forceinline__ void store_elems(uint8_t* dst, const float* f) {
  if constexpr (DT == GW_KV_BF16) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    if constexpr (N == 2)
      *reinterpret_cast<uint32_t*>(dst) = w[0];
    else if constexpr (N == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint32_t h[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      h[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    if constexpr (N == 2)
      *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(h[0]);
    else if constexpr (N == 4)
      *reinterpret_cast<uint32_t*>(dst) = h[0] | (h[1] << 16);
    else
      *reinterpret_cast<uint2*>(dst) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  }
}

// f(piece size, first dim, the piece's elements) over a lane's pieces.
template <bool kLocal, class F>
__device__ __forceinline__ void each_piece(int lane, F f) {
  using std::integral_constant;
  if constexpr (kLocal) {
    f(integral_constant<int, 4>{}, 4 * lane, 0);
    f(integral_constant<int, 4>{}, 128 + 4 * lane, 4);
  } else {
    f(integral_constant<int, 2>{}, 2 * lane, 0);
    f(integral_constant<int, 2>{}, 64 + 2 * lane, 2);
    f(integral_constant<int, 8>{}, 128 + 8 * lane, 4);
    f(integral_constant<int, 4>{}, 384 + 4 * lane, 12);
  }
}

template <int LAYOUT, int DT>
__global__ void __launch_bounds__(kNrThreads, LAYOUT == GW_LAYOUT_LOCAL ? 4 : 3) norm_rope_kernel(const NormRopeArgs a) {
  constexpr bool kLocal = LAYOUT == GW_LAYOUT_LOCAL;
  constexpr bool kFolded = LAYOUT == GW_LAYOUT_GLOBAL_FOLDED || LAYOUT == GW_LAYOUT_GLOBAL_FOLDED_E4M3;
  using P = Pieces<kLocal>;
  constexpr int kB = P::kBatch, kE = P::kElems;
  const int lane = threadIdx.x & 31;
  // runs of a row: of q, of k, then of v unless v is k's projection
  const int qruns = (a.num_q_heads + a.run - 1) / a.run, kruns = (a.kv_heads + a.run - 1) / a.run;
  const int runs = qruns + (a.tied ? 1 : 2) * kruns;
  const int64_t units = static_cast<int64_t>(a.num_rows) * runs;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kNrThreads / 32);
  bool waited = a.early_inputs == 0;
  if (waited) {
    pdl_wait();
    pdl_trigger();
  }
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kNrThreads / 32) + (threadIdx.x >> 5); u < units; u += step) {
    const int64_t row = u / runs;
    const int r = static_cast<int>(u - row * runs);
    const bool is_q = r < qruns, is_k = !is_q && r < qruns + kruns;
    const int h0 = (is_q ? r : r - qruns - (is_k ? 0 : kruns)) * a.run;
    const int h1 = min(is_q ? a.num_q_heads : a.kv_heads, h0 + a.run);
    const uint16_t* src = is_q ? a.q + row * a.q_row : is_k ? a.k + row * a.k_row : a.v + row * a.v_row;
    const int64_t head = is_q ? a.q_head : is_k ? a.k_head : a.v_head;
    auto load = [&](int h, uint32_t (&w)[kE / 2]) {
      const uint16_t* p = src + h * head;
      each_piece<kLocal>(lane, [&](auto n, int dim, int e) { load_words<n>(p + dim, w + e / 2); });
    };
    uint32_t raw[kB][kE / 2];
    if (waited) {  // before the chain of position, angles and weights
#pragma unroll
      for (int b = 0; b < kB; ++b)
        if (h0 + b < h1) load(h0 + b, raw[b]);
    }
    const int pos = a.pos[row], slot = a.slot[row];
    const bool pos_ok = pos >= 0 && pos < a.max_pos;
    const bool slot_ok = slot >= 0 && slot < a.num_pages * kPage;
    float cs[2 * P::kPair];  // cos, sin of the lane's pairs
    if (!is_q && !is_k) {
#pragma unroll
      for (int i = 0; i < 2 * P::kPair; ++i) cs[i] = 0.f;
    } else {
      load_floats<2 * P::kPair>(
          a.rope_cs + (static_cast<int64_t>(pos_ok ? pos : 0) * P::kHalf + P::kPair * lane) * 2, cs);
    }
    if (!waited) {
      pdl_wait();
      pdl_trigger();
      waited = true;
#pragma unroll
      for (int b = 0; b < kB; ++b)
        if (h0 + b < h1) load(h0 + b, raw[b]);
    }
    if (r == 0 && lane == 0) {
      if (!pos_ok) set_status(a.status, GW_DEV_POS_RANGE);
      if (!slot_ok) set_status(a.status, GW_DEV_SLOT_RANGE);
    }
    if (!pos_ok || (!is_q && !slot_ok)) continue;
    float w[kE];
    {
      const float* weight = is_q ? a.q_weight : a.k_weight;
      each_piece<kLocal>(lane, [&](auto n, int dim, int e) { load_floats<n>(weight + dim, w + e); });
      if (kFolded && is_q) {  // K[128:] = V[128:] wk: the gain goes into q
        float g[kE];
        each_piece<kLocal>(lane, [&](auto n, int dim, int e) { load_floats<n>(a.k_weight + dim, g + e); });
#pragma unroll
        for (int i = 4; i < kE; ++i) w[i] *= g[i];
      }
    }
    const int64_t page = slot_ok ? slot / kPage : 0;
    const int off = slot & (kPage - 1);
    for (int hb = h0; hb < h1; hb += kB) {
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const int h = hb + b;
        if (h >= h1) break;
        float x[kE];
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) {
          x[2 * i] = __uint_as_float(raw[b][i] << 16);
          x[2 * i + 1] = __uint_as_float(raw[b][i] & 0xFFFF0000u);
        }
        if (h + kB < h1) load(h + kB, raw[b]);
        float inv = 1.f;
        if (is_q || is_k || a.v_norm) {
          float s = 0.f;
#pragma unroll
          for (int i = 0; i < kE; ++i) s = fmaf(x[i], x[i], s);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          inv = rsqrtf(fmaf(s, 1.f / P::kDim, a.eps));
        }
        if constexpr (!kLocal) {
          if (!is_q && (!is_k || a.tied)) {  // V: the projection without weights
            const float vn = a.v_norm ? inv : 1.f;
            each_piece<kLocal>(lane, [&](auto n, int dim, int e) {
              float v[n];
#pragma unroll
              for (int i = 0; i < n; ++i) v[i] = x[e + i] * vn;
              const int at = (kFolded ? 0 : 512) + dim;
              if constexpr (LAYOUT == GW_LAYOUT_GLOBAL_FOLDED_E4M3)
                store_elems<n, DT>(a.pool + tiled_e4m3(page, off, at), v);
              else
                store_elems<n, DT>(a.pool + 2 * tiled<GlobalRow<LAYOUT>::kRow>(page, off, at), v);
            });
            if (!is_k) continue;
          }
        }
        if (is_q || is_k) {
#pragma unroll
          for (int i = 0; i < kE; ++i) x[i] *= inv * w[i];
#pragma unroll
          for (int i = 0; i < P::kPair; ++i) {
            const float x0 = x[i], x1 = x[P::kPair + i], c = cs[2 * i], s = cs[2 * i + 1];
            x[i] = fmaf(x0, c, -(x1 * s));
            x[P::kPair + i] = fmaf(x1, c, x0 * s);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kE; ++i) x[i] *= inv;
        }
        if (is_q) {
          uint8_t* dst = reinterpret_cast<uint8_t*>(a.out + (row * a.num_q_heads + h) * P::kDim);
          each_piece<kLocal>(lane,
                             [&](auto n, int dim, int e) { store_elems<n, GW_KV_BF16>(dst + 2 * dim, x + e); });
        } else if constexpr (kLocal) {
          constexpr int kSize = DT == GW_KV_BF16 ? 2 : 1;
          uint8_t* dst = a.pool + (((page * a.kv_heads + h) * 2 + (is_k ? 0 : 1)) * kPage + off) * (256 * kSize);
          each_piece<kLocal>(lane, [&](auto n, int dim, int e) { store_elems<n, DT>(dst + dim * kSize, x + e); });
        } else {
          each_piece<kLocal>(lane, [&](auto n, int dim, int e) {
            if (kFolded && e >= 4) return;  // a folded page holds the rotated dims only
            const int at = (kFolded ? 512 : 0) + dim;
            if constexpr (LAYOUT == GW_LAYOUT_GLOBAL_FOLDED_E4M3)
              store_elems<n, DT>(a.pool + tiled_e4m3(page, off, at), x + e);
            else
              store_elems<n, DT>(a.pool + 2 * tiled<GlobalRow<LAYOUT>::kRow>(page, off, at), x + e);
          });
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope(int layout, int dtype, const NormRopeArgs& args, cudaStream_t st) {
  NormRopeArgs a = args;
  const int heads = a.num_q_heads + (a.tied ? 1 : 2) * a.kv_heads;
  // Heads per warp: one while there are fewer heads than warps of a full GPU
  // (a decode step is latency), up to kMaxRun when rows abound.
  const int64_t warps = static_cast<int64_t>(grid_ctas()) * 32;
  const int64_t per = (static_cast<int64_t>(a.num_rows) * heads + warps - 1) / warps;
  a.run = static_cast<int>(per < kMaxRun ? per : kMaxRun);
  const int runs = (a.num_q_heads + a.run - 1) / a.run + (a.tied ? 1 : 2) * ((a.kv_heads + a.run - 1) / a.run);
  const int64_t blocks = (static_cast<int64_t>(a.num_rows) * runs + kNrThreads / 32 - 1) / (kNrThreads / 32);
  const int64_t cap = static_cast<int64_t>(grid_ctas()) * 16;
  const dim3 grid(static_cast<unsigned>(blocks < cap ? blocks : cap)), block(kNrThreads);
  if (layout == GW_LAYOUT_LOCAL)
    return dtype == GW_KV_BF16 ? launch_pdl(norm_rope_kernel<GW_LAYOUT_LOCAL, GW_KV_BF16>, grid, block, 0, st, a)
                               : launch_pdl(norm_rope_kernel<GW_LAYOUT_LOCAL, GW_KV_E4M3>, grid, block, 0, st, a);
  if (layout == GW_LAYOUT_GLOBAL_FOLDED)
    return launch_pdl(norm_rope_kernel<GW_LAYOUT_GLOBAL_FOLDED, GW_KV_BF16>, grid, block, 0, st, a);
  if (layout == GW_LAYOUT_GLOBAL_FULL)
    return launch_pdl(norm_rope_kernel<GW_LAYOUT_GLOBAL_FULL, GW_KV_BF16>, grid, block, 0, st, a);
  return launch_pdl(norm_rope_kernel<GW_LAYOUT_GLOBAL_FOLDED_E4M3, GW_KV_E4M3>, grid, block, 0, st, a);
}

}  // namespace gw
