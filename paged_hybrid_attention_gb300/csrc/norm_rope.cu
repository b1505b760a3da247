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
// A warp takes a head: a lane holds 8 (head dim 256) or 2 x 8 (512) of its
// elements as one or two 16-byte loads, the mean square is one shuffle sum, and
// a pair's other element comes from the lane 16 (or 8) further by a shuffle.
// Everything stays in float32 registers until the one rounding of each output.
// A warp walks a run of heads of one row, so that the row's (cos, sin) and the
// weights are loaded once for the run, with the next heads' loads in flight.
#include "append_row.cuh"

namespace gw {
namespace {

constexpr int kNrThreads = 256;

template <int LAYOUT>
struct NrTraits {
  static constexpr bool kLocal = LAYOUT == GW_LAYOUT_LOCAL;
  static constexpr int kDim = kLocal ? 256 : 512;
  static constexpr int kHalf = kLocal ? 128 : 64;    // pairs of a head
  static constexpr int kVec = kDim / 256;            // 16-byte pieces of a lane
  static constexpr int kPartner = kHalf / 8;         // lanes between a pair's elements
  static constexpr int kBatch = kLocal ? 4 : 2;      // heads in flight per step
};

// One lane's part of a head, float32: piece p holds dims 256 p + 8 lane + i.
template <int kVec>
struct HeadPart {
  float x[kVec][8];
};

template <int kVec>
__device__ __forceinline__ HeadPart<kVec> unpack(const uint4 (&raw)[kVec]) {
  HeadPart<kVec> h;
#pragma unroll
  for (int p = 0; p < kVec; ++p) bf16x8_to_f32(raw[p], h.x[p]);
  return h;
}

// 1 / sqrt(mean square + eps) of the head that the warp holds.
template <int kVec>
__device__ __forceinline__ float inv_rms(const HeadPart<kVec>& h, float eps) {
  float s = 0.f;
#pragma unroll
  for (int p = 0; p < kVec; ++p)
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(h.x[p][i], h.x[p][i], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return rsqrtf(fmaf(s, 1.f / (256 * kVec), eps));
}

template <int kVec>
__device__ __forceinline__ void scale(HeadPart<kVec>& h, float inv, const float (&w)[kVec][8]) {
#pragma unroll
  for (int p = 0; p < kVec; ++p)
#pragma unroll
    for (int i = 0; i < 8; ++i) h.x[p][i] *= inv * w[p][i];
}

// The half pairs of the head's first 2 kHalf dims (all in piece 0) by cs.
template <class T>
__device__ __forceinline__ void turn(HeadPart<T::kVec>& h, const CosSin8& cs, int lane) {
  const bool second = lane & T::kPartner, rotated = lane < 2 * T::kPartner;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = h.x[0][i];
    const float other = __shfl_xor_sync(0xffffffffu, x, T::kPartner);
    const float y = fmaf(x, cs.c[i], second ? other * cs.s[i] : -(other * cs.s[i]));
    h.x[0][i] = rotated ? y : x;
  }
}

template <int LAYOUT, int DT>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NormRopeArgs a) {
  using T = NrTraits<LAYOUT>;
  constexpr int kVec = T::kVec, kB = T::kBatch;
  constexpr bool kFolded = LAYOUT == GW_LAYOUT_GLOBAL_FOLDED || LAYOUT == GW_LAYOUT_GLOBAL_FOLDED_E4M3;
  const int lane = threadIdx.x & 31;
  // heads of a row: q, then k, then v unless v is k's projection
  const int heads = a.num_q_heads + (a.tied ? 1 : 2) * a.kv_heads;
  const int runs = (heads + a.run - 1) / a.run;
  const int64_t units = static_cast<int64_t>(a.num_rows) * runs;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kNrThreads / 32);
  bool waited = a.early_inputs == 0;
  if (waited) {
    pdl_wait();
    pdl_trigger();
  }
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kNrThreads / 32) + (threadIdx.x >> 5); u < units; u += step) {
    const int64_t row = u / runs;
    const int h0 = static_cast<int>(u - row * runs) * a.run, h1 = min(heads, h0 + a.run);
    auto load = [&](int h, uint4 (&raw)[kVec]) {
      const uint16_t* src = h < a.num_q_heads ? a.q + row * a.q_row + h * a.q_head
                            : h < a.num_q_heads + a.kv_heads
                                ? a.k + row * a.k_row + (h - a.num_q_heads) * a.k_head
                                : a.v + row * a.v_row + (h - a.num_q_heads - a.kv_heads) * a.v_head;
#pragma unroll
      for (int p = 0; p < kVec; ++p) raw[p] = *reinterpret_cast<const uint4*>(src + 256 * p + 8 * lane);
    };
    const int pos = a.pos[row], slot = a.slot[row];
    const bool pos_ok = pos >= 0 && pos < a.max_pos;
    const bool slot_ok = slot >= 0 && slot < a.num_pages * kPage;
    const CosSin8 cs =
        load_cs8(a.rope_cs + (static_cast<int64_t>(pos_ok ? pos : 0) * T::kHalf + 8 * (lane & (T::kPartner - 1))) * 2);
    if (!waited) {
      pdl_wait();
      pdl_trigger();
      waited = true;
    }
    uint4 raw[kB][kVec];
#pragma unroll
    for (int b = 0; b < kB; ++b)
      if (h0 + b < h1) load(h0 + b, raw[b]);
    float qw[kVec][8], kw[kVec][8];
#pragma unroll
    for (int p = 0; p < kVec; ++p)
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(a.q_weight + 256 * p + 8 * lane + i);
        const float4 y = *reinterpret_cast<const float4*>(a.k_weight + 256 * p + 8 * lane + i);
        qw[p][i] = x.x, qw[p][i + 1] = x.y, qw[p][i + 2] = x.z, qw[p][i + 3] = x.w;
        kw[p][i] = y.x, kw[p][i + 1] = y.y, kw[p][i + 2] = y.z, kw[p][i + 3] = y.w;
      }
    if (kFolded) {  // K[128:] = V[128:] wk: the gain goes into q
#pragma unroll
      for (int p = 0; p < kVec; ++p)
        if (p > 0 || lane >= 16)
#pragma unroll
          for (int i = 0; i < 8; ++i) qw[p][i] *= kw[p][i];
    }
    if (h0 == 0 && lane == 0) {
      if (!pos_ok) set_status(a.status, GW_DEV_POS_RANGE);
      if (!slot_ok) set_status(a.status, GW_DEV_SLOT_RANGE);
    }
    if (!pos_ok) continue;
    const int64_t page = slot_ok ? slot / kPage : 0;
    const int off = slot & (kPage - 1);
    for (int hb = h0; hb < h1; hb += kB) {
      uint4 next[kB][kVec];
#pragma unroll
      for (int b = 0; b < kB; ++b)
        if (hb + kB + b < h1) load(hb + kB + b, next[b]);
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const int h = hb + b;
        if (h >= h1) break;
        HeadPart<kVec> x = unpack<kVec>(raw[b]);
        if (h < a.num_q_heads) {
          scale<kVec>(x, inv_rms<kVec>(x, a.eps), qw);
          turn<T>(x, cs, lane);
          uint16_t* dst = a.out + (row * a.num_q_heads + h) * T::kDim + 8 * lane;
#pragma unroll
          for (int p = 0; p < kVec; ++p) *reinterpret_cast<uint4*>(dst + 256 * p) = f32x8_to_bf16(x.x[p]);
          continue;
        }
        const bool is_k = h < a.num_q_heads + a.kv_heads;
        const int g = h - a.num_q_heads - (is_k ? 0 : a.kv_heads);
        const float inv = is_k || a.v_norm ? inv_rms<kVec>(x, a.eps) : 1.f;
        if constexpr (T::kLocal) {
          if (is_k) {
            scale<kVec>(x, inv, kw);
            turn<T>(x, cs, lane);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x.x[0][i] *= inv;
          }
          if (slot_ok)
            store8<DT>(a.pool, (((page * a.kv_heads + g) * 2 + (is_k ? 0 : 1)) * kPage + off) * 256 + 8 * lane, x.x[0]);
        } else {
          using R = GlobalRow<LAYOUT>;
          auto put = [&](int e, const float (&f)[8]) {
            if constexpr (R::kE4)
              *reinterpret_cast<uint2*>(a.pool + tiled_e4m3(page, off, e)) = f32x8_to_e4m3(f);
            else
              *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.pool) + tiled<R::kRow>(page, off, e)) =
                  f32x8_to_bf16(f);
          };
          if (!is_k || a.tied) {  // V: the same projection, without weights
            HeadPart<kVec> v = x;
#pragma unroll
            for (int p = 0; p < kVec; ++p) {
#pragma unroll
              for (int i = 0; i < 8; ++i) v.x[p][i] *= (a.v_norm ? inv : 1.f);
              if (slot_ok) put((kFolded ? 0 : 512) + 256 * p + 8 * lane, v.x[p]);
            }
          }
          if (is_k) {
            scale<kVec>(x, inv, kw);
            turn<T>(x, cs, lane);
            if (slot_ok) {
              if constexpr (kFolded) {
                if (lane < 16) put(512 + 8 * lane, x.x[0]);
              } else {
#pragma unroll
                for (int p = 0; p < kVec; ++p) put(256 * p + 8 * lane, x.x[p]);
              }
            }
          }
        }
      }
#pragma unroll
      for (int b = 0; b < kB; ++b)
#pragma unroll
        for (int p = 0; p < kVec; ++p) raw[b][p] = next[b][p];
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope(int layout, int dtype, const NormRopeArgs& args, cudaStream_t st) {
  NormRopeArgs a = args;
  const int heads = a.num_q_heads + (a.tied ? 1 : 2) * a.kv_heads;
  // Heads per warp: one while there are fewer heads than warps of a full GPU
  // (a decode step is latency), up to a whole row's when rows abound.
  const int64_t warps = static_cast<int64_t>(grid_ctas()) * 32;
  const int64_t per = (static_cast<int64_t>(a.num_rows) * heads + warps - 1) / warps;
  a.run = static_cast<int>(per < heads ? per : heads);
  const int64_t units = static_cast<int64_t>(a.num_rows) * ((heads + a.run - 1) / a.run);
  const int64_t blocks = (units + kNrThreads / 32 - 1) / (kNrThreads / 32);
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
