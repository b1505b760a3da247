// What the four kernels of drafted trees (attn_tree_local.cu,
// attn_tree_local_rows.cu, attn_tree_global.cu, attn_tree_global_rows.cu) share.
#pragma once

#include "plan.cuh"
#include "tcgen05.cuh"

namespace gw {

constexpr int kRowRing = 4;  // units whose rows' keys are in shared memory
// The softmax's reference m (base 2).  A new one lies kBelow below the logit that
// asks for it, and one is asked for, and O rescaled, when a logit exceeds it by
// more than kRaise.  e4m3 pools: weights reach 2^15 and are held in steps of 2^-16
// or less (split_e5m2), so that one of 2^-22 of the largest has 6 bits and 131072
// of them, 3 % of the sum and all of the output where the largest has no value of
// its own, are still right.  kBelow = 7 ends 5 powers of two earlier and rescales
// less: 61 local sequences, 7 drafts 90.5 us as here (with logits of standard
// deviation 4 instead of 1 94 and here 104), 16 with 64 drafts 58 (80) and 68 (80);
// global, 8 x 131072, 8 heads, 4 drafts 144 (153) and 146 (166), 33 drafts of 16
// heads 404 (459) and 418 (471).
template <bool kE4>
struct Reference {
  static constexpr float kBelow = kE4 ? 12.f : 0.f, kRaise = kE4 ? 15.f : 8.f;
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
}

// Waits for a role's own copies or products before its CTA may end: the last use of
// each of a ring of N barriers that `issued` of them complete, in turn.  They are
// complete already unless a wait gave up.
template <int N>
__device__ __forceinline__ void drain(uint64_t* bars, uint32_t issued) {
  for (uint32_t k = issued > N ? issued - N : 0; k < issued; ++k) mbar_wait(&bars[k % N], (k / N) & 1, nullptr);
}

__device__ __forceinline__ void zero16(uint32_t dst) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(dst), "r"(0) : "memory");
}

// x as two e4m3 terms, hi = e4m3(x) and lo = e4m3(x - hi), two values at a time.
__device__ __forceinline__ void split_e4m3(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __nv_fp8x2_storage_t h2 = __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
  const float2 hf = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(h2, __NV_E4M3)));
  hi = h2;
  lo = __nv_cvt_float2_to_fp8x2(make_float2(x0 - hf.x, x1 - hf.y), __NV_SATFINITE, __NV_E4M3);
}

// x[r] of row r reduced over N lanes, each lane keeping half of its rows and
// merging the other's: lane l gets row l's, x[0].  x is used up.
template <int N, bool kMax>
__device__ __forceinline__ void row_fold(float* x, int lane) {
  if constexpr (N > 1) {
    constexpr int H = N / 2;
    const bool up = lane & H;
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const float send = up ? x[i] : x[i + H];
      const float keep = up ? x[i + H] : x[i];
      const float recv = __shfl_xor_sync(0xffffffffu, send, H);
      x[i] = kMax ? fmaxf(keep, recv) : keep + recv;
    }
    row_fold<H, kMax>(x, lane);
  }
}

}  // namespace gw
