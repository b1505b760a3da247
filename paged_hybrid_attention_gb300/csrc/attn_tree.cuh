// What the four kernels of drafted trees (attn_tree_local.cu,
// attn_tree_local_rows.cu, attn_tree_global.cu, attn_tree_global_rows.cu) share.
#pragma once

#include "plan.cuh"
#include "tcgen05.cuh"

namespace gw {

constexpr int kRowRing = 4;  // units whose rows' keys are in shared memory
// O is rescaled when a logit exceeds the reference by more than kLazy; on e4m3
// pools a new reference lies kBelowMax below its logit, so that weights reach
// 2^15 and a long tail counts down to 2^-23 of the largest.
constexpr float kLazy = 8.f, kBelowMax = 7.f;

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
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
