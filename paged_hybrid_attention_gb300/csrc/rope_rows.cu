// gw_rope_rows and gw_rope_cs_scaled: rotation of rows outside the KV append,
// and its (cos, sin) table for contexts longer than the trained one.
//
// A pair (x0, x1) at position p turns by the angle p * f_i:
//   y0 = x0 cos - x1 sin,   y1 = x1 cos + x0 sin,
// evaluated as the append evaluates it (explicitly rounded binary32 multiply
// and add, no fused multiply-add), so that q and K of one position are turned
// by the same arithmetic.
#include <cuda_fp16.h>

#include "common.cuh"

namespace gw {
namespace {

template <int ELEM>
struct Elem;
template <>
struct Elem<GW_ELEM_BF16> {
  using T = __nv_bfloat16;
  __device__ static float get(T v) { return __bfloat162float(v); }
  __device__ static T put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<GW_ELEM_F16> {
  using T = __half;
  __device__ static float get(T v) { return __half2float(v); }
  __device__ static T put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<GW_ELEM_F32> {
  using T = float;
  __device__ static float get(T v) { return v; }
  __device__ static T put(float v) { return v; }
};

__device__ __forceinline__ void rotate(float& x0, float& x1, float c, float s) {
  const float y0 = __fsub_rn(__fmul_rn(x0, c), __fmul_rn(x1, s));
  const float y1 = __fadd_rn(__fmul_rn(x1, c), __fmul_rn(x0, s));
  x0 = y0;
  x1 = y1;
}

// One item is a pair or a copied element of one (row, head).
template <int ELEM>
__global__ void __launch_bounds__(256) rope_rows_kernel(const RopeRowsArgs a) {
  using E = Elem<ELEM>;
  using T = typename E::T;
  pdl_wait();
  pdl_trigger();
  const int half = a.rot_dim / 2;
  const int per_head = half + (a.inplace ? 0 : a.head_dim - a.rot_dim);
  const int64_t total = static_cast<int64_t>(a.num_rows) * a.num_heads * per_head;
  for (int64_t w = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; w < total;
       w += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int j = static_cast<int>(w % per_head);
    const int64_t rh = w / per_head;
    const int h = static_cast<int>(rh % a.num_heads);
    const int64_t row = rh / a.num_heads;
    const int32_t pos = a.pos[row];
    if (pos < 0 || pos >= a.max_pos) {
      if (j == 0 && h == 0) set_status(a.status, GW_DEV_POS_RANGE);
      continue;
    }
    const T* x = static_cast<const T*>(a.x) + row * a.x_row + h * a.x_head;
    T* y = static_cast<T*>(a.y) + row * a.y_row + h * a.y_head;
    if (j >= half) {
      const int d = a.rot_dim + j - half;
      y[d] = x[d];
      continue;
    }
    const float2 cs = reinterpret_cast<const float2*>(a.rope_cs)[static_cast<int64_t>(pos) * half + j];
    const int d0 = a.pairs == GW_PAIRS_HALF ? j : 2 * j, d1 = a.pairs == GW_PAIRS_HALF ? j + half : 2 * j + 1;
    float x0 = E::get(x[d0]), x1 = E::get(x[d1]);
    rotate(x0, x1, cs.x, a.inverse ? -cs.y : cs.y);
    y[d0] = E::put(x0);
    y[d1] = E::put(x1);
  }
}

// One (cos, sin) entry per item, angle and values in float64.
__global__ void __launch_bounds__(256)
    rope_cs_scaled_kernel(float2* out, const RopeFreqs fr, double amplitude, int half, int64_t total) {
  pdl_wait();
  pdl_trigger();
  for (int64_t w = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; w < total;
       w += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    double s, c;
    sincos(static_cast<double>(w / half) * fr.f[w % half], &s, &c);
    out[w] = make_float2(__double2float_rn(c * amplitude), __double2float_rn(s * amplitude));
  }
}

int grid_for(int64_t items, int block) {
  const int64_t blocks = (items + block - 1) / block, cap = static_cast<int64_t>(grid_ctas()) * 16;
  return static_cast<int>(blocks < cap ? blocks : cap);
}

}  // namespace

cudaError_t launch_rope_rows(int elem, const RopeRowsArgs& a, cudaStream_t st) {
  const int64_t per_head = a.rot_dim / 2 + (a.inplace ? 0 : a.head_dim - a.rot_dim);
  const dim3 grid(grid_for(static_cast<int64_t>(a.num_rows) * a.num_heads * per_head, 256));
  if (elem == GW_ELEM_BF16) return launch_pdl(rope_rows_kernel<GW_ELEM_BF16>, grid, dim3(256), 0, st, a);
  if (elem == GW_ELEM_F16) return launch_pdl(rope_rows_kernel<GW_ELEM_F16>, grid, dim3(256), 0, st, a);
  return launch_pdl(rope_rows_kernel<GW_ELEM_F32>, grid, dim3(256), 0, st, a);
}

cudaError_t launch_rope_cs_scaled(float* out, const RopeFreqs& freqs, double amplitude, int half, int max_pos,
                                  cudaStream_t st) {
  const int64_t total = static_cast<int64_t>(max_pos) * half;
  return launch_pdl(rope_cs_scaled_kernel, dim3(grid_for(total, 256)), dim3(256), 0, st,
                    reinterpret_cast<float2*>(out), freqs, amplitude, half, total);
}

}  // namespace gw
