// The weights pass of gw_decode_attn_global_acc: acc[b][j] = decay * acc[b][j]
// + sum over the heads of 2^(S[j][h] - M_h) / l_h, with S the logits that the
// decode kernel stored (base-2 units) and (M_h, 1 / l_h) the row's softmax
// statistics that the combine stored.
//
// A weight needs the statistics of the whole row, which no chunk of the
// split-KV decode has; keeping the logits (4 HQ bytes per token) and reading
// them once is a tenth to a fifth of the cache row's 640 to 2048 bytes, where a
// second pass over K would be four fifths.
#include "common.cuh"

namespace gw {
namespace {

// Threads take (token, 4-head quarter-lines): HQ / 4 lanes read a token's
// logits as 16-byte pieces, and add up their sums by shuffles.
template <int HQ>
__global__ void __launch_bounds__(256) attn_acc_kernel(const LocalArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int kLanes = HQ / 4;           // lanes per token
  constexpr int kTokens = 256 / kLanes;    // tokens per block and step
  const int s = blockIdx.y;
  const int L = a.seq_lens[s];
  if (a.cu_q_rows[s + 1] - a.cu_q_rows[s] != 1 || L < 1 || L > a.max_pages * kPage ||
      a.unit_base[a.batch] > a.max_units)
    return;
  const int part = threadIdx.x % kLanes;
  float m[4], inv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 st = a.stat[static_cast<int64_t>(s) * HQ + 4 * part + i];
    m[i] = st.x;
    inv[i] = st.y;
  }
  const float4* score = reinterpret_cast<const float4*>(a.score + static_cast<int64_t>(s) * a.max_pages * kPage * HQ);
  float* acc = a.acc + s * a.acc_stride;
  const int step = gridDim.x * kTokens;
  for (int t0 = blockIdx.x * kTokens; t0 < L; t0 += step) {
    const int t = t0 + threadIdx.x / kLanes;
    float w = 0.f;
    if (t < L) {
      const float4 x = score[static_cast<int64_t>(t) * kLanes + part];
      // a head without keys (M = -inf) has 1 / l = 0 and no logit above -inf
      w += inv[0] > 0.f ? ex2(x.x - m[0]) * inv[0] : 0.f;
      w += inv[1] > 0.f ? ex2(x.y - m[1]) * inv[1] : 0.f;
      w += inv[2] > 0.f ? ex2(x.z - m[2]) * inv[2] : 0.f;
      w += inv[3] > 0.f ? ex2(x.w - m[3]) * inv[3] : 0.f;
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    if (t < L && part == 0) acc[t] = a.decay > 0.f ? fmaf(a.decay, acc[t], w) : w;
  }
}

}  // namespace

cudaError_t launch_attn_acc(const LocalArgs& a, cudaStream_t st) {
  const int64_t tokens = static_cast<int64_t>(a.max_pages) * kPage;
  const int per_block = 256 / (a.num_q_heads / 4);
  int64_t blocks = (tokens + per_block - 1) / per_block;
  const int64_t cap = (static_cast<int64_t>(grid_ctas()) * 16 + a.batch - 1) / a.batch;
  if (blocks > cap) blocks = cap;
  const dim3 grid(static_cast<unsigned>(blocks), a.batch);
  if (a.num_q_heads == 8) return launch_pdl(attn_acc_kernel<8>, grid, dim3(256), 0, st, a);
  if (a.num_q_heads == 16) return launch_pdl(attn_acc_kernel<16>, grid, dim3(256), 0, st, a);
  return launch_pdl(attn_acc_kernel<32>, grid, dim3(256), 0, st, a);
}

}  // namespace gw
