// gw_rope_rows and gw_rope_cs_scaled: rotation of rows outside the KV append,
// and its (cos, sin) table for contexts longer than the trained one.
//
// A pair (x0, x1) at position p turns by the angle p * f_i:
//   y0 = x0 cos - x1 sin,   y1 = x1 cos + x0 sin,
// evaluated as the append evaluates it (explicitly rounded binary32 multiply
// and add, no fused multiply-add), so that q and K of one position are turned
// by the same arithmetic.
#include "common.cuh"

namespace gw {
namespace {

// ---- rows ---------------------------------------------------------------------
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

// VB bytes of elements in one access, and as floats: two 16-bit elements are
// packed by one conversion.
template <int ELEM, int VB>
struct alignas(VB) Chunk {
  using E = Elem<ELEM>;
  using T = typename E::T;
  static constexpr int kE = VB / static_cast<int>(sizeof(T));
  T v[kE];
  __device__ __forceinline__ void get(float (&f)[kE]) const {
    if constexpr (ELEM == GW_ELEM_F32 || kE == 1) {
#pragma unroll
      for (int i = 0; i < kE; ++i) f[i] = E::get(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kE; i += 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(&v[i]);
        if constexpr (ELEM == GW_ELEM_BF16) {
          f[i] = __uint_as_float(w << 16);
          f[i + 1] = __uint_as_float(w & 0xffff0000u);
        } else {
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w));
          f[i] = x.x;
          f[i + 1] = x.y;
        }
      }
    }
  }
  __device__ __forceinline__ void put(const float (&f)[kE]) {
    if constexpr (ELEM == GW_ELEM_F32 || kE == 1) {
#pragma unroll
      for (int i = 0; i < kE; ++i) v[i] = E::put(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kE; i += 2) {
        if constexpr (ELEM == GW_ELEM_BF16)
          *reinterpret_cast<__nv_bfloat162*>(&v[i]) = __floats2bfloat162_rn(f[i], f[i + 1]);
        else
          *reinterpret_cast<__half2*>(&v[i]) = __floats2half2_rn(f[i], f[i + 1]);
      }
    }
  }
};

// How a call's rows are dealt to threads.  A thread keeps its item and so its
// (cos, sin) entries for all heads of its row that it takes, which leaves the
// rows themselves as the only traffic beyond L1.
struct RowsPlan {
  int per_head;  // items of a (row, head)
  int lanes;     // heads that a block takes at a time: thread t has item t % per_head of head t / per_head
  int sweeps;    // times it takes `lanes` heads
  int groups;    // blocks' tasks per row
  int64_t tasks;
};

// Most threads of a block: a head of 1024 elements has an item per access.
template <int ELEM, int VB>
constexpr int kRowThreads = (ELEM == GW_ELEM_F32 ? 4096 : 2048) / VB > 256 ? (ELEM == GW_ELEM_F32 ? 4096 : 2048) / VB : 256;

// In place, and out of place where all of a head rotates: an item is the pairs
// of one VB-byte access (half pairs: of two, one in each half of the rotated
// dims).  Bound by memory: 8192 x 32 x 512 bf16 rows, all dims rotated, take 82
// to 85 us for 541 MB (0.94 to 0.97 of a copy), 4093 x 16 x 256 fp32 rows 24.6 us
// for 138 MB.  Interleaved pairs have one access an item and keep four in
// flight (two: 94 us), half pairs two of two (three: 87 us).
template <int ELEM, bool INTER, int VB>
__global__ void __launch_bounds__(kRowThreads<ELEM, VB>, 4 * 256 / kRowThreads<ELEM, VB>)
    rope_pairs_kernel(const RopeRowsArgs a, const RowsPlan p) {
  using E = Elem<ELEM>;
  using T = typename E::T;
  constexpr int kE = VB / static_cast<int>(sizeof(T));        // elements per access
  constexpr bool kTwo = !INTER || kE == 1;                    // the pairs' elements come from two accesses
  constexpr int kP = kTwo ? kE : kE / 2;                      // pairs per item
  constexpr int kUn = kTwo ? 2 : 4;
  using V = Chunk<ELEM, VB>;
  bool waited = a.early_inputs == 0;  // pos and the table rows may be read before the wait
  auto pass = [&]() {
    if (!waited) {
      pdl_wait();
      pdl_trigger();
      waited = true;
    }
  };
  if (waited) {
    pdl_wait();
    pdl_trigger();
  }
  const int half = a.rot_dim / 2;
  const int t = threadIdx.x, item = t % p.per_head, lane = t / p.per_head;
  // offsets of the item's accesses within a head
  const int d0 = INTER ? 2 * kP * item : kP * item;
  const int d1 = INTER ? d0 + 1 : d0 + half;
  for (int64_t task = blockIdx.x; task < p.tasks; task += gridDim.x) {
    const int64_t row = task / p.groups;
    const int h0 = static_cast<int>(task - row * p.groups) * p.lanes * p.sweeps + lane;
    const int32_t pos = a.pos[row];
    if (pos < 0 || pos >= a.max_pos) {
      pass();
      if (t == 0 && task == row * p.groups) set_status(a.status, GW_DEV_POS_RANGE);
      continue;
    }
    if (lane >= p.lanes) continue;
    const T* x = static_cast<const T*>(a.x) + row * a.x_row;
    T* y = static_cast<T*>(a.y) + row * a.y_row;
    float c[kP], s[kP];
    const float* cs = a.rope_cs + (static_cast<int64_t>(pos) * half + kP * item) * 2;
    if constexpr (kP == 1) {
      const float2 e = *reinterpret_cast<const float2*>(cs);
      c[0] = e.x;
      s[0] = e.y;
    } else {
#pragma unroll
      for (int i = 0; i < kP; i += 2) {
        const float4 e = *reinterpret_cast<const float4*>(cs + 2 * i);
        c[i] = e.x;
        s[i] = e.y;
        c[i + 1] = e.z;
        s[i + 1] = e.w;
      }
    }
    if (a.inverse) {
#pragma unroll
      for (int i = 0; i < kP; ++i) s[i] = -s[i];
    }
    pass();
    for (int k0 = 0; k0 < p.sweeps; k0 += kUn) {
      V v0[kUn], v1[kUn];
#pragma unroll
      for (int k = 0; k < kUn; ++k) {
        const int h = h0 + (k0 + k) * p.lanes;
        if (k0 + k < p.sweeps && h < a.num_heads) {
          const T* from = x + h * a.x_head;
          v0[k] = *reinterpret_cast<const V*>(from + d0);
          if constexpr (kTwo) v1[k] = *reinterpret_cast<const V*>(from + d1);
        }
      }
#pragma unroll
      for (int k = 0; k < kUn; ++k) {
        const int h = h0 + (k0 + k) * p.lanes;
        if (k0 + k < p.sweeps && h < a.num_heads) {
          T* to = y + h * a.y_head;
          float f[kE], g[kE];
          v0[k].get(f);
          if constexpr (kTwo) {
            v1[k].get(g);
#pragma unroll
            for (int i = 0; i < kP; ++i) rotate(f[i], g[i], c[i], s[i]);
            v1[k].put(g);
            *reinterpret_cast<V*>(to + d1) = v1[k];
          } else {
#pragma unroll
            for (int i = 0; i < kP; ++i) rotate(f[(2 * i) % kE], f[(2 * i + 1) % kE], c[i], s[i]);
          }
          v0[k].put(f);
          *reinterpret_cast<V*>(to + d0) = v0[k];
        }
      }
    }
  }
  pass();
}

// Out of place, an item can be any aligned chunk of a head: it loads the
// partners of its elements beside them and writes only itself, so that heads
// fall into equal items however their parts are cut.  An element turns by
// y = x c + x' s', with s' = -s for the first of a pair and s for the second,
// which is the pair's arithmetic bit for bit.  Half pairs whose distance is no
// whole number of chunks take their partners one by one (from L1: they are some
// other thread's chunk).
enum { kInterleaved, kHalfChunks, kHalfScattered };

template <int ELEM, int KIND, int VB>
__global__ void __launch_bounds__(kRowThreads<ELEM, VB>, 4 * 256 / kRowThreads<ELEM, VB>)
    rope_chunks_kernel(const RopeRowsArgs a, const RowsPlan p) {
  using E = Elem<ELEM>;
  using T = typename E::T;
  constexpr int kE = VB / static_cast<int>(sizeof(T));
  constexpr bool INTER = KIND == kInterleaved;
  constexpr bool kInside = INTER && kE > 1;     // partners lie in the same chunk
  constexpr bool kWhole = KIND == kHalfChunks;  // the partners are a chunk themselves
  constexpr int kUn = KIND == kHalfScattered ? 1 : KIND == kHalfChunks ? 2 : 4;
  using V = Chunk<ELEM, VB>;
  bool waited = a.early_inputs == 0;  // pos and the table rows may be read before the wait
  auto pass = [&]() {
    if (!waited) {
      pdl_wait();
      pdl_trigger();
      waited = true;
    }
  };
  if (waited) {
    pdl_wait();
    pdl_trigger();
  }
  const int half = a.rot_dim / 2;
  const int t = threadIdx.x, item = t % p.per_head, lane = t / p.per_head;
  const int d0 = item * kE;
  const bool rotates = d0 < a.rot_dim;
  // element d's pair and partner
  auto pair_of = [&](int d) { return INTER ? d / 2 : d < half ? d : d - half; };
  auto partner_of = [&](int d) { return INTER ? d ^ 1 : d < half ? d + half : d - half; };
  for (int64_t task = blockIdx.x; task < p.tasks; task += gridDim.x) {
    const int64_t row = task / p.groups;
    const int h0 = static_cast<int>(task - row * p.groups) * p.lanes * p.sweeps + lane;
    const int32_t pos = a.pos[row];
    if (pos < 0 || pos >= a.max_pos) {
      pass();
      if (t == 0 && task == row * p.groups) set_status(a.status, GW_DEV_POS_RANGE);
      continue;
    }
    if (lane >= p.lanes) continue;
    const T* x = static_cast<const T*>(a.x) + row * a.x_row;
    T* y = static_cast<T*>(a.y) + row * a.y_row;
    float c[kE], s[kE];
    if (rotates) {
      const float* cs = a.rope_cs + static_cast<int64_t>(pos) * a.rot_dim;
      if constexpr (kE > 1 && kWhole) {
        const int i0 = pair_of(d0);
#pragma unroll
        for (int i = 0; i + 1 < kE; i += 2) {
          const float4 e = *reinterpret_cast<const float4*>(cs + 2 * (i0 + i));
          c[i] = e.x;
          s[i] = e.y;
          c[i + 1] = e.z;
          s[i + 1] = e.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kE; i += kInside ? 2 : 1) {
          if (d0 + i < a.rot_dim) {
            const float2 e = *reinterpret_cast<const float2*>(cs + 2 * pair_of(d0 + i));
            c[i] = e.x;
            s[i] = e.y;
            if (kInside) {
              c[(i + 1) % kE] = e.x;
              s[(i + 1) % kE] = e.y;
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        const bool first = INTER ? (d0 + i) % 2 == 0 : d0 + i < half;
        if (first != (a.inverse != 0)) s[i] = -s[i];
      }
    }
    pass();
    for (int k0 = 0; k0 < p.sweeps; k0 += kUn) {
      V v[kUn], w[kUn];
#pragma unroll
      for (int k = 0; k < kUn; ++k) {
        const int h = h0 + (k0 + k) * p.lanes;
        if (k0 + k < p.sweeps && h < a.num_heads) {
          const T* from = x + h * a.x_head;
          v[k] = *reinterpret_cast<const V*>(from + d0);
          if (!kInside && rotates) {
            if constexpr (kWhole) {
              w[k] = *reinterpret_cast<const V*>(from + partner_of(d0));
            } else {
#pragma unroll
              for (int i = 0; i < kE; ++i)
                if (d0 + i < a.rot_dim) w[k].v[i] = from[partner_of(d0 + i)];
            }
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kUn; ++k) {
        const int h = h0 + (k0 + k) * p.lanes;
        if (k0 + k < p.sweeps && h < a.num_heads) {
          V out = v[k];
          if (rotates) {
            float f[kE], g[kE], r[kE];
            v[k].get(f);
            if constexpr (!kInside) w[k].get(g);
#pragma unroll
            for (int i = 0; i < kE; ++i)
              r[i] = __fadd_rn(__fmul_rn(f[i], c[i]), __fmul_rn(kInside ? f[i ^ 1] : g[i], s[i]));
            out.put(r);
            if (d0 + kE > a.rot_dim) {  // the chunk in which the rotated part ends
#pragma unroll
              for (int i = 0; i < kE; ++i)
                if (d0 + i >= a.rot_dim) out.v[i] = v[k].v[i];
            }
          }
          *reinterpret_cast<V*>(y + h * a.y_head + d0) = out;
        }
      }
    }
  }
  pass();
}

// Deals a call's rows to blocks, per_head given; returns a block's threads.
int plan_rows(const RopeRowsArgs& a, int sweeps, RowsPlan& p) {
  const int block = p.per_head <= 256 ? 256 : (p.per_head + 31) / 32 * 32;
  p.lanes = block / p.per_head < a.num_heads ? block / p.per_head : a.num_heads;
  // Up to `sweeps` times the lanes' heads a block (one read of pos and of the
  // table entries for all), fewer while that leaves SMs without a block.
  p.sweeps = sweeps;
  const int64_t want = 4 * static_cast<int64_t>(grid_ctas());
  auto tasks_of = [&](int n) {
    return static_cast<int64_t>(a.num_rows) * ((a.num_heads + p.lanes * n - 1) / (p.lanes * n));
  };
  while (p.sweeps > 1 && tasks_of(p.sweeps) < want) p.sweeps /= 2;
  p.groups = (a.num_heads + p.lanes * p.sweeps - 1) / (p.lanes * p.sweeps);
  p.tasks = tasks_of(p.sweeps);
  return block;
}

dim3 rows_grid(const RowsPlan& p) {
  const int64_t cap = static_cast<int64_t>(grid_ctas()) * 16;
  return dim3(static_cast<unsigned>(p.tasks < cap ? p.tasks : cap));
}

template <int ELEM, int VB>
cudaError_t launch_pairs(const RopeRowsArgs& a, cudaStream_t st) {
  constexpr int kE = VB / (ELEM == GW_ELEM_F32 ? 4 : 2);
  const bool inter = a.pairs == GW_PAIRS_INTERLEAVED;
  RowsPlan p{};
  p.per_head = inter && kE > 1 ? a.rot_dim / kE : a.rot_dim / 2 / kE;
  const int block = plan_rows(a, 4, p);
  if (inter) return launch_pdl(rope_pairs_kernel<ELEM, true, VB>, rows_grid(p), dim3(block), 0, st, a, p);
  return launch_pdl(rope_pairs_kernel<ELEM, false, VB>, rows_grid(p), dim3(block), 0, st, a, p);
}

template <int ELEM, int VB>
cudaError_t launch_chunks(const RopeRowsArgs& a, cudaStream_t st) {
  RowsPlan p{};
  p.per_head = a.head_dim / (VB / (ELEM == GW_ELEM_F32 ? 4 : 2));
  const int block = plan_rows(a, 8, p);
  constexpr int kE = VB / (ELEM == GW_ELEM_F32 ? 4 : 2);
  auto kern = a.pairs == GW_PAIRS_INTERLEAVED ? rope_chunks_kernel<ELEM, kInterleaved, VB>
              : a.rot_dim / 2 % kE == 0       ? rope_chunks_kernel<ELEM, kHalfChunks, VB>
                                              : rope_chunks_kernel<ELEM, kHalfScattered, VB>;
  return launch_pdl(kern, rows_grid(p), dim3(block), 0, st, a, p);
}

template <int ELEM>
cudaError_t launch_rows(const RopeRowsArgs& a, cudaStream_t st) {
  constexpr int kSize = ELEM == GW_ELEM_F32 ? 4 : 2;
  // every offset of a head, in bytes
  uint64_t at = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y);
  if (a.num_rows > 1) at |= static_cast<uint64_t>(a.x_row | a.y_row) * kSize;
  if (a.num_heads > 1) at |= static_cast<uint64_t>(a.x_head | a.y_head) * kSize;
  const uint64_t pairs = at | static_cast<uint64_t>(a.pairs == GW_PAIRS_HALF ? a.rot_dim / 2 : a.rot_dim) * kSize;
  const uint64_t chunks = at | static_cast<uint64_t>(a.head_dim) * kSize;
  if (a.inplace || (a.rot_dim == a.head_dim && pairs % 16 == 0)) {
    if (pairs % 16 == 0) return launch_pairs<ELEM, 16>(a, st);
    if (pairs % 8 == 0) return launch_pairs<ELEM, 8>(a, st);
    if (pairs % 4 == 0) return launch_pairs<ELEM, 4>(a, st);
    if constexpr (kSize == 2) return launch_pairs<ELEM, 2>(a, st);
  } else {
    if (chunks % 16 == 0) return launch_chunks<ELEM, 16>(a, st);
    if (chunks % 8 == 0) return launch_chunks<ELEM, 8>(a, st);
    if (chunks % 4 == 0) return launch_chunks<ELEM, 4>(a, st);
    if constexpr (kSize == 2) return launch_chunks<ELEM, 2>(a, st);
  }
  return cudaErrorInvalidValue;  // not reached: the entry point checks the alignment to an element
}

// ---- table --------------------------------------------------------------------
// Entry (p, i) is amplitude * e^(i p f_i).  The FP64 pipes of this GPU have
// about 1/60 of the FP32 rate, so nothing here is float64: angles are 64-bit
// fractions of a turn, whose products wrap as angles do, and values are pairs
// of floats (hi + lo, about 48 bits; products split exactly by a fused
// multiply-add, sums by Knuth's two-sum).  A thread takes e^(i p f) at the first
// of its positions by Taylor series and gets the others by complex products with
// e^(i f) and e^(4 i f), up to 3 + 31 of them, each of which adds the error of a
// series and of a product.  Over 200000 random chains of that length the values
// were off by 2^-42 at most (the host's arithmetic, against 113 bits); each is
// rounded once to float32.
// 262144 x 64 entries take 33.5 us (134 MB, the floor 20 us), 32768 x 128 14.6 us
// (the floor 5): about forty FP32 operations an entry bound it, at the start of a
// thread some 700 more, and a last wave that is not full: with three blocks to an
// SM 456 run at once, and these tables have 1024 and 512.
struct Ff {
  float h, l;
};
struct Cplx {
  Ff re, im;
};

__host__ __device__ constexpr Ff split(double v) {
  const float h = static_cast<float>(v);
  return Ff{h, static_cast<float>(v - static_cast<double>(h))};
}

// s = a + b and its rounding error
__device__ __forceinline__ float two_sum(float a, float b, float& err) {
  const float s = __fadd_rn(a, b);
  const float v = __fsub_rn(s, a);
  err = __fadd_rn(__fsub_rn(a, __fsub_rn(s, v)), __fsub_rn(b, v));
  return s;
}

__device__ __forceinline__ Ff renorm(float s, float low) {
  const float h = __fadd_rn(s, low);
  return Ff{h, __fsub_rn(low, __fsub_rn(h, s))};
}

// a b + c in pairs of floats
__device__ __forceinline__ Ff mul_add(const Ff& a, const Ff& b, const Ff& c) {
  const float p = __fmul_rn(a.h, b.h);
  float low = __fmaf_rn(a.h, b.h, -p);
  low = __fmaf_rn(a.h, b.l, low);
  low = __fmaf_rn(a.l, b.h, low);
  float err;
  const float s = two_sum(p, c.h, err);
  return renorm(s, __fadd_rn(__fadd_rn(err, low), c.l));
}

// a b + SIGN c d in pairs of floats, SIGN = +-1
template <int SIGN>
__device__ __forceinline__ Ff dot2(const Ff& a, const Ff& b, const Ff& c, const Ff& d) {
  const float ch = SIGN > 0 ? c.h : -c.h, cl = SIGN > 0 ? c.l : -c.l;
  const float p = __fmul_rn(a.h, b.h), q = __fmul_rn(ch, d.h);
  float err;
  const float s = two_sum(p, q, err);
  float low = __fadd_rn(__fadd_rn(__fmaf_rn(a.h, b.h, -p), __fmaf_rn(ch, d.h, -q)), err);
  low = __fmaf_rn(a.h, b.l, low);
  low = __fmaf_rn(a.l, b.h, low);
  low = __fmaf_rn(ch, d.l, low);
  low = __fmaf_rn(cl, d.h, low);
  return renorm(s, low);
}

__device__ __forceinline__ Cplx mul(const Cplx& a, const Cplx& b) {
  return Cplx{dot2<-1>(a.re, b.re, a.im, b.im), dot2<1>(a.re, b.im, a.im, b.re)};
}

// p * f as a fraction of a turn in units of 2^-64, from f's 96-bit fraction.
__device__ __forceinline__ uint64_t turns(uint32_t p, const RopeFreqs& fr, int i) {
  return p * fr.hi[i] + __umulhi(p, fr.lo[i]);
}

// e^(2 pi i x), x a fraction of a turn in units of 2^-64, good to about 2^-45.
// With k the nearest quarter turn, y = 2 pi (x - k/4) has |y| < 0.79, and the
// series of
//   sin y = y + y z (-1/3! + z (1/5! - ...)),  cos y = 1 + z (-1/2! + z (...)),
// z = y^2, are cut behind y^15 and y^16 (the next terms are below 2^-54 and
// 2^-58).  The terms from z^5 on are below 2^-25, where plain floats do: off by
// 2^-46.8 at most over two million angles (with the terms of z^4, 2^-18, in plain
// floats too it was 2^-42.3).
__device__ __forceinline__ Cplx unit(uint64_t x) {
  const int k = static_cast<int>((x + (1ull << 61)) >> 62);
  const int64_t r = static_cast<int64_t>(x - (static_cast<uint64_t>(k) << 62));  // in [-2^61, 2^61)
  const float rh = __ll2float_rn(r);
  const Ff frac{rh, __ll2float_rn(r - __float2ll_rn(rh))};
  constexpr Ff kUnit = split(6.283185307179586 / 18446744073709551616.0);  // 2 pi 2^-64
  const Ff y = mul_add(frac, kUnit, Ff{0.f, 0.f});
  const Ff z = mul_add(y, y, Ff{0.f, 0.f});
  constexpr Ff kOne{1.f, 0.f};
  constexpr Ff kS1 = split(-1.0 / 6), kS2 = split(1.0 / 120), kS3 = split(-1.0 / 5040);
  constexpr Ff kC1 = split(-1.0 / 2), kC2 = split(1.0 / 24), kC3 = split(-1.0 / 720);
  constexpr Ff kS4 = split(1.0 / 362880), kC4 = split(1.0 / 40320);
  constexpr float kS5 = -1.0 / 39916800, kS6 = 1.0 / 6227020800.0, kS7 = -1.0 / 1307674368000.0;
  constexpr float kC5 = -1.0 / 3628800, kC6 = 1.0 / 479001600, kC7 = -1.0 / 87178291200.0, kC8 = 1.0 / 20922789888000.0;
  const float ts = fmaf(z.h, fmaf(z.h, kS7, kS6), kS5);
  const float tc = fmaf(z.h, fmaf(z.h, fmaf(z.h, kC8, kC7), kC6), kC5);
  Ff ps = mul_add(z, mul_add(z, Ff{ts, 0.f}, kS4), kS3);
  ps = mul_add(z, ps, kS2);
  ps = mul_add(z, ps, kS1);
  const Ff sn = mul_add(mul_add(y, z, Ff{0.f, 0.f}), ps, y);
  Ff pc = mul_add(z, mul_add(z, Ff{tc, 0.f}, kC4), kC3);
  pc = mul_add(z, pc, kC2);
  pc = mul_add(z, pc, kC1);
  const Ff cs = mul_add(z, pc, kOne);
  const Ff a = k & 1 ? sn : cs, b = k & 1 ? cs : sn;
  const float sa = k == 1 || k == 2 ? -1.f : 1.f, sb = k >= 2 ? -1.f : 1.f;  // k in [0, 3]
  return Cplx{Ff{sa * a.h, sa * a.l}, Ff{sb * b.h, sb * b.l}};
}

constexpr int kTableThreads = 256;
constexpr int kMaxRun = 128;

// Thread (pair i, run r) writes the `run` positions from p0 + r * run on, four
// chains of every fourth position at a time.
__global__ void __launch_bounds__(kTableThreads, 3)
    rope_cs_scaled_kernel(float2* out, const RopeFreqs fr, float amp_h, float amp_l, int half, int run, int runs, int max_pos) {
  __shared__ Cplx s_w[2 * kMaxRopePairs];  // e^(i f), then e^(4 i f)
  pdl_wait();
  pdl_trigger();
  const int t = threadIdx.x;
  for (int job = t; job < 2 * half; job += kTableThreads)
    s_w[job] = unit(job < half ? turns(1, fr, job) : turns(4, fr, job - half));
  __syncthreads();
  const int r = t / half, i = t - r * half;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * runs + r) * run;
  if (r >= runs || first >= max_pos) return;
  Cplx z[4];
  z[0] = unit(turns(static_cast<uint32_t>(first), fr, i));
  const Ff amp{amp_h, amp_l}, zero{0.f, 0.f};
  z[0] = Cplx{mul_add(z[0].re, amp, zero), mul_add(z[0].im, amp, zero)};
  const Cplx w = s_w[i], w4 = s_w[half + i];
#pragma unroll
  for (int k = 1; k < 4; ++k) z[k] = mul(z[k - 1], w);
  float2* o = out + first * half + i;
  const int n = max_pos - first < run ? static_cast<int>(max_pos - first) : run;
  for (int k0 = 0; k0 < n; k0 += 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k0 + k < n) o[static_cast<int64_t>(k0 + k) * half] = make_float2(z[k].re.h, z[k].im.h);
      z[k] = mul(z[k], w4);
    }
  }
}

}  // namespace

cudaError_t launch_rope_rows(int elem, const RopeRowsArgs& a, cudaStream_t st) {
  if (elem == GW_ELEM_BF16) return launch_rows<GW_ELEM_BF16>(a, st);
  if (elem == GW_ELEM_F16) return launch_rows<GW_ELEM_F16>(a, st);
  return launch_rows<GW_ELEM_F32>(a, st);
}

cudaError_t launch_rope_cs_scaled(float* out, const RopeFreqs& freqs, double amplitude, int half, int max_pos,
                                  cudaStream_t st) {
  // Long runs need fewer series, short ones keep every SM busy.  kMaxRopePairs
  // is kTableThreads, so a block has at least one run of every pair.
  static_assert(kMaxRopePairs <= kTableThreads, "a thread per pair");
  const int runs = kTableThreads / half;
  int run = kMaxRun;
  while (run > 32 && max_pos < static_cast<int64_t>(run) * runs * 4 * grid_ctas()) run /= 2;
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(max_pos) - 1) / (run * runs) + 1);
  const Ff amp = split(amplitude);
  return launch_pdl(rope_cs_scaled_kernel, dim3(blocks), dim3(kTableThreads), 0, st, reinterpret_cast<float2*>(out),
                    freqs, amp.h, amp.l, half, run, runs, max_pos);
}

}  // namespace gw
