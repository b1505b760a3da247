// C-ABI entry points: host-side validation, workspace carving and dispatch.
//
// Nothing here allocates, frees or synchronises.  Each entry point checks its
// arguments, records a message naming itself on failure, and enqueues kernels
// on the caller's stream.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>
#include <mutex>

#include "gw_internal.h"

namespace gw {
namespace {

thread_local char g_err[512] = "";

gw_status fail(gw_status code, const char* fn, const char* fmt, ...) {
  int n = std::snprintf(g_err, sizeof(g_err), "%s: ", fn);
  if (n < 0) n = 0;
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(g_err + n, sizeof(g_err) - static_cast<size_t>(n), fmt, ap);
  va_end(ap);
  return code;
}

// Bound on the strides that callers give (elements): offsets stay in 64 bits.
constexpr int64_t kMaxRowStride = int64_t{1} << 40;

// gw_rope_rows counts heads in 32 bits, some thousands past the last one.
constexpr int32_t kMaxRopeHeads = 1 << 30;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Pool description checks shared by every entry point.
// `need_base` is false for the size queries, which may run before the pool
// memory exists.
gw_status check_pool(const gw_kv_pool* p, const char* fn, bool need_base = true) {
  if (!p) return fail(GW_ERR_INVALID_ARG, fn, "pool is NULL");
  if (need_base && (!p->base || !aligned(p->base, 256)))
    return fail(GW_ERR_INVALID_ARG, fn, "pool base is NULL or not 256-byte aligned");
  if (p->num_pages < 1) return fail(GW_ERR_INVALID_ARG, fn, "num_pages must be >= 1");
  if (p->page_size != 16) return fail(GW_ERR_INVALID_ARG, fn, "page_size must be 16 (got %d)", p->page_size);
  if (p->dtype != GW_KV_BF16 && p->dtype != GW_KV_E4M3) return fail(GW_ERR_INVALID_ARG, fn, "unknown dtype %d", p->dtype);
  if (p->layout == GW_LAYOUT_LOCAL) {
    if (p->head_dim != 256 || p->rot_dim != 256)
      return fail(GW_ERR_INVALID_ARG, fn, "local pool needs head_dim 256 and rot_dim 256");
    if (p->kv_heads < 1 || p->kv_heads > 64) return fail(GW_ERR_INVALID_ARG, fn, "kv_heads must be in [1, 64]");
  } else if (p->layout == GW_LAYOUT_GLOBAL_FOLDED || p->layout == GW_LAYOUT_GLOBAL_FULL ||
             p->layout == GW_LAYOUT_GLOBAL_FOLDED_E4M3) {
    if (p->head_dim != 512 || p->rot_dim != 128)
      return fail(GW_ERR_INVALID_ARG, fn, "global pool needs head_dim 512 and rot_dim 128");
    if (p->kv_heads != 1) return fail(GW_ERR_INVALID_ARG, fn, "global pool has exactly one KV head");
    if (p->layout == GW_LAYOUT_GLOBAL_FOLDED_E4M3) {
      if (p->dtype != GW_KV_E4M3)
        return fail(GW_ERR_INVALID_ARG, fn, "layout GLOBAL_FOLDED_E4M3 needs dtype e4m3");
    } else if (p->dtype != GW_KV_BF16) {
      return fail(GW_ERR_UNSUPPORTED, fn,
                  "e4m3 KV supports only local (sliding) layers; the opt-in e4m3 global pool is layout "
                  "GLOBAL_FOLDED_E4M3");
    }
  } else {
    return fail(GW_ERR_INVALID_ARG, fn, "unknown layout %d", p->layout);
  }
  return GW_OK;
}

size_t page_bytes(const gw_kv_pool* p) {
  if (p->layout == GW_LAYOUT_LOCAL) return static_cast<size_t>(p->kv_heads) * 2 * 16 * 256 * (p->dtype == GW_KV_BF16 ? 2 : 1);
  if (p->layout == GW_LAYOUT_GLOBAL_FOLDED_E4M3) return 16 * 640;
  return p->layout == GW_LAYOUT_GLOBAL_FOLDED ? 16 * 640 * 2 : 16 * 1024 * 2;
}

gw_status cuda_status(cudaError_t e, const char* fn) {
  if (e == cudaSuccess) return GW_OK;
  return fail(GW_ERR_CUDA, fn, "CUDA error %d (%s)", static_cast<int>(e), cudaGetErrorString(e));
}

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

}  // namespace

gw_status set_error(gw_status code, const char* fn, const char* fmt, ...) {
  int n = std::snprintf(g_err, sizeof(g_err), "%s: ", fn);
  if (n < 0) n = 0;
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(g_err + n, sizeof(g_err) - static_cast<size_t>(n), fmt, ap);
  va_end(ap);
  return code;
}

thread_local int g_max_ctas = 0;
thread_local bool g_early_launch = true;
thread_local bool g_early_inputs = false;

bool early_launch() { return g_early_launch; }
bool early_inputs() { return g_early_inputs; }

int grid_ctas() {
  const int n = num_sms();
  return g_max_ctas > 0 && g_max_ctas < n ? g_max_ctas : n;
}

int num_sms() {
  static int cached = 0;
  static std::once_flag once;
  std::call_once(once, [] {
    int dev = 0;
    cudaGetDevice(&dev);
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    cached = n > 0 ? n : 1;
  });
  return cached;
}

WsLayout ws_layout(int layout, int dtype, int kv_heads, int num_q_heads, int batch, int max_seq_len, int window) {
  WsLayout w{};
  int64_t units;
  if (layout == GW_LAYOUT_LOCAL) {
    const int chunk = dtype == GW_KV_BF16 ? kLocalChunkPagesBf16 : kLocalChunkPagesE4m3;
    const int64_t span = window < max_seq_len ? window : max_seq_len;
    const int64_t pages = ceil_div(span, 16) + 1;
    units = static_cast<int64_t>(batch) * kv_heads * ceil_div(pages, chunk);
    w.heads_per_unit = num_q_heads / kv_heads;
  } else {
    // global_chunks(L) <= min(kGlobalMaxChunks, ceil(pages(L) / 16)) for every L
    const int64_t c16 = ceil_div(ceil_div(max_seq_len, 16), kGlobalChunkPagesMin);
    units = static_cast<int64_t>(batch) * (c16 < kGlobalMaxChunks ? c16 : kGlobalMaxChunks);
    w.heads_per_unit = num_q_heads;
  }
  const int D = layout == GW_LAYOUT_LOCAL ? 256 : 512;
  w.max_units = units;
  w.reserved = 0;
  w.unit_base = 256;
  w.ml = w.unit_base + round_up(static_cast<size_t>(batch + 1) * 4, 256);
  w.o = w.ml + round_up(static_cast<size_t>(units) * w.heads_per_unit * 8, 256);
  w.prompt_base = w.o + round_up(static_cast<size_t>(units) * w.heads_per_unit * D * 4, 256);
  w.total = w.prompt_base + round_up(static_cast<size_t>(batch + 1) * 4, 256);
  return w;
}

}  // namespace gw

using namespace gw;

extern "C" {

const char* gw_last_error(void) { return g_err; }

int32_t gw_version(void) { return 1; }

size_t gw_pool_page_bytes(const gw_kv_pool* pool) {
  if (check_pool(pool, "gw_pool_page_bytes", false) != GW_OK) return 0;
  return page_bytes(pool);
}

gw_status gw_kv_append(const gw_kv_pool* pool, const void* k, const void* v, int32_t num_rows, const int32_t* slot,
                       const int32_t* pos, const float* rope_cs, int32_t max_pos, int32_t* dev_status,
                       void* stream) {
  const char* fn = "gw_kv_append";
  g_err[0] = 0;
  gw_status s = check_pool(pool, fn);
  if (s != GW_OK) return s;
  if (num_rows < 0) return fail(GW_ERR_INVALID_ARG, fn, "num_rows < 0");
  if (num_rows == 0) return GW_OK;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return fail(GW_ERR_INVALID_ARG, fn, "k/v NULL or not 16-byte aligned");
  if (!slot || !pos || !aligned(slot, 4) || !aligned(pos, 4)) return fail(GW_ERR_INVALID_ARG, fn, "slot/pos NULL or misaligned");
  if (!rope_cs || !aligned(rope_cs, 16)) return fail(GW_ERR_INVALID_ARG, fn, "rope_cs NULL or not 16-byte aligned");
  if (max_pos < 1) return fail(GW_ERR_INVALID_ARG, fn, "max_pos must be >= 1");
  if (dev_status && !aligned(dev_status, 4)) return fail(GW_ERR_INVALID_ARG, fn, "dev_status misaligned");
  AppendArgs a{};
  a.pool = static_cast<uint8_t*>(pool->base);
  a.num_pages = pool->num_pages;
  a.kv_heads = pool->kv_heads;
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.num_rows = num_rows;
  a.slot = slot;
  a.pos = pos;
  a.rope_cs = rope_cs;
  a.max_pos = max_pos;
  a.early_inputs = g_early_inputs ? 1 : 0;
  a.status = dev_status;
  return cuda_status(launch_append(pool->layout, pool->dtype, a, static_cast<cudaStream_t>(stream)), fn);
}

gw_status gw_rope_cs(float* rope_cs, double theta, int32_t rot_dim, int32_t head_dim, int32_t max_pos,
                     void* stream) {
  const char* fn = "gw_rope_cs";
  g_err[0] = 0;
  if (!rope_cs || !aligned(rope_cs, 16)) return fail(GW_ERR_INVALID_ARG, fn, "rope_cs NULL or not 16-byte aligned");
  if (!(theta > 0.0) || !std::isfinite(theta)) return fail(GW_ERR_INVALID_ARG, fn, "theta must be finite and > 0");
  if (head_dim < 2 || rot_dim < 2 || rot_dim > head_dim || rot_dim % 2)
    return fail(GW_ERR_INVALID_ARG, fn, "need an even rot_dim in [2, head_dim] (rot_dim %d, head_dim %d)", rot_dim,
                head_dim);
  if (max_pos < 1) return fail(GW_ERR_INVALID_ARG, fn, "max_pos must be >= 1");
  return cuda_status(launch_rope_cs(rope_cs, theta, rot_dim, head_dim, max_pos, static_cast<cudaStream_t>(stream)),
                     fn);
}

gw_status gw_rope_rows(const void* x, int64_t x_row_stride, int64_t x_head_stride, void* y, int64_t y_row_stride,
                       int64_t y_head_stride, int32_t elem, int32_t num_rows, int32_t num_heads, int32_t head_dim,
                       int32_t rot_dim, int32_t pairs, int32_t inverse, const int32_t* pos, const float* rope_cs,
                       int32_t max_pos, int32_t* dev_status, void* stream) {
  const char* fn = "gw_rope_rows";
  g_err[0] = 0;
  if (elem != GW_ELEM_BF16 && elem != GW_ELEM_F16 && elem != GW_ELEM_F32)
    return fail(GW_ERR_INVALID_ARG, fn, "unknown elem %d", elem);
  if (pairs != GW_PAIRS_HALF && pairs != GW_PAIRS_INTERLEAVED)
    return fail(GW_ERR_INVALID_ARG, fn, "unknown pairs %d", pairs);
  if (num_rows < 0 || num_heads < 0) return fail(GW_ERR_INVALID_ARG, fn, "num_rows < 0 or num_heads < 0");
  if (num_heads > kMaxRopeHeads) return fail(GW_ERR_INVALID_ARG, fn, "num_heads (%d) above 2^30", num_heads);
  if (head_dim < 2 || head_dim > 1024 || rot_dim < 2 || rot_dim > head_dim || rot_dim % 2)
    return fail(GW_ERR_INVALID_ARG, fn, "need head_dim in [2, 1024] and an even rot_dim in [2, head_dim] (%d, %d)",
                head_dim, rot_dim);
  if (max_pos < 1) return fail(GW_ERR_INVALID_ARG, fn, "max_pos must be >= 1");
  if (num_rows == 0 || num_heads == 0) return GW_OK;
  const size_t size = elem == GW_ELEM_F32 ? 4 : 2;
  if (!x || !y || !aligned(x, size) || !aligned(y, size)) return fail(GW_ERR_INVALID_ARG, fn, "x/y NULL or misaligned");
  if (!pos || !aligned(pos, 4)) return fail(GW_ERR_INVALID_ARG, fn, "pos NULL or misaligned");
  if (!rope_cs || !aligned(rope_cs, 16)) return fail(GW_ERR_INVALID_ARG, fn, "rope_cs NULL or not 16-byte aligned");
  if (dev_status && !aligned(dev_status, 4)) return fail(GW_ERR_INVALID_ARG, fn, "dev_status misaligned");
  if (x_row_stride < 0 || x_head_stride < 0 || y_row_stride < 0 || y_head_stride < 0 || x_row_stride > kMaxRowStride ||
      x_head_stride > kMaxRowStride || y_row_stride > kMaxRowStride || y_head_stride > kMaxRowStride)
    return fail(GW_ERR_INVALID_ARG, fn, "a stride is negative or above 2^40");
  using wide = unsigned __int128;
  const wide rows1 = num_rows - 1, heads1 = num_heads - 1, dim = head_dim;
  // y: heads within rows, or rows within heads (a dimension of one never overlaps)
  const bool by_row = (num_heads == 1 || y_head_stride >= head_dim) &&
                      (num_rows == 1 || wide(y_row_stride) >= heads1 * y_head_stride + dim);
  const bool by_head = (num_rows == 1 || y_row_stride >= head_dim) &&
                       (num_heads == 1 || wide(y_head_stride) >= rows1 * y_row_stride + dim);
  if (!by_row && !by_head) return fail(GW_ERR_INVALID_ARG, fn, "rows of y overlap one another");
  const bool inplace = x == y;
  if (inplace) {
    if ((num_rows > 1 && x_row_stride != y_row_stride) || (num_heads > 1 && x_head_stride != y_head_stride))
      return fail(GW_ERR_INVALID_ARG, fn, "in place, x and y need the same strides");
  } else {
    const wide x0 = reinterpret_cast<uintptr_t>(x), y0 = reinterpret_cast<uintptr_t>(y);
    const wide x1 = x0 + (rows1 * x_row_stride + heads1 * x_head_stride + dim) * size;
    const wide y1 = y0 + (rows1 * y_row_stride + heads1 * y_head_stride + dim) * size;
    if (x0 < y1 && y0 < x1) return fail(GW_ERR_INVALID_ARG, fn, "x and y overlap and are not the same rows");
  }
  RopeRowsArgs a{};
  a.x = x;
  a.y = y;
  a.x_row = x_row_stride;
  a.x_head = x_head_stride;
  a.y_row = y_row_stride;
  a.y_head = y_head_stride;
  a.num_rows = num_rows;
  a.num_heads = num_heads;
  a.head_dim = head_dim;
  a.rot_dim = rot_dim;
  a.pairs = pairs;
  a.inverse = inverse != 0;
  a.inplace = inplace;
  a.pos = pos;
  a.rope_cs = rope_cs;
  a.max_pos = max_pos;
  a.status = dev_status;
  a.early_inputs = g_early_inputs ? 1 : 0;
  return cuda_status(launch_rope_rows(elem, a, static_cast<cudaStream_t>(stream)), fn);
}

gw_status gw_rope_cs_scaled(float* rope_cs, double theta, int32_t rot_dim, int32_t head_dim, int32_t max_pos,
                            const gw_rope_scaling* scaling, void* stream) {
  const char* fn = "gw_rope_cs_scaled";
  g_err[0] = 0;
  if (!rope_cs || !aligned(rope_cs, 16)) return fail(GW_ERR_INVALID_ARG, fn, "rope_cs NULL or not 16-byte aligned");
  if (!(theta > 0.0) || !std::isfinite(theta)) return fail(GW_ERR_INVALID_ARG, fn, "theta must be finite and > 0");
  if (head_dim < 2 || rot_dim < 2 || rot_dim > head_dim || rot_dim % 2 || rot_dim > 2 * kMaxRopePairs)
    return fail(GW_ERR_INVALID_ARG, fn, "need an even rot_dim in [2, min(head_dim, %d)] (rot_dim %d, head_dim %d)",
                2 * kMaxRopePairs, rot_dim, head_dim);
  if (max_pos < 1) return fail(GW_ERR_INVALID_ARG, fn, "max_pos must be >= 1");
  if (!scaling) return fail(GW_ERR_INVALID_ARG, fn, "scaling is NULL");
  const gw_rope_scaling& sc = *scaling;
  if (sc.kind < GW_ROPE_NONE || sc.kind > GW_ROPE_RAMP || sc.reserved != 0)
    return fail(GW_ERR_INVALID_ARG, fn, "unknown scaling kind %d, or reserved not 0", sc.kind);
  auto positive = [](double v) { return v > 0.0 && std::isfinite(v); };
  if (!(sc.amplitude >= 1e-6 && sc.amplitude <= 1e6))
    return fail(GW_ERR_INVALID_ARG, fn, "amplitude must be in [1e-6, 1e6]");
  if (sc.kind != GW_ROPE_NONE && !positive(sc.factor))
    return fail(GW_ERR_INVALID_ARG, fn, "factor must be finite and > 0");
  if (sc.kind == GW_ROPE_NTK && head_dim <= 2) return fail(GW_ERR_INVALID_ARG, fn, "NTK needs head_dim > 2");
  if (sc.kind == GW_ROPE_RAMP &&
      (!positive(sc.orig_max_pos) || !(sc.low >= 0.0) || !(sc.high > sc.low) || !std::isfinite(sc.high)))
    return fail(GW_ERR_INVALID_ARG, fn, "RAMP needs orig_max_pos > 0 and 0 <= low < high, all finite");
  if (sc.kind == GW_ROPE_NTK) {
    theta *= std::pow(sc.factor, static_cast<double>(head_dim) / (head_dim - 2));
    if (!std::isnormal(theta)) return fail(GW_ERR_INVALID_ARG, fn, "NTK: theta * factor^(...) leaves float64's range");
  }
  RopeFreqs fr{};
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(theta, (-2.0 * i) / head_dim);
    if (sc.kind == GW_ROPE_LINEAR) f /= sc.factor;
    if (sc.kind == GW_ROPE_RAMP) {
      const double turns = sc.orig_max_pos * f / 6.283185307179586;
      double g = (turns - sc.low) / (sc.high - sc.low);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f *= g + (1.0 - g) / sc.factor;
    }
    // beyond 2^52 a float64 angle has no fraction left
    if (!(f * max_pos < 4503599627370496.0)) return fail(GW_ERR_INVALID_ARG, fn, "the angles of pair %d exceed 2^52", i);
    // exact: a double's fraction has at most 53 significant bits, and those
    // below 2^-96 of a turn do not matter over 2^31 positions
    const double turn = f / 6.283185307179586;
    const double hi = std::ldexp(turn - std::floor(turn), 64);
    const double whole = std::floor(hi);
    fr.hi[i] = static_cast<uint64_t>(whole);
    fr.lo[i] = static_cast<uint32_t>(std::ldexp(hi - whole, 32));
  }
  return cuda_status(launch_rope_cs_scaled(rope_cs, fr, sc.amplitude, rot_dim / 2, max_pos,
                                           static_cast<cudaStream_t>(stream)),
                     fn);
}

size_t gw_attn_workspace_bytes(const gw_kv_pool* pool, int32_t num_q_heads, int32_t batch, int32_t max_seq_len,
                               int32_t max_q_rows, int32_t window) {
  (void)max_q_rows;
  if (check_pool(pool, "gw_attn_workspace_bytes", false) != GW_OK) return 0;
  if (num_q_heads < 1 || batch < 0 || max_seq_len < 0) return 0;
  if (pool->layout == GW_LAYOUT_LOCAL && window < 1) return 0;
  if (num_q_heads % pool->kv_heads) return 0;
  const int ms = max_seq_len > 0 ? max_seq_len : 1;
  return ws_layout(pool->layout, pool->dtype, pool->kv_heads, num_q_heads, batch, ms,
                   pool->layout == GW_LAYOUT_LOCAL ? window : 0)
      .total;
}

// Layout of a gw_decode_attn_global_acc workspace: the attention's own, then
// the logits.
struct AccLayout {
  size_t score, total;
};

static AccLayout acc_layout(const WsLayout& w, int num_q_heads, int batch, int max_pages) {
  AccLayout l{};
  l.score = round_up(w.total, 256);
  l.total = l.score + round_up(static_cast<size_t>(batch) * max_pages * 16 * num_q_heads * 4, 256);
  return l;
}

size_t gw_attn_acc_workspace_bytes(const gw_kv_pool* pool, int32_t num_q_heads, int32_t batch,
                                   int32_t max_pages_per_seq) {
  const char* fn = "gw_attn_acc_workspace_bytes";
  if (check_pool(pool, fn, false) != GW_OK) return 0;
  if (pool->layout == GW_LAYOUT_LOCAL || num_q_heads < 1 || batch < 0 || max_pages_per_seq < 1 ||
      max_pages_per_seq > 0x7fffffff / 16) {
    fail(GW_ERR_INVALID_ARG, fn, "needs a global pool, num_q_heads >= 1, batch >= 0 and max_pages_per_seq in [1, 2^27)");
    return 0;
  }
  const WsLayout w = ws_layout(pool->layout, pool->dtype, 1, num_q_heads, batch, max_pages_per_seq * 16, 0);
  return acc_layout(w, num_q_heads, batch, max_pages_per_seq).total;
}

// What gw_decode_attn_global_acc adds to its attention call.
struct AccOut {
  float* acc;
  int64_t stride;
  float decay;
};

// The step's K/V rows of a gw_append_decode_attn_* call.
struct FusedAppend {
  const void* k;
  const void* v;
  const float* rope_cs;
  int32_t max_pos;
};

static gw_status attn_common(const char* fn, bool local, const gw_kv_pool* pool, const void* q, void* out,
                             int32_t num_q_heads, int32_t batch, const int32_t* cu_q_rows, const int32_t* seq_lens,
                             const int32_t* block_table, int32_t max_pages_per_seq, int32_t max_q_rows,
                             int32_t window, float scale, void* workspace, size_t workspace_bytes,
                             int32_t* dev_status, void* stream, bool validate_only = false,
                             float* lse = nullptr, const FusedAppend* app = nullptr, const AccOut* acc = nullptr) {
  g_err[0] = 0;
  gw_status s = check_pool(pool, fn);
  if (s != GW_OK) return s;
  if (app) {
    if (!app->k || !app->v || !aligned(app->k, 16) || !aligned(app->v, 16))
      return fail(GW_ERR_INVALID_ARG, fn, "k/v NULL or not 16-byte aligned");
    if (!app->rope_cs || !aligned(app->rope_cs, 16))
      return fail(GW_ERR_INVALID_ARG, fn, "rope_cs NULL or not 16-byte aligned");
    if (app->max_pos < 1) return fail(GW_ERR_INVALID_ARG, fn, "max_pos must be >= 1");
  }
  if (local && pool->layout != GW_LAYOUT_LOCAL) return fail(GW_ERR_INVALID_ARG, fn, "pool layout is not LOCAL");
  if (!local && pool->layout == GW_LAYOUT_LOCAL) return fail(GW_ERR_INVALID_ARG, fn, "pool layout is not GLOBAL");
  if (batch < 0) return fail(GW_ERR_INVALID_ARG, fn, "batch < 0");
  if (batch == 0) return GW_OK;
  if (num_q_heads < 1 || num_q_heads % pool->kv_heads)
    return fail(GW_ERR_INVALID_ARG, fn, "num_q_heads (%d) must be a positive multiple of kv_heads (%d)", num_q_heads,
                pool->kv_heads);
  const int group = num_q_heads / pool->kv_heads;
  if (local && group != 1 && group != 2 && group != 4 && group != 8)
    return fail(GW_ERR_UNSUPPORTED, fn, "query heads per KV head must be 1, 2, 4 or 8 (got %d)", group);
  if (!local && num_q_heads != 8 && num_q_heads != 16 && num_q_heads != 32)
    return fail(GW_ERR_UNSUPPORTED, fn, "num_q_heads must be 8, 16 or 32 (got %d)", num_q_heads);
  if (local && window < 1) return fail(GW_ERR_INVALID_ARG, fn, "window must be >= 1");
  if (batch > kMaxBatch)
    return fail(GW_ERR_UNSUPPORTED, fn, "batch (%d) exceeds %d sequences per call", batch, kMaxBatch);
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(GW_ERR_INVALID_ARG, fn, "scale must be finite and > 0");
  if (max_pages_per_seq < 1) return fail(GW_ERR_INVALID_ARG, fn, "max_pages_per_seq must be >= 1");
  if (max_q_rows < 1) return fail(GW_ERR_INVALID_ARG, fn, "max_q_rows must be >= 1");
  if (!local && pool->dtype == GW_KV_E4M3 && max_q_rows > 1)
    return fail(GW_ERR_UNSUPPORTED, fn, "prompt rows (max_q_rows %d > 1) on an e4m3 global pool: the global "
                "prompt-row kernel reads bf16 pages only", max_q_rows);
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16)) return fail(GW_ERR_INVALID_ARG, fn, "q/out NULL or not 16-byte aligned");
  if (!cu_q_rows || !seq_lens || !block_table || !aligned(cu_q_rows, 4) || !aligned(seq_lens, 4) ||
      !aligned(block_table, 4))
    return fail(GW_ERR_INVALID_ARG, fn, "cu_q_rows/seq_lens/block_table NULL or misaligned");
  if (dev_status && !aligned(dev_status, 4)) return fail(GW_ERR_INVALID_ARG, fn, "dev_status misaligned");
  if (!workspace || !aligned(workspace, 256)) return fail(GW_ERR_INVALID_ARG, fn, "workspace NULL or not 256-byte aligned");
  const int64_t max_len64 = static_cast<int64_t>(max_pages_per_seq) * 16;
  const int max_len = max_len64 > 0x7fffffff ? 0x7fffffff : static_cast<int>(max_len64);
  const WsLayout w = ws_layout(pool->layout, pool->dtype, pool->kv_heads, num_q_heads, batch, max_len,
                               local ? window : 0);
  size_t ws_need = w.total;
  AccLayout al{};
  if (acc) {
    if (!acc->acc || !aligned(acc->acc, 4)) return fail(GW_ERR_INVALID_ARG, fn, "acc NULL or misaligned");
    if (lse && !aligned(lse, 4)) return fail(GW_ERR_INVALID_ARG, fn, "lse misaligned");
    if (max_pages_per_seq > 0x7fffffff / 16) return fail(GW_ERR_INVALID_ARG, fn, "max_pages_per_seq must be < 2^27");
    if (acc->stride < max_len64)
      return fail(GW_ERR_INVALID_ARG, fn, "acc_stride %lld below max_pages_per_seq * 16 = %lld",
                  static_cast<long long>(acc->stride), static_cast<long long>(max_len64));
    if (!(acc->decay >= 0.f) || !std::isfinite(acc->decay))
      return fail(GW_ERR_INVALID_ARG, fn, "decay must be finite and >= 0");
    al = acc_layout(w, num_q_heads, batch, max_pages_per_seq);
    ws_need = al.total;
  }
  if (workspace_bytes < ws_need)
    return fail(GW_ERR_WORKSPACE, fn, "workspace_bytes %zu < %zu needed", workspace_bytes, ws_need);
  if (validate_only) return GW_OK;

  LocalArgs a{};
  a.pool = static_cast<const uint8_t*>(pool->base);
  a.num_pages = pool->num_pages;
  a.kv_heads = pool->kv_heads;
  a.num_q_heads = num_q_heads;
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.batch = batch;
  a.cu_q_rows = cu_q_rows;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.max_pages = max_pages_per_seq;
  a.window = local ? window : 0x7fffffff;
  a.scale_log2 = scale * 1.4426950408889634f;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.unit_base = reinterpret_cast<int32_t*>(ws + w.unit_base);
  a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.part_o = reinterpret_cast<float*>(ws + w.o);
  a.prompt_base = reinterpret_cast<int32_t*>(ws + w.prompt_base);
  a.max_units = w.max_units;
  a.status = dev_status;
  a.early_inputs = g_early_inputs ? 1 : 0;
  a.lse = lse;
  if (app) {
    a.k_new = static_cast<const uint16_t*>(app->k);
    a.v_new = static_cast<const uint16_t*>(app->v);
    a.rope_cs = app->rope_cs;
    a.max_pos = app->max_pos;
  }
  if (acc) {
    a.score = reinterpret_cast<float*>(ws + al.score);
    a.acc = acc->acc;
    a.acc_stride = acc->stride;
    a.decay = acc->decay;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (local) {
    e = launch_local_decode(pool->dtype, group, a, st);
    if (e == cudaSuccess && max_q_rows > 1) e = launch_local_prompt(pool->dtype, group, a, max_q_rows, st);
  } else {
    e = launch_global_decode(pool->layout, a, st);
    if (e == cudaSuccess && max_q_rows > 1) e = launch_global_prompt(pool->layout, a, max_q_rows, st);
  }
  return cuda_status(e, fn);
}

gw_status gw_decode_attn_local(const gw_kv_pool* pool, const void* q, void* out, int32_t num_q_heads, int32_t batch,
                               const int32_t* cu_q_rows, const int32_t* seq_lens, const int32_t* block_table,
                               int32_t max_pages_per_seq, int32_t max_q_rows, int32_t window, float scale,
                               void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  return attn_common("gw_decode_attn_local", true, pool, q, out, num_q_heads, batch, cu_q_rows, seq_lens, block_table,
                     max_pages_per_seq, max_q_rows, window, scale, workspace, workspace_bytes, dev_status, stream);
}

}  // extern "C"

namespace gw {
gw_status validate_local_call(const char* fn, const gw_kv_pool* pool, const void* q, void* out, int32_t num_q_heads,
                              int32_t batch, const int32_t* cu_q_rows, const int32_t* seq_lens,
                              const int32_t* block_table, int32_t max_pages_per_seq, int32_t max_q_rows,
                              int32_t window, float scale, size_t workspace_bytes, int32_t* dev_status) {
  // Any 256-byte aligned non-null address stands in for the workspace: only
  // its size is checked, and nothing is launched.
  return attn_common(fn, true, pool, q, out, num_q_heads, batch, cu_q_rows, seq_lens, block_table, max_pages_per_seq,
                     max_q_rows, window, scale, reinterpret_cast<void*>(static_cast<uintptr_t>(256)), workspace_bytes,
                     dev_status, nullptr, true);
}
}  // namespace gw

extern "C" {

gw_status gw_append_decode_attn_local(const gw_kv_pool* pool, const void* k, const void* v, const float* rope_cs,
                                      int32_t max_pos, const void* q, void* out, int32_t num_q_heads, int32_t batch,
                                      const int32_t* cu_q_rows, const int32_t* seq_lens, const int32_t* block_table,
                                      int32_t max_pages_per_seq, int32_t window, float scale, void* workspace,
                                      size_t workspace_bytes, int32_t* dev_status, void* stream) {
  const FusedAppend app{k, v, rope_cs, max_pos};
  return attn_common("gw_append_decode_attn_local", true, pool, q, out, num_q_heads, batch, cu_q_rows, seq_lens,
                     block_table, max_pages_per_seq, 1, window, scale, workspace, workspace_bytes, dev_status, stream,
                     false, nullptr, &app);
}

gw_status gw_append_decode_attn_global(const gw_kv_pool* pool, const void* k, const void* v, const float* rope_cs,
                                       int32_t max_pos, const void* q, void* out, int32_t num_q_heads, int32_t batch,
                                       const int32_t* cu_q_rows, const int32_t* seq_lens, const int32_t* block_table,
                                       int32_t max_pages_per_seq, float scale, void* workspace,
                                       size_t workspace_bytes, int32_t* dev_status, void* stream) {
  const FusedAppend app{k, v, rope_cs, max_pos};
  return attn_common("gw_append_decode_attn_global", false, pool, q, out, num_q_heads, batch, cu_q_rows, seq_lens,
                     block_table, max_pages_per_seq, 1, 0, scale, workspace, workspace_bytes, dev_status, stream,
                     false, nullptr, &app);
}

gw_status gw_decode_attn_global(const gw_kv_pool* pool, const void* q, void* out, int32_t num_q_heads, int32_t batch,
                                const int32_t* cu_q_rows, const int32_t* seq_lens, const int32_t* block_table,
                                int32_t max_pages_per_seq, int32_t max_q_rows, float scale, void* workspace,
                                size_t workspace_bytes, int32_t* dev_status, void* stream) {
  return attn_common("gw_decode_attn_global", false, pool, q, out, num_q_heads, batch, cu_q_rows, seq_lens,
                     block_table, max_pages_per_seq, max_q_rows, 0, scale, workspace, workspace_bytes, dev_status,
                     stream);
}

gw_status gw_decode_attn_global_lse(const gw_kv_pool* pool, const void* q, void* out, float* lse,
                                    int32_t num_q_heads, int32_t batch, const int32_t* cu_q_rows,
                                    const int32_t* seq_lens, const int32_t* block_table, int32_t max_pages_per_seq,
                                    float scale, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                    void* stream) {
  const char* fn = "gw_decode_attn_global_lse";
  if (!lse || !aligned(lse, 4)) {
    g_err[0] = 0;
    return fail(GW_ERR_INVALID_ARG, fn, "lse NULL or misaligned");
  }
  return attn_common(fn, false, pool, q, out, num_q_heads, batch, cu_q_rows, seq_lens, block_table,
                     max_pages_per_seq, 1, 0, scale, workspace, workspace_bytes, dev_status, stream, false, lse);
}

gw_status gw_decode_attn_global_acc(const gw_kv_pool* pool, const void* q, void* out, float* lse, float* acc,
                                    int64_t acc_stride, float decay, int32_t num_q_heads, int32_t batch,
                                    const int32_t* cu_q_rows, const int32_t* seq_lens, const int32_t* block_table,
                                    int32_t max_pages_per_seq, float scale, void* workspace, size_t workspace_bytes,
                                    int32_t* dev_status, void* stream) {
  const AccOut ao{acc, acc_stride, decay};
  return attn_common("gw_decode_attn_global_acc", false, pool, q, out, num_q_heads, batch, cu_q_rows, seq_lens,
                     block_table, max_pages_per_seq, 1, 0, scale, workspace, workspace_bytes, dev_status, stream, false,
                     lse, nullptr, &ao);
}

gw_status gw_kv_evict_select(const float* acc, int64_t acc_stride, int32_t batch, const int32_t* seq_lens,
                             int32_t budget, int32_t sinks, int32_t recent, int32_t* keep_idx, int64_t keep_stride,
                             int32_t* keep_lens, int32_t* dev_status, void* stream) {
  const char* fn = "gw_kv_evict_select";
  g_err[0] = 0;
  if (batch < 0 || batch > 65535) return fail(GW_ERR_INVALID_ARG, fn, "batch (%d) outside [0, 65535]", batch);
  if (budget < 1 || sinks < 0 || recent < 0 || static_cast<int64_t>(sinks) + recent > budget)
    return fail(GW_ERR_INVALID_ARG, fn, "need budget >= 1, sinks >= 0, recent >= 0 and sinks + recent <= budget (%d, %d, %d)",
                budget, sinks, recent);
  if (acc_stride < 1 || acc_stride > kMaxRowStride || keep_stride < budget || keep_stride > kMaxRowStride)
    return fail(GW_ERR_INVALID_ARG, fn, "acc_stride < 1, keep_stride < budget, or one above 2^40");
  if (batch == 0) return GW_OK;
  if (!acc || !aligned(acc, 4)) return fail(GW_ERR_INVALID_ARG, fn, "acc NULL or misaligned");
  if (!seq_lens || !keep_idx || !keep_lens || !aligned(seq_lens, 4) || !aligned(keep_idx, 4) || !aligned(keep_lens, 4))
    return fail(GW_ERR_INVALID_ARG, fn, "seq_lens/keep_idx/keep_lens NULL or misaligned");
  if (seq_lens == keep_lens) return fail(GW_ERR_INVALID_ARG, fn, "seq_lens and keep_lens are the same array");
  if (dev_status && !aligned(dev_status, 4)) return fail(GW_ERR_INVALID_ARG, fn, "dev_status misaligned");
  SelectArgs a{};
  a.acc = acc;
  a.acc_stride = acc_stride;
  a.batch = batch;
  a.seq_lens = seq_lens;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  a.keep_idx = keep_idx;
  a.keep_stride = keep_stride;
  a.keep_lens = keep_lens;
  a.status = dev_status;
  return cuda_status(launch_evict_select(a, static_cast<cudaStream_t>(stream)), fn);
}

gw_status gw_kv_evict_compact(const gw_kv_pool* pool, int32_t batch, const int32_t* block_table,
                              int32_t max_pages_per_seq, const int32_t* seq_lens, const int32_t* keep_idx,
                              int64_t keep_stride, const int32_t* keep_lens, const int32_t* dst_block_table,
                              int32_t dst_max_pages, float* acc, int64_t acc_stride, int32_t* dev_status,
                              void* stream) {
  const char* fn = "gw_kv_evict_compact";
  g_err[0] = 0;
  gw_status s = check_pool(pool, fn);
  if (s != GW_OK) return s;
  if (pool->layout == GW_LAYOUT_LOCAL)
    return fail(GW_ERR_UNSUPPORTED, fn, "a LOCAL pool: sliding-window layers evict by their window");
  if (batch < 0 || batch > 65535) return fail(GW_ERR_INVALID_ARG, fn, "batch (%d) outside [0, 65535]", batch);
  if (max_pages_per_seq < 1 || max_pages_per_seq > 0x7fffffff / 16)
    return fail(GW_ERR_INVALID_ARG, fn, "max_pages_per_seq must be in [1, 2^27)");
  if (dst_block_table && (dst_max_pages < 1 || dst_max_pages > 0x7fffffff / 16))
    return fail(GW_ERR_INVALID_ARG, fn, "dst_max_pages must be in [1, 2^27)");
  if (keep_stride < 1 || keep_stride > kMaxRowStride) return fail(GW_ERR_INVALID_ARG, fn, "keep_stride < 1 or above 2^40");
  if (acc && (!aligned(acc, 4) || acc_stride < static_cast<int64_t>(max_pages_per_seq) * 16 || acc_stride > kMaxRowStride))
    return fail(GW_ERR_INVALID_ARG, fn, "acc misaligned, or acc_stride below max_pages_per_seq * 16 or above 2^40");
  if (batch == 0) return GW_OK;
  if (!block_table || !seq_lens || !keep_idx || !keep_lens || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(keep_idx, 4) || !aligned(keep_lens, 4) || !aligned(dst_block_table, 4))
    return fail(GW_ERR_INVALID_ARG, fn, "block_table/seq_lens/keep_idx/keep_lens NULL or misaligned");
  if (seq_lens == keep_lens) return fail(GW_ERR_INVALID_ARG, fn, "seq_lens and keep_lens are the same array");
  if (dev_status && !aligned(dev_status, 4)) return fail(GW_ERR_INVALID_ARG, fn, "dev_status misaligned");
  CompactArgs a{};
  a.pool = static_cast<uint8_t*>(pool->base);
  a.num_pages = pool->num_pages;
  a.batch = batch;
  a.block_table = block_table;
  a.max_pages = max_pages_per_seq;
  a.seq_lens = seq_lens;
  a.keep_idx = keep_idx;
  a.keep_stride = keep_stride;
  a.keep_lens = keep_lens;
  a.dst_table = dst_block_table ? dst_block_table : block_table;
  a.dst_max_pages = dst_block_table ? dst_max_pages : max_pages_per_seq;
  a.acc = acc;
  a.acc_stride = acc_stride;
  a.status = dev_status;
  return cuda_status(launch_evict_compact(pool->layout, a, static_cast<cudaStream_t>(stream)), fn);
}

// Layout of a gw_tree_attn_* workspace: the plan, then (m, l) and the fp32 rows
// of every unit of sequences that have several chunks.
struct TreeLayout {
  size_t unit_base, ml, o, total;
  int part_rows;
};

static TreeLayout tree_layout(const gw_kv_pool* pool, int num_q_heads, int batch, int max_pages, int max_q_rows,
                              int window) {
  const bool local = pool->layout == GW_LAYOUT_LOCAL;
  const int group = local ? num_q_heads / pool->kv_heads : num_q_heads;
  const int per = kTreeRows / group, copies = local ? pool->kv_heads : 2;
  const bool few = !local && max_q_rows * group <= tree_few_rows(pool->layout);
  const TreeRule rule = local ? tree_rule_local(group) : few ? tree_rule_few(group) : tree_rule_global(group);
  const int chunks = tree_max_chunks(max_pages, max_q_rows, local ? window : 0x7fffffff, rule);
  // the most units of a sequence, over the blocks of its rows
  int64_t units = 0;
  for (int blocks = 1; blocks <= ceil_div(max_q_rows, per); ++blocks) {
    const int most = tree_most_chunks(rule, blocks);
    const int64_t u = static_cast<int64_t>(blocks) * (chunks < most ? chunks : most);
    if (u > units) units = u;
  }
  units *= static_cast<int64_t>(copies) * batch;
  TreeLayout l{};
  l.part_rows = group * (per < max_q_rows ? per : max_q_rows);
  l.unit_base = 0;
  l.ml = round_up(static_cast<size_t>(batch + 1) * 4, 256);
  if (chunks == 1) {
    l.o = l.total = l.ml;
    return l;
  }
  l.o = l.ml + round_up(static_cast<size_t>(units) * l.part_rows * 8, 256);
  l.total = l.o + round_up(static_cast<size_t>(units) * l.part_rows * 256 * 4, 256);
  return l;
}

// What a call of this size or any smaller one needs.  With fewer rows or heads a
// global call takes the kernel that has them along N, whose chunks are shorter and
// more: 8 heads over 2560 tokens, 64 rows have one chunk and 4 rows 5.  For one
// count of heads and one kernel the need grows with the rows, so that the most rows
// of each kernel are enough.
static size_t tree_bytes(const gw_kv_pool* pool, int num_q_heads, int batch, int max_pages, int max_q_rows,
                         int window) {
  const bool local = pool->layout == GW_LAYOUT_LOCAL;
  const int kv = local ? pool->kv_heads : 1, few = tree_few_rows(pool->layout);
  size_t most = 0;
  for (int group = local ? 1 : 8; group <= num_q_heads / kv; group *= 2) {
    auto need = [&](int rows) {
      const size_t n = tree_layout(pool, group * kv, batch, max_pages, rows, window).total;
      if (n > most) most = n;
    };
    need(max_q_rows);
    if (!local && max_q_rows * group > few) need(few / group);
  }
  return most;
}

// The geometry that a gw_tree_attn_* call and its workspace share.
static gw_status check_tree(const char* fn, const gw_kv_pool* pool, int32_t num_q_heads, int32_t batch,
                            int32_t max_pages_per_seq, int32_t max_q_rows, int32_t window) {
  const bool local = pool->layout == GW_LAYOUT_LOCAL;
  if (batch < 0) return fail(GW_ERR_INVALID_ARG, fn, "batch < 0");
  if (num_q_heads < 1 || num_q_heads % pool->kv_heads)
    return fail(GW_ERR_INVALID_ARG, fn, "num_q_heads (%d) must be a positive multiple of kv_heads (%d)", num_q_heads,
                pool->kv_heads);
  const int group = num_q_heads / pool->kv_heads;
  if (local && group != 1 && group != 2 && group != 4 && group != 8)
    return fail(GW_ERR_UNSUPPORTED, fn, "query heads per KV head must be 1, 2, 4 or 8 (got %d)", group);
  if (!local && num_q_heads != 8 && num_q_heads != 16 && num_q_heads != 32)
    return fail(GW_ERR_UNSUPPORTED, fn, "num_q_heads must be 8, 16 or 32 (got %d)", num_q_heads);
  if (batch > kMaxTreeBatch)
    return fail(GW_ERR_UNSUPPORTED, fn, "batch (%d) exceeds %d sequences per call", batch, kMaxTreeBatch);
  if (local && window < 1) return fail(GW_ERR_INVALID_ARG, fn, "window must be >= 1");
  // a token's index and the end of its tile fit 31 bits
  if (max_pages_per_seq < 1 || max_pages_per_seq >= 1 << 26)
    return fail(GW_ERR_INVALID_ARG, fn, "max_pages_per_seq must be in [1, 2^26)");
  if (max_q_rows < 1 || max_q_rows > kMaxTreeRows)
    return fail(GW_ERR_INVALID_ARG, fn, "max_q_rows (%d) outside [1, %d]", max_q_rows, kMaxTreeRows);
  return GW_OK;
}

size_t gw_tree_workspace_bytes(const gw_kv_pool* pool, int32_t num_q_heads, int32_t batch, int32_t max_pages_per_seq,
                               int32_t max_q_rows, int32_t window) {
  const char* fn = "gw_tree_workspace_bytes";
  g_err[0] = 0;
  if (check_pool(pool, fn, false) != GW_OK) return 0;
  if (check_tree(fn, pool, num_q_heads, batch, max_pages_per_seq, max_q_rows, window) != GW_OK) return 0;
  return tree_bytes(pool, num_q_heads, batch, max_pages_per_seq, max_q_rows, window);
}

static gw_status tree_attn(const char* fn, bool local, const gw_kv_pool* pool, const void* q, void* out,
                           int32_t num_q_heads, int32_t batch, const int32_t* cu_q_rows, const int32_t* seq_lens,
                           const int32_t* block_table, int32_t max_pages_per_seq, const uint64_t* tree_mask,
                           const int32_t* pos, int32_t max_q_rows, int32_t window, float scale, void* workspace,
                           size_t workspace_bytes, int32_t* dev_status, void* stream) {
  g_err[0] = 0;
  gw_status s = check_pool(pool, fn);
  if (s != GW_OK) return s;
  if (local && pool->layout != GW_LAYOUT_LOCAL) return fail(GW_ERR_INVALID_ARG, fn, "pool layout is not LOCAL");
  if (!local && pool->layout == GW_LAYOUT_LOCAL) return fail(GW_ERR_INVALID_ARG, fn, "pool layout is not GLOBAL");
  s = check_tree(fn, pool, num_q_heads, batch, max_pages_per_seq, max_q_rows, window);
  if (s != GW_OK) return s;
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(GW_ERR_INVALID_ARG, fn, "scale must be finite and > 0");
  if (batch == 0) return GW_OK;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16)) return fail(GW_ERR_INVALID_ARG, fn, "q/out NULL or not 16-byte aligned");
  if (!cu_q_rows || !seq_lens || !block_table || !aligned(cu_q_rows, 4) || !aligned(seq_lens, 4) ||
      !aligned(block_table, 4))
    return fail(GW_ERR_INVALID_ARG, fn, "cu_q_rows/seq_lens/block_table NULL or misaligned");
  if (!tree_mask || !aligned(tree_mask, 8)) return fail(GW_ERR_INVALID_ARG, fn, "tree_mask NULL or not 8-byte aligned");
  if (local && (!pos || !aligned(pos, 4))) return fail(GW_ERR_INVALID_ARG, fn, "pos NULL or misaligned");
  if (dev_status && !aligned(dev_status, 4)) return fail(GW_ERR_INVALID_ARG, fn, "dev_status misaligned");
  if (!workspace || !aligned(workspace, 256)) return fail(GW_ERR_INVALID_ARG, fn, "workspace NULL or not 256-byte aligned");
  const TreeLayout w = tree_layout(pool, num_q_heads, batch, max_pages_per_seq, max_q_rows, window);
  if (workspace_bytes < w.total)
    return fail(GW_ERR_WORKSPACE, fn, "workspace_bytes %zu < %zu needed", workspace_bytes, w.total);
  // one half of a row may be written while the other half's unit has yet to read q
  if (!local && q == out) return fail(GW_ERR_INVALID_ARG, fn, "out is q: a global call's rows are not computed in place");
  LocalArgs a{};
  a.pool = static_cast<const uint8_t*>(pool->base);
  a.num_pages = pool->num_pages;
  a.kv_heads = pool->kv_heads;
  a.num_q_heads = num_q_heads;
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.batch = batch;
  a.cu_q_rows = cu_q_rows;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.max_pages = max_pages_per_seq;
  a.window = local ? window : 0x7fffffff;
  a.scale_log2 = scale * 1.4426950408889634f;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.unit_base = reinterpret_cast<int32_t*>(ws + w.unit_base);
  a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.part_o = reinterpret_cast<float*>(ws + w.o);
  a.status = dev_status;
  a.tree_mask = tree_mask;
  a.tree_pos = pos;
  a.max_q_rows = max_q_rows;
  a.part_rows = w.part_rows;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cuda_status(local ? launch_local_tree(pool->dtype, num_q_heads / pool->kv_heads, a, st)
                           : launch_global_tree(pool->layout, a, st),
                     fn);
}

gw_status gw_tree_attn_local(const gw_kv_pool* pool, const void* q, void* out, int32_t num_q_heads, int32_t batch,
                             const int32_t* cu_q_rows, const int32_t* seq_lens, const int32_t* block_table,
                             int32_t max_pages_per_seq, const uint64_t* tree_mask, const int32_t* pos,
                             int32_t max_q_rows, int32_t window, float scale, void* workspace, size_t workspace_bytes,
                             int32_t* dev_status, void* stream) {
  return tree_attn("gw_tree_attn_local", true, pool, q, out, num_q_heads, batch, cu_q_rows, seq_lens, block_table,
                   max_pages_per_seq, tree_mask, pos, max_q_rows, window, scale, workspace, workspace_bytes,
                   dev_status, stream);
}

gw_status gw_tree_attn_global(const gw_kv_pool* pool, const void* q, void* out, int32_t num_q_heads, int32_t batch,
                              const int32_t* cu_q_rows, const int32_t* seq_lens, const int32_t* block_table,
                              int32_t max_pages_per_seq, const uint64_t* tree_mask, int32_t max_q_rows, float scale,
                              void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  return tree_attn("gw_tree_attn_global", false, pool, q, out, num_q_heads, batch, cu_q_rows, seq_lens, block_table,
                   max_pages_per_seq, tree_mask, nullptr, max_q_rows, 0, scale, workspace, workspace_bytes, dev_status,
                   stream);
}

gw_status gw_norm_rope_append(const gw_kv_pool* pool, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                              const void* k, int64_t k_row_stride, int64_t k_head_stride, const void* v,
                              int64_t v_row_stride, int64_t v_head_stride, int32_t num_rows, int32_t num_q_heads,
                              const float* q_weight, const float* k_weight, float eps, int32_t v_norm,
                              const int32_t* slot, const int32_t* pos, const float* rope_cs, int32_t max_pos,
                              void* q_out, int32_t* dev_status, void* stream) {
  const char* fn = "gw_norm_rope_append";
  g_err[0] = 0;
  gw_status s = check_pool(pool, fn);
  if (s != GW_OK) return s;
  if (num_rows < 0) return fail(GW_ERR_INVALID_ARG, fn, "num_rows < 0");
  if (num_q_heads < 1 || num_q_heads > 1024)
    return fail(GW_ERR_INVALID_ARG, fn, "num_q_heads (%d) outside [1, 1024]", num_q_heads);
  if (!(eps > 0.f) || !std::isfinite(eps)) return fail(GW_ERR_INVALID_ARG, fn, "eps must be finite and > 0");
  if (max_pos < 1) return fail(GW_ERR_INVALID_ARG, fn, "max_pos must be >= 1");
  if (num_rows == 0) return GW_OK;
  if (!q || !k || !v || !q_out || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16))
    return fail(GW_ERR_INVALID_ARG, fn, "q/k/v/q_out NULL or not 16-byte aligned");
  // the stride of a dimension of one is not used
  if (num_rows == 1) q_row_stride = k_row_stride = v_row_stride = 0;
  if (num_q_heads == 1) q_head_stride = 0;
  if (pool->kv_heads == 1) k_head_stride = v_head_stride = 0;
  for (int64_t d : {q_row_stride, q_head_stride, k_row_stride, k_head_stride, v_row_stride, v_head_stride})
    if (d < 0 || d > kMaxRowStride || d % 8)
      return fail(GW_ERR_INVALID_ARG, fn, "a stride (%lld) is negative, above 2^40 or not a multiple of 8 elements",
                  static_cast<long long>(d));
  if (!q_weight || !k_weight || !aligned(q_weight, 16) || !aligned(k_weight, 16))
    return fail(GW_ERR_INVALID_ARG, fn, "q_weight/k_weight NULL or not 16-byte aligned");
  if (!slot || !pos || !aligned(slot, 4) || !aligned(pos, 4)) return fail(GW_ERR_INVALID_ARG, fn, "slot/pos NULL or misaligned");
  if (!rope_cs || !aligned(rope_cs, 16)) return fail(GW_ERR_INVALID_ARG, fn, "rope_cs NULL or not 16-byte aligned");
  if (dev_status && !aligned(dev_status, 4)) return fail(GW_ERR_INVALID_ARG, fn, "dev_status misaligned");
  const bool same_kv = k == v && k_row_stride == v_row_stride;  // a global pool has one KV head
  const bool folded = pool->layout == GW_LAYOUT_GLOBAL_FOLDED || pool->layout == GW_LAYOUT_GLOBAL_FOLDED_E4M3;
  if (folded && (!same_kv || !v_norm))
    return fail(GW_ERR_INVALID_ARG, fn, "a folded pool's K and V are one projection: v must be k, with v_norm");
  using wide = unsigned __int128;
  const wide dim = pool->head_dim, rows1 = num_rows - 1, q0 = reinterpret_cast<uintptr_t>(q_out);
  const wide out_end = q0 + (wide(num_rows) * num_q_heads * dim) * 2;
  auto overlaps = [&](const void* x, int64_t row, int64_t head, int heads) {
    const wide x0 = reinterpret_cast<uintptr_t>(x);
    return x0 < out_end && q0 < x0 + (rows1 * row + wide(heads - 1) * head + dim) * 2;
  };
  if (q == q_out) {
    if ((num_q_heads > 1 && wide(q_head_stride) != dim) || (num_rows > 1 && wide(q_row_stride) != num_q_heads * dim))
      return fail(GW_ERR_INVALID_ARG, fn, "in place, q must be contiguous");
  } else if (overlaps(q, q_row_stride, q_head_stride, num_q_heads)) {
    return fail(GW_ERR_INVALID_ARG, fn, "q_out overlaps q and is not the same rows");
  }
  if (overlaps(k, k_row_stride, k_head_stride, pool->kv_heads) || overlaps(v, v_row_stride, v_head_stride, pool->kv_heads))
    return fail(GW_ERR_INVALID_ARG, fn, "q_out overlaps k or v");
  NormRopeArgs a{};
  a.pool = static_cast<uint8_t*>(pool->base);
  a.num_pages = pool->num_pages;
  a.kv_heads = pool->kv_heads;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_row = q_row_stride;
  a.q_head = q_head_stride;
  a.k_row = k_row_stride;
  a.k_head = k_head_stride;
  a.v_row = v_row_stride;
  a.v_head = v_head_stride;
  a.num_rows = num_rows;
  a.num_q_heads = num_q_heads;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.v_norm = v_norm != 0;
  a.tied = pool->layout != GW_LAYOUT_LOCAL && same_kv;
  a.slot = slot;
  a.pos = pos;
  a.rope_cs = rope_cs;
  a.max_pos = max_pos;
  a.out = static_cast<uint16_t*>(q_out);
  a.status = dev_status;
  a.early_inputs = g_early_inputs ? 1 : 0;
  return cuda_status(launch_norm_rope(pool->layout, pool->dtype, a, static_cast<cudaStream_t>(stream)), fn);
}

gw_status gw_tree_accept(int32_t batch, const int32_t* cu_q_rows, const int32_t* seq_lens, int32_t max_q_rows,
                         const int32_t* parent, const int32_t* draft, const int32_t* target, int32_t* path,
                         int64_t path_stride, int32_t* path_lens, int32_t* next_tokens, int32_t* new_lens,
                         int32_t* dev_status, void* stream) {
  const char* fn = "gw_tree_accept";
  g_err[0] = 0;
  if (batch < 0 || batch > 65535) return fail(GW_ERR_INVALID_ARG, fn, "batch (%d) outside [0, 65535]", batch);
  if (max_q_rows < 1 || max_q_rows > kMaxTreeRows)
    return fail(GW_ERR_INVALID_ARG, fn, "max_q_rows (%d) outside [1, %d]", max_q_rows, kMaxTreeRows);
  if (path_stride < max_q_rows || path_stride > kMaxRowStride)
    return fail(GW_ERR_INVALID_ARG, fn, "path_stride below max_q_rows or above 2^40");
  if (batch == 0) return GW_OK;
  const void* in[] = {cu_q_rows, seq_lens, parent, draft, target, path, path_lens};
  for (const void* p : in)
    if (!p || !aligned(p, 4))
      return fail(GW_ERR_INVALID_ARG, fn, "cu_q_rows/seq_lens/parent/draft/target/path/path_lens NULL or misaligned");
  if (!aligned(next_tokens, 4) || !aligned(new_lens, 4)) return fail(GW_ERR_INVALID_ARG, fn, "next_tokens/new_lens misaligned");
  if (dev_status && !aligned(dev_status, 4)) return fail(GW_ERR_INVALID_ARG, fn, "dev_status misaligned");
  if (seq_lens == path_lens) return fail(GW_ERR_INVALID_ARG, fn, "seq_lens and path_lens are the same array");
  const void* outs[] = {path, path_lens, next_tokens, new_lens};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (outs[i] && outs[i] == outs[j])
        return fail(GW_ERR_INVALID_ARG, fn, "two of path, path_lens, next_tokens and new_lens are the same array");
  TreeAcceptArgs a{};
  a.batch = batch;
  a.max_q_rows = max_q_rows;
  a.cu_q_rows = cu_q_rows;
  a.seq_lens = seq_lens;
  a.parent = parent;
  a.draft = draft;
  a.target = target;
  a.path = path;
  a.path_stride = path_stride;
  a.path_lens = path_lens;
  a.next_tokens = next_tokens;
  a.new_lens = new_lens;
  a.status = dev_status;
  return cuda_status(launch_tree_accept(a, static_cast<cudaStream_t>(stream)), fn);
}

gw_status gw_kv_tree_move(const gw_kv_pool* pools, int32_t n_pools, int32_t batch, const int32_t* cu_q_rows,
                          const int32_t* seq_lens, const int32_t* block_table, int32_t max_pages_per_seq,
                          const int32_t* path, int64_t path_stride, const int32_t* path_lens, int32_t* dev_status,
                          void* stream) {
  const char* fn = "gw_kv_tree_move";
  g_err[0] = 0;
  if (!pools) return fail(GW_ERR_INVALID_ARG, fn, "pools is NULL");
  if (n_pools < 1 || n_pools > kMaxTreePools)
    return fail(GW_ERR_INVALID_ARG, fn, "n_pools (%d) outside [1, %d]", n_pools, kMaxTreePools);
  TreeMoveArgs a{};
  for (int i = 0; i < n_pools; ++i) {
    const gw_status s = check_pool(pools + i, fn);
    if (s != GW_OK) return s;
    if (pools[i].layout != pools[0].layout || pools[i].dtype != pools[0].dtype || pools[i].kv_heads != pools[0].kv_heads)
      return fail(GW_ERR_INVALID_ARG, fn, "pool %d differs from the first in layout, dtype or kv_heads", i);
    a.pools[i] = static_cast<uint8_t*>(pools[i].base);
    a.num_pages[i] = pools[i].num_pages;
    for (int j = 0; j < i; ++j)
      if (a.pools[j] == a.pools[i]) return fail(GW_ERR_INVALID_ARG, fn, "pools %d and %d are the same memory", j, i);
  }
  if (batch < 0 || batch > 65535) return fail(GW_ERR_INVALID_ARG, fn, "batch (%d) outside [0, 65535]", batch);
  if (max_pages_per_seq < 1 || max_pages_per_seq > 0x7fffffff / 16)
    return fail(GW_ERR_INVALID_ARG, fn, "max_pages_per_seq must be in [1, 2^27)");
  if (path_stride < 1 || path_stride > kMaxRowStride) return fail(GW_ERR_INVALID_ARG, fn, "path_stride < 1 or above 2^40");
  if (batch == 0) return GW_OK;
  const void* in[] = {cu_q_rows, seq_lens, block_table, path, path_lens};
  for (const void* p : in)
    if (!p || !aligned(p, 4))
      return fail(GW_ERR_INVALID_ARG, fn, "cu_q_rows/seq_lens/block_table/path/path_lens NULL or misaligned");
  if (dev_status && !aligned(dev_status, 4)) return fail(GW_ERR_INVALID_ARG, fn, "dev_status misaligned");
  a.page_bytes = static_cast<int64_t>(page_bytes(pools));
  a.pieces = static_cast<int32_t>(a.page_bytes / (16 * kPageTokens));
  a.batch = batch;
  a.cu_q_rows = cu_q_rows;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.max_pages = max_pages_per_seq;
  a.path = path;
  a.path_stride = path_stride;
  a.path_lens = path_lens;
  a.status = dev_status;
  return cuda_status(launch_tree_move(pools->layout, pools->dtype, n_pools, a, static_cast<cudaStream_t>(stream)), fn);
}

gw_status gw_merge_lse(int32_t n_parts, const void* const* o_parts, const float* const* lse_parts, void* out,
                       float* lse_out, int32_t rows, int32_t num_heads, int32_t head_dim, void* stream) {
  const char* fn = "gw_merge_lse";
  g_err[0] = 0;
  if (n_parts < 1 || n_parts > kMaxMergeParts)
    return fail(GW_ERR_INVALID_ARG, fn, "n_parts (%d) outside [1, %d]", n_parts, kMaxMergeParts);
  if (rows < 0 || num_heads < 1) return fail(GW_ERR_INVALID_ARG, fn, "rows < 0 or num_heads < 1");
  if (head_dim != 256 && head_dim != 512) return fail(GW_ERR_INVALID_ARG, fn, "head_dim must be 256 or 512");
  if (!o_parts || !lse_parts) return fail(GW_ERR_INVALID_ARG, fn, "o_parts/lse_parts NULL");
  if (!out || !aligned(out, 16)) return fail(GW_ERR_INVALID_ARG, fn, "out NULL or not 16-byte aligned");
  if (lse_out && !aligned(lse_out, 4)) return fail(GW_ERR_INVALID_ARG, fn, "lse_out misaligned");
  MergeArgs m{};
  for (int r = 0; r < n_parts; ++r) {
    if (!o_parts[r] || !aligned(o_parts[r], 16) || !lse_parts[r] || !aligned(lse_parts[r], 4))
      return fail(GW_ERR_INVALID_ARG, fn, "part %d: o NULL or not 16-byte aligned, or lse NULL or misaligned", r);
    m.o[r] = static_cast<const uint16_t*>(o_parts[r]);
    m.lse[r] = lse_parts[r];
  }
  if (rows == 0) return GW_OK;
  m.n_parts = n_parts;
  m.rows = rows;
  m.heads = num_heads;
  m.head_dim = head_dim;
  m.out = static_cast<uint16_t*>(out);
  m.lse_out = lse_out;
  return cuda_status(launch_merge_lse(m, static_cast<cudaStream_t>(stream)), fn);
}

gw_status gw_set_max_ctas(int32_t max_ctas) {
  g_err[0] = 0;
  if (max_ctas < 0) return fail(GW_ERR_INVALID_ARG, "gw_set_max_ctas", "max_ctas (%d) < 0", max_ctas);
  g_max_ctas = max_ctas;
  return GW_OK;
}

gw_status gw_set_early_launch(int32_t on) {
  g_err[0] = 0;
  g_early_launch = on != 0;
  return GW_OK;
}

gw_status gw_set_early_inputs(int32_t on) {
  g_err[0] = 0;
  g_early_inputs = on != 0;
  return GW_OK;
}

gw_status gw_bw_probe(const void* buf, size_t bytes, int32_t* dev_status, void* stream) {
  const char* fn = "gw_bw_probe";
  g_err[0] = 0;
  if (!buf || !aligned(buf, 16)) return fail(GW_ERR_INVALID_ARG, fn, "buf NULL or not 16-byte aligned");
  if (bytes < 8192) return fail(GW_ERR_INVALID_ARG, fn, "bytes (%zu) < 8192", bytes);
  if (dev_status && !aligned(dev_status, 4)) return fail(GW_ERR_INVALID_ARG, fn, "dev_status misaligned");
  return cuda_status(launch_bw_probe(buf, static_cast<int64_t>(bytes / 8192), dev_status,
                                     static_cast<cudaStream_t>(stream)),
                     fn);
}

gw_status gw_bw_probe_tma(const void* buf, size_t bytes, int32_t* dev_status, void* stream) {
  const char* fn = "gw_bw_probe_tma";
  g_err[0] = 0;
  if (!buf || !aligned(buf, 256)) return fail(GW_ERR_INVALID_ARG, fn, "buf NULL or not 256-byte aligned");
  if (bytes < 16384) return fail(GW_ERR_INVALID_ARG, fn, "bytes (%zu) < 16384", bytes);
  if (bytes / 16384 > (static_cast<size_t>(1) << 22))  // tensor-map rows stay below 2^31
    return fail(GW_ERR_INVALID_ARG, fn, "bytes (%zu) above 2^36", bytes);
  if (dev_status && !aligned(dev_status, 4)) return fail(GW_ERR_INVALID_ARG, fn, "dev_status misaligned");
  return cuda_status(launch_bw_probe_tma(buf, static_cast<int64_t>(bytes / 16384), dev_status,
                                         static_cast<cudaStream_t>(stream)),
                     fn);
}

gw_status gw_wait_selftest(int32_t* dev_status, int32_t* result, int64_t limit_ns, void* stream) {
  const char* fn = "gw_wait_selftest";
  g_err[0] = 0;
  if (!dev_status || !aligned(dev_status, 4)) return fail(GW_ERR_INVALID_ARG, fn, "dev_status NULL or misaligned");
  if (!result || !aligned(result, 4)) return fail(GW_ERR_INVALID_ARG, fn, "result NULL or misaligned");
  if (limit_ns < 1000 || limit_ns > 1000000000)
    return fail(GW_ERR_INVALID_ARG, fn, "limit_ns (%lld) outside [1e3, 1e9]", static_cast<long long>(limit_ns));
  return cuda_status(launch_wait_selftest(dev_status, result, limit_ns, static_cast<cudaStream_t>(stream)), fn);
}

}  // extern "C"
