"""Python binding of the gw C ABI (include/gw.h) over ctypes.

Argument marshalling only: tensors are passed by ``data_ptr()`` and the
current CUDA stream; every step of the computation runs in libgw.so.  There
is no CPU path: if the library is missing this module raises ImportError.
"""

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgw.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libgw.so is not built (%s); run `python -c 'import __graft_entry__ as g; g.build()'`"
                      % LIB_PATH)
_lib = ctypes.CDLL(LIB_PATH)

# ---- constants (mirror include/gw.h) -----------------------------------------
GW_OK, GW_ERR_INVALID_ARG, GW_ERR_UNSUPPORTED, GW_ERR_WORKSPACE, GW_ERR_CUDA = 0, 1, 2, 3, 4
GW_DEV_SLOT_RANGE, GW_DEV_POS_RANGE, GW_DEV_PAGE_RANGE, GW_DEV_LEN_RANGE = 1, 2, 4, 8
GW_DEV_TIMEOUT, GW_DEV_WORKSPACE, GW_DEV_KEEP_RANGE = 16, 32, 64
KV_BF16, KV_E4M3 = 0, 1
LAYOUT_LOCAL, LAYOUT_GLOBAL_FOLDED, LAYOUT_GLOBAL_FULL, LAYOUT_GLOBAL_FOLDED_E4M3 = 0, 1, 2, 3
LAYOUTS = {"local": LAYOUT_LOCAL, "folded": LAYOUT_GLOBAL_FOLDED, "full": LAYOUT_GLOBAL_FULL,
           "folded_e4m3": LAYOUT_GLOBAL_FOLDED_E4M3}
DTYPES = {"bf16": KV_BF16, "e4m3": KV_E4M3}
EXPORTS = ["gw_pool_page_bytes", "gw_kv_append", "gw_decode_attn_local", "gw_decode_attn_global",
           "gw_attn_workspace_bytes", "gw_last_error", "gw_version", "gw_decode_attn_local_noalloc",
           "gw_noalloc_scratch_bytes", "gw_bw_probe", "gw_set_max_ctas", "gw_set_early_launch",
           "gw_set_early_inputs", "gw_rope_cs", "gw_wait_selftest", "gw_bw_probe_tma",
           "gw_decode_attn_global_lse", "gw_merge_lse", "gw_append_decode_attn_local",
           "gw_append_decode_attn_global", "gw_rope_rows", "gw_rope_cs_scaled",
           "gw_decode_attn_global_acc", "gw_attn_acc_workspace_bytes", "gw_kv_evict_select", "gw_kv_evict_compact"]


ELEMS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
PAIRS_HALF, PAIRS_INTERLEAVED = 0, 1
ROPE_KINDS = {"none": 0, "linear": 1, "ntk": 2, "ramp": 3}


class GwError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__("gw status %d: %s" % (code, msg))
        self.code = code


class PoolDesc(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("dtype", ctypes.c_int32), ("base", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32)]


class RopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("reserved", ctypes.c_int32), ("factor", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("orig_max_pos", ctypes.c_double),
                ("amplitude", ctypes.c_double)]


_vp, _i32, _i64, _f32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_P = ctypes.POINTER(PoolDesc)
_lib.gw_pool_page_bytes.argtypes = [_P]
_lib.gw_pool_page_bytes.restype = _sz
_lib.gw_kv_append.argtypes = [_P, _vp, _vp, _i32, _vp, _vp, _vp, _i32, _vp, _vp]
_lib.gw_kv_append.restype = _i32
_lib.gw_decode_attn_local.argtypes = [_P, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _f32, _vp, _sz,
                                      _vp, _vp]
_lib.gw_decode_attn_local.restype = _i32
_lib.gw_append_decode_attn_local.argtypes = [_P, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _i32, _i32,
                                             _f32, _vp, _sz, _vp, _vp]
_lib.gw_append_decode_attn_local.restype = _i32
_lib.gw_append_decode_attn_global.argtypes = [_P, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _i32,
                                              _f32, _vp, _sz, _vp, _vp]
_lib.gw_append_decode_attn_global.restype = _i32
_lib.gw_decode_attn_global.argtypes = [_P, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _i32, _i32, _f32, _vp, _sz,
                                       _vp, _vp]
_lib.gw_decode_attn_global.restype = _i32
_lib.gw_decode_attn_global_lse.argtypes = [_P, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _i32, _f32, _vp, _sz,
                                           _vp, _vp]
_lib.gw_decode_attn_global_lse.restype = _i32
_lib.gw_decode_attn_global_acc.argtypes = [_P, _vp, _vp, _vp, _vp, _i64, _f32, _i32, _i32, _vp, _vp, _vp, _i32, _f32,
                                           _vp, _sz, _vp, _vp]
_lib.gw_decode_attn_global_acc.restype = _i32
_lib.gw_attn_acc_workspace_bytes.argtypes = [_P, _i32, _i32, _i32]
_lib.gw_attn_acc_workspace_bytes.restype = _sz
_lib.gw_kv_evict_select.argtypes = [_vp, _i64, _i32, _vp, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _vp]
_lib.gw_kv_evict_select.restype = _i32
_lib.gw_kv_evict_compact.argtypes = [_P, _i32, _vp, _i32, _vp, _vp, _i64, _vp, _vp, _i32, _vp, _i64, _vp, _vp]
_lib.gw_kv_evict_compact.restype = _i32
_lib.gw_merge_lse.argtypes = [_i32, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp]
_lib.gw_merge_lse.restype = _i32
_lib.gw_rope_cs.argtypes = [_vp, ctypes.c_double, _i32, _i32, _i32, _vp]
_lib.gw_rope_cs.restype = _i32
_lib.gw_rope_rows.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp,
                              _i32, _vp, _vp]
_lib.gw_rope_rows.restype = _i32
_lib.gw_rope_cs_scaled.argtypes = [_vp, ctypes.c_double, _i32, _i32, _i32, ctypes.POINTER(RopeScaling), _vp]
_lib.gw_rope_cs_scaled.restype = _i32
_lib.gw_attn_workspace_bytes.argtypes = [_P, _i32, _i32, _i32, _i32, _i32]
_lib.gw_attn_workspace_bytes.restype = _sz
_lib.gw_decode_attn_local_noalloc.argtypes = [_P, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _f32,
                                              _vp, _vp]
_lib.gw_decode_attn_local_noalloc.restype = _i32
_lib.gw_noalloc_scratch_bytes.argtypes = []
_lib.gw_noalloc_scratch_bytes.restype = _sz
_lib.gw_bw_probe.argtypes = [_vp, _sz, _vp, _vp]
_lib.gw_bw_probe.restype = _i32
_lib.gw_bw_probe_tma.argtypes = [_vp, _sz, _vp, _vp]
_lib.gw_bw_probe_tma.restype = _i32
_lib.gw_wait_selftest.argtypes = [_vp, _vp, _i64, _vp]
_lib.gw_wait_selftest.restype = _i32
_lib.gw_set_max_ctas.argtypes = [_i32]
_lib.gw_set_max_ctas.restype = _i32
_lib.gw_set_early_launch.argtypes = [_i32]
_lib.gw_set_early_launch.restype = _i32
_lib.gw_set_early_inputs.argtypes = [_i32]
_lib.gw_set_early_inputs.restype = _i32
_lib.gw_last_error.argtypes = []
_lib.gw_last_error.restype = ctypes.c_char_p
_lib.gw_version.argtypes = []
_lib.gw_version.restype = _i32


def lib():
    return _lib


def last_error():
    return _lib.gw_last_error().decode()


def version():
    return _lib.gw_version()


def _check(code):
    if code != GW_OK:
        raise GwError(code, last_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _invalid(fn, what):
    raise GwError(GW_ERR_INVALID_ARG, "%s: %s" % (fn, what))


def _missing(fn, **tensors):
    """Refuses the first of these that is None, by its name."""
    for name, t in tensors.items():
        if t is None:
            _invalid(fn, "%s is None" % name)


def _on_device(fn, stream, *tensors):
    """Every tensor (None: left out, but not the first) on one CUDA device,
    which the stream (the current one if None) belongs to and which is the
    current device, since the library launches there.  Returns the stream's
    handle."""
    dev = tensors[0].get_device()  # -1 on the CPU
    for t in tensors:
        if t is not None and t.get_device() != dev:
            _invalid(fn, "tensors on %s and %s" % (tensors[0].device, t.device))
    if dev < 0:
        _invalid(fn, "tensors on %s, not on a CUDA device" % tensors[0].device)
    if dev != torch.cuda.current_device() or (stream is not None and stream.device.index != dev):
        _invalid(fn, "tensors on %s, but the current device or the stream is another" % tensors[0].device)
    # the raw handle costs 0.1 us, a torch.cuda.Stream object 2.9 us
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """A new tensor for a call on this stream (None: the current one), out of
    that stream's memory: a block of another stream's may still be read there
    by work that came before."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _addr(t):
    return None if t is None else t.data_ptr()


def _dense(fn, name, t, dtype, *shape):
    """`t` has this dtype and shape (None: any length) and is contiguous."""
    want = tuple(m if n is None else n for n, m in zip(shape, t.shape)) if None in shape else shape
    if t.dtype != dtype or t.shape != want or len(want) != len(shape):
        _invalid(fn, "%s must be %s of shape %s (got %s %s)" % (name, dtype, list(shape), t.dtype, list(t.shape)))
    if not t.is_contiguous():
        _invalid(fn, "%s must be contiguous" % name)


def _vector(fn, name, t, n):
    """`t` is int32 [n], contiguous."""
    if t.dtype != torch.int32 or t.shape != (n,) or not t.is_contiguous():
        _dense(fn, name, t, torch.int32, n)


def _row_stride(fn, name, t, dtype, rows):
    """The row stride of `t`, [rows, columns] of this dtype whose columns are
    adjacent and whose rows do not overlap; each row, the last one too, has
    the stride's length of memory behind it."""
    if t.dtype != dtype or t.dim() != 2 or t.shape[0] != rows:
        _invalid(fn, "%s must be %s [%d, columns] (got %s %s)" % (name, dtype, rows, t.dtype, list(t.shape)))
    cols = int(t.shape[1])
    if (cols > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < cols):
        _invalid(fn, "%s must have adjacent columns and rows that do not overlap" % name)
    stride = int(t.stride(0)) if rows > 1 else cols
    if stride > cols and t.storage_offset() + rows * stride > t.untyped_storage().nbytes() // t.element_size():
        _invalid(fn, "%s: the last row ends before its stride" % name)
    return stride


# ---- pools ---------------------------------------------------------------------
class KVPool:
    """A paged pool held in a torch uint8 device buffer plus its ABI descriptor."""

    def __init__(self, layout, dtype, num_pages, kv_heads=1, device="cuda", storage=None):
        self.layout, self.dtype = layout, dtype
        self.kv_heads = kv_heads if layout == "local" else 1
        head_dim, rot_dim = (256, 256) if layout == "local" else (512, 128)
        self.desc = PoolDesc(LAYOUTS[layout], DTYPES[dtype], None, num_pages, 16, self.kv_heads, head_dim, rot_dim)
        pb = _lib.gw_pool_page_bytes(ctypes.byref(self.desc))
        if pb == 0:
            raise GwError(GW_ERR_INVALID_ARG, last_error())
        self.page_bytes = pb
        self.num_pages = num_pages
        if storage is None:
            storage = torch.zeros(num_pages * pb + 256, dtype=torch.uint8, device=device)
        self._storage = storage
        off = (-storage.data_ptr()) % 256
        self.data = storage[off:off + num_pages * pb]
        self.desc.base = self.data.data_ptr()

    @property
    def nbytes(self):
        return self.num_pages * self.page_bytes


def rope_cs(theta, rot_dim, head_dim, max_pos, out=None, device="cuda", stream=None):
    """gw_rope_cs: the float32 [max_pos, rot_dim/2, 2] (cos, sin) table of
    gw_kv_append, computed by the library on the GPU (into `out` if given)."""
    if out is None:
        out = _empty((max_pos, rot_dim // 2, 2), torch.float32, device, stream)
    _check(_lib.gw_rope_cs(_ptr(out), float(theta), int(rot_dim), int(head_dim), int(max_pos), _stream(stream)))
    return out


def rope_cs_scaled(theta, rot_dim, head_dim, max_pos, kind="none", factor=1.0, low=1.0, high=32.0, orig_max_pos=0,
                   amplitude=1.0, out=None, device="cuda", stream=None):
    """gw_rope_cs_scaled: rope_cs for a context longer than the trained one, by
    `kind` "none", "linear", "ntk" or "ramp" (include/gw.h states each)."""
    fn = "gw_rope_cs_scaled"
    if kind not in ROPE_KINDS:
        _invalid(fn, "unknown kind %r" % (kind,))
    if out is None:
        out = _empty((max_pos, rot_dim // 2, 2), torch.float32, device, stream)
    handle = _on_device(fn, stream, out)
    _dense(fn, "out", out, torch.float32, max_pos, rot_dim // 2, 2)
    sc = RopeScaling(ROPE_KINDS[kind], 0, factor, low, high, orig_max_pos, amplitude)
    _check(_lib.gw_rope_cs_scaled(out.data_ptr(), float(theta), int(rot_dim), int(head_dim), int(max_pos),
                                  ctypes.byref(sc), handle))
    return out


def rope_rows(x, pos, rope_cs, out=None, rot_dim=None, interleaved=False, inverse=False, dev_status=None,
              stream=None):
    """gw_rope_rows: the rows x [rows, heads, head_dim] (bf16, fp16 or fp32;
    any strides, the last one 1) rotated by pos int32 [rows] into `out` (x
    itself: in place; a new contiguous tensor if None), which is returned."""
    fn = "gw_rope_rows"
    if x is None or pos is None or rope_cs is None:  # a call of _missing costs as much as all checks below
        _missing(fn, x=x, pos=pos, rope_cs=rope_cs)
    if out is None:
        out = _empty(x.shape, x.dtype, x.device, stream)
    handle = _on_device(fn, stream, x, out, pos, rope_cs, dev_status)
    elem = ELEMS.get(x.dtype)
    if x.dim() != 3 or elem is None or out.dtype != x.dtype or out.shape != x.shape:
        _invalid(fn, "x and out must be [rows, heads, head_dim] of one of bf16, fp16, fp32 (got %s %s and %s %s)" %
                 (x.dtype, list(x.shape), out.dtype, list(out.shape)))
    rows, heads, dim = x.shape
    rot_dim = dim if rot_dim is None else int(rot_dim)
    xr, xh, x1 = x.stride()
    yr, yh, y1 = out.stride()
    if dim > 1 and (x1 != 1 or y1 != 1):
        _invalid(fn, "the last dimension of x and out must have stride 1")
    _vector(fn, "pos", pos, rows)
    max_pos = rope_cs.shape[0]
    _dense(fn, "rope_cs", rope_cs, torch.float32, max_pos, rot_dim // 2, 2)
    _check(_lib.gw_rope_rows(x.data_ptr(), xr, xh, out.data_ptr(), yr, yh, elem, rows, heads, dim, rot_dim,
                             PAIRS_INTERLEAVED if interleaved else PAIRS_HALF, 1 if inverse else 0, pos.data_ptr(),
                             rope_cs.data_ptr(), max_pos, _addr(dev_status), handle))
    return out


# ---- entry points ------------------------------------------------------------------
def kv_append(pool, k, v, slot, pos, rope_cs, dev_status=None, stream=None):
    """gw_kv_append: k, v bf16 CUDA tensors, slot/pos int32, rope_cs float32 [max_pos, R/2, 2]."""
    n = int(slot.numel())
    _check(_lib.gw_kv_append(ctypes.byref(pool.desc), _ptr(k), _ptr(v), n, _ptr(slot), _ptr(pos), _ptr(rope_cs),
                             int(rope_cs.shape[0]), _ptr(dev_status), _stream(stream)))


def workspace_bytes(pool, num_q_heads, batch, max_pages_per_seq, max_q_rows=1, window=1024):
    w = _lib.gw_attn_workspace_bytes(ctypes.byref(pool.desc), num_q_heads, batch, max_pages_per_seq * 16,
                                     max_q_rows, window)
    if w == 0 and batch > 0:
        raise GwError(GW_ERR_INVALID_ARG, last_error() or "invalid workspace request")
    return w


def alloc_workspace(pool, num_q_heads, batch, max_pages_per_seq, max_q_rows=1, window=1024, device="cuda"):
    n = workspace_bytes(pool, num_q_heads, batch, max_pages_per_seq, max_q_rows, window)
    buf = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    return buf[off:off + n]


def decode_attn_local(pool, q, out, cu_q_rows, seq_lens, block_table, workspace, window, scale=None,
                      max_q_rows=1, dev_status=None, stream=None):
    hq = int(q.shape[1])
    scale = 1.0 / math.sqrt(256) if scale is None else scale
    _check(_lib.gw_decode_attn_local(ctypes.byref(pool.desc), _ptr(q), _ptr(out), hq, int(seq_lens.numel()),
                                     _ptr(cu_q_rows), _ptr(seq_lens), _ptr(block_table), int(block_table.shape[1]),
                                     int(max_q_rows), int(window), float(scale), _ptr(workspace),
                                     int(workspace.numel()), _ptr(dev_status), _stream(stream)))


def append_decode_attn_local(pool, k, v, rope_cs, q, out, cu_q_rows, seq_lens, block_table, workspace, window,
                             scale=None, dev_status=None, stream=None):
    """gw_append_decode_attn_local: gw_kv_append of each decode row's k, v at
    position seq_len - 1, then its attention, in one call."""
    hq = int(q.shape[1])
    scale = 1.0 / math.sqrt(256) if scale is None else scale
    _check(_lib.gw_append_decode_attn_local(ctypes.byref(pool.desc), _ptr(k), _ptr(v), _ptr(rope_cs),
                                            int(rope_cs.shape[0]), _ptr(q), _ptr(out), hq, int(seq_lens.numel()),
                                            _ptr(cu_q_rows), _ptr(seq_lens), _ptr(block_table),
                                            int(block_table.shape[1]), int(window), float(scale), _ptr(workspace),
                                            int(workspace.numel()), _ptr(dev_status), _stream(stream)))


def append_decode_attn_global(pool, k, v, rope_cs, q, out, cu_q_rows, seq_lens, block_table, workspace, scale=None,
                              dev_status=None, stream=None):
    """gw_append_decode_attn_global: gw_kv_append of each decode row's k, v
    ([rows, 512]) at position seq_len - 1, then its attention, in one call."""
    hq = int(q.shape[1])
    scale = 1.0 / math.sqrt(512) if scale is None else scale
    _check(_lib.gw_append_decode_attn_global(ctypes.byref(pool.desc), _ptr(k), _ptr(v), _ptr(rope_cs),
                                             int(rope_cs.shape[0]), _ptr(q), _ptr(out), hq, int(seq_lens.numel()),
                                             _ptr(cu_q_rows), _ptr(seq_lens), _ptr(block_table),
                                             int(block_table.shape[1]), float(scale), _ptr(workspace),
                                             int(workspace.numel()), _ptr(dev_status), _stream(stream)))


def decode_attn_global(pool, q, out, cu_q_rows, seq_lens, block_table, workspace, scale=None, max_q_rows=1,
                       dev_status=None, stream=None):
    hq = int(q.shape[1])
    scale = 1.0 / math.sqrt(512) if scale is None else scale
    _check(_lib.gw_decode_attn_global(ctypes.byref(pool.desc), _ptr(q), _ptr(out), hq, int(seq_lens.numel()),
                                      _ptr(cu_q_rows), _ptr(seq_lens), _ptr(block_table), int(block_table.shape[1]),
                                      int(max_q_rows), float(scale), _ptr(workspace), int(workspace.numel()),
                                      _ptr(dev_status), _stream(stream)))


def decode_attn_global_lse(pool, q, out, lse, cu_q_rows, seq_lens, block_table, workspace, scale=None,
                           dev_status=None, stream=None):
    """gw_decode_attn_global_lse: decode rows, plus each row's log-sum-exp (float32 [rows, heads])."""
    hq = int(q.shape[1])
    scale = 1.0 / math.sqrt(512) if scale is None else scale
    _check(_lib.gw_decode_attn_global_lse(ctypes.byref(pool.desc), _ptr(q), _ptr(out), _ptr(lse), hq,
                                          int(seq_lens.numel()), _ptr(cu_q_rows), _ptr(seq_lens), _ptr(block_table),
                                          int(block_table.shape[1]), float(scale), _ptr(workspace),
                                          int(workspace.numel()), _ptr(dev_status), _stream(stream)))


def alloc_workspace_acc(pool, num_q_heads, batch, max_pages_per_seq, device="cuda"):
    """The workspace of decode_attn_global_acc calls of at most this size."""
    n = _lib.gw_attn_acc_workspace_bytes(ctypes.byref(pool.desc), num_q_heads, batch, max_pages_per_seq)
    if n == 0:
        raise GwError(GW_ERR_INVALID_ARG, last_error() or "invalid workspace request")
    buf = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    return buf[off:off + n]


def decode_attn_global_acc(pool, q, out, lse, acc, cu_q_rows, seq_lens, block_table, workspace, decay=1.0, scale=None,
                           dev_status=None, stream=None):
    """gw_decode_attn_global_acc: decode rows, each row's log-sum-exp (lse
    float32 [rows, heads] or None), and acc [batch, stride] = decay * acc +
    each cached token's softmax weights summed over the heads."""
    fn = "gw_decode_attn_global_acc"
    if (q is None or out is None or acc is None or cu_q_rows is None or seq_lens is None or block_table is None or
            workspace is None):
        _missing(fn, q=q, out=out, acc=acc, cu_q_rows=cu_q_rows, seq_lens=seq_lens, block_table=block_table,
                 workspace=workspace)
    handle = _on_device(fn, stream, pool.data, q, out, lse, acc, cu_q_rows, seq_lens, block_table, workspace,
                        dev_status)
    batch = seq_lens.numel()
    if q.dim() != 3:
        _invalid(fn, "q must be [rows, heads, 512] (got %s)" % list(q.shape))
    rows, hq = q.shape[0], q.shape[1]
    _dense(fn, "q", q, torch.bfloat16, rows, hq, 512)
    _dense(fn, "out", out, torch.bfloat16, rows, hq, 512)
    if lse is not None:
        _dense(fn, "lse", lse, torch.float32, rows, hq)
    stride = _row_stride(fn, "acc", acc, torch.float32, batch)
    _vector(fn, "cu_q_rows", cu_q_rows, batch + 1)
    _vector(fn, "seq_lens", seq_lens, batch)
    _dense(fn, "block_table", block_table, torch.int32, batch, None)
    pages = block_table.shape[1]
    if acc.shape[1] < 16 * pages:
        _invalid(fn, "acc has %d columns, the block table names %d tokens" % (acc.shape[1], 16 * pages))
    if not workspace.is_contiguous():
        _invalid(fn, "workspace must be contiguous")
    scale = 1.0 / math.sqrt(512) if scale is None else scale
    _check(_lib.gw_decode_attn_global_acc(pool.desc, q.data_ptr(), out.data_ptr(), _addr(lse), acc.data_ptr(), stride,
                                          float(decay), hq, batch, cu_q_rows.data_ptr(), seq_lens.data_ptr(),
                                          block_table.data_ptr(), pages, float(scale), workspace.data_ptr(),
                                          workspace.numel() * workspace.element_size(), _addr(dev_status), handle))


def kv_evict_select(acc, seq_lens, budget, keep_idx, keep_lens, sinks=0, recent=0, dev_status=None, stream=None):
    """gw_kv_evict_select: the indices of the `budget` tokens that each
    sequence keeps (the first `sinks`, the last `recent`, the largest acc
    between), ascending, into keep_idx int32 [batch, >= budget], and their
    number into keep_lens int32 [batch]."""
    fn = "gw_kv_evict_select"
    if acc is None or seq_lens is None or keep_idx is None or keep_lens is None:
        _missing(fn, acc=acc, seq_lens=seq_lens, keep_idx=keep_idx, keep_lens=keep_lens)
    handle = _on_device(fn, stream, acc, seq_lens, keep_idx, keep_lens, dev_status)
    batch = seq_lens.numel()
    _vector(fn, "seq_lens", seq_lens, batch)
    _vector(fn, "keep_lens", keep_lens, batch)
    acc_stride = _row_stride(fn, "acc", acc, torch.float32, batch)
    keep_stride = _row_stride(fn, "keep_idx", keep_idx, torch.int32, batch)
    if keep_idx.shape[1] < budget:
        _invalid(fn, "keep_idx has %d columns, the budget is %d" % (keep_idx.shape[1], budget))
    _check(_lib.gw_kv_evict_select(acc.data_ptr(), acc_stride, batch, seq_lens.data_ptr(), int(budget), int(sinks),
                                   int(recent), keep_idx.data_ptr(), keep_stride, keep_lens.data_ptr(), _addr(dev_status), handle))


def kv_evict_compact(pool, block_table, seq_lens, keep_idx, keep_lens, acc=None, dst_block_table=None,
                     dev_status=None, stream=None):
    """gw_kv_evict_compact: each sequence's kept rows moved to its front, in
    its own pages or into those of dst_block_table; acc moves along in place."""
    fn = "gw_kv_evict_compact"
    if block_table is None or seq_lens is None or keep_idx is None or keep_lens is None:
        _missing(fn, block_table=block_table, seq_lens=seq_lens, keep_idx=keep_idx, keep_lens=keep_lens)
    handle = _on_device(fn, stream, pool.data, block_table, seq_lens, keep_idx, keep_lens, acc, dst_block_table,
                        dev_status)
    batch = seq_lens.numel()
    _vector(fn, "seq_lens", seq_lens, batch)
    _vector(fn, "keep_lens", keep_lens, batch)
    _dense(fn, "block_table", block_table, torch.int32, batch, None)
    pages = block_table.shape[1]
    keep_stride = _row_stride(fn, "keep_idx", keep_idx, torch.int32, batch)
    acc_stride, dst_pages = 0, 0
    if acc is not None:
        acc_stride = _row_stride(fn, "acc", acc, torch.float32, batch)
        if acc.shape[1] < 16 * pages:
            _invalid(fn, "acc has %d columns, the block table names %d tokens" % (acc.shape[1], 16 * pages))
    if dst_block_table is not None:
        _dense(fn, "dst_block_table", dst_block_table, torch.int32, batch, None)
        dst_pages = dst_block_table.shape[1]
    _check(_lib.gw_kv_evict_compact(pool.desc, batch, block_table.data_ptr(), pages, seq_lens.data_ptr(),
                                    keep_idx.data_ptr(), keep_stride, keep_lens.data_ptr(), _addr(dst_block_table),
                                    dst_pages, _addr(acc), acc_stride, _addr(dev_status), handle))


def merge_lse(outs, lses, out, lse_out=None, stream=None):
    """gw_merge_lse: merge the parts (bf16 [rows, heads, D] outputs and their
    float32 [rows, heads] log-sum-exps) into `out`."""
    n = len(outs)
    o_arr = (ctypes.c_void_p * n)(*[o.data_ptr() for o in outs])
    l_arr = (ctypes.c_void_p * n)(*[l.data_ptr() for l in lses])
    rows, heads, dim = (int(x) for x in out.shape)
    _check(_lib.gw_merge_lse(n, o_arr, l_arr, _ptr(out), _ptr(lse_out), rows, heads, dim, _stream(stream)))


def decode_attn_local_noalloc(pool, q, out, cu_q_rows, seq_lens, block_table, window, scale=None, max_q_rows=1,
                              dev_status=None, stream=None):
    """gw_decode_attn_local_noalloc: same as decode_attn_local, scratch from the library's static array."""
    hq = int(q.shape[1])
    scale = 1.0 / math.sqrt(256) if scale is None else scale
    _check(_lib.gw_decode_attn_local_noalloc(ctypes.byref(pool.desc), _ptr(q), _ptr(out), hq,
                                             int(seq_lens.numel()), _ptr(cu_q_rows), _ptr(seq_lens),
                                             _ptr(block_table), int(block_table.shape[1]), int(max_q_rows),
                                             int(window), float(scale), _ptr(dev_status), _stream(stream)))


def set_max_ctas(max_ctas):
    """gw_set_max_ctas: cap the CTAs (= SMs) of this thread's later attention
    calls; 0 restores one per SM."""
    _check(_lib.gw_set_max_ctas(int(max_ctas)))


def set_early_launch(on):
    """gw_set_early_launch: allow (True) or forbid programmatic early launch
    for this thread's later calls."""
    _check(_lib.gw_set_early_launch(1 if on else 0))


def set_early_inputs(on):
    """gw_set_early_inputs: let this thread's later decode calls read cu_q_rows,
    seq_lens and block_table, and its appends slot, pos and rope_cs, before
    the previous kernel of their stream ends (the caller guarantees that
    kernel does not write them)."""
    _check(_lib.gw_set_early_inputs(1 if on else 0))


def bw_probe(buf, dev_status=None, stream=None):
    """gw_bw_probe: stream `buf` (a CUDA tensor) through the decode kernels' copy pipeline."""
    _check(_lib.gw_bw_probe(_ptr(buf), int(buf.numel() * buf.element_size()), _ptr(dev_status), _stream(stream)))


def bw_probe_tma(buf, dev_status=None, stream=None):
    """gw_bw_probe_tma: stream `buf` through the bf16 decode kernel's tensor-map copy pipeline."""
    _check(_lib.gw_bw_probe_tma(_ptr(buf), int(buf.numel() * buf.element_size()), _ptr(dev_status),
                                _stream(stream)))


def wait_selftest(dev_status, result, limit_ns, stream=None):
    """gw_wait_selftest: run the kernels' bounded wait on a phase nothing
    completes, with a limit of limit_ns; result (int32[3] on the device)
    receives {first wait ok, second wait gave up, microseconds waited}."""
    _check(_lib.gw_wait_selftest(_ptr(dev_status), _ptr(result), int(limit_ns), _stream(stream)))
