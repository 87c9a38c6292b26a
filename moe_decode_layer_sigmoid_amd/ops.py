"""ctypes binding of the operators beside the MoE layer (include/moe_decode_ops.h):
the activation quantiser, the block-scaled fp8 product and the 8-bit paged
cache's append, attention and eviction.

The functions keep the C names.  Tensors are torch tensors on the plan's
device (the quantiser: on one device, which need not be the current one);
their types, shapes and strides are checked here, the rest in the library.
The stream is the tensors' device's current torch stream unless one is given.
A tensor that was made on another stream is the caller's to order and to keep.
"""

from __future__ import annotations

import ctypes
import struct

from .binding import ERR_INVALID_ARG, MoeDecodeError, SCALE_E8M0, SCALE_FP32, lib

OUT_BF16, OUT_FP32 = 0, 1  # moe_decode_out_fmt
PAGE_TOKENS = 64  # MOE_DECODE_PAGE_TOKENS

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class ProductDesc(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("n", "k", "max_rows", "scale_fmt", "out_fmt")]


class ProductArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("codes", "scales", "w", "w_scale", "out")] + [
        ("out_stride", _i64)]


class CacheDesc(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("heads", "kv_heads", "head_dim", "pages", "max_batch",
                                    "max_pages", "max_q", "with_mass")]


class Cache(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("pool", "pool_scale", "page_table", "seq_lens", "q_start")]


class AppendArgs(ctypes.Structure):
    _fields_ = [("cache", Cache), ("k", _vp), ("v", _vp), ("k_stride", _i64), ("v_stride", _i64)]


class AttendArgs(ctypes.Structure):
    _fields_ = [("cache", Cache), ("q", _vp), ("q_stride", _i64), ("out", _vp),
                ("out_stride", _i64), ("sm_scale", ctypes.c_float), ("mass_in", _vp),
                ("mass_out", _vp)]


class EvictArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("page_table", "seq_lens", "mass", "out_table", "out_lens",
                                   "out_mass", "freed", "n_freed")] + [
        (n, _i32) for n in ("keep", "sink", "recent")]


# The argument structs as one call makes them: packing costs a quarter of
# filling a ctypes.Structure.
_pack_product = struct.Struct("5Qq").pack
_pack_append = struct.Struct("5Q2Q2q").pack
_pack_attend = struct.Struct("5QQqQqf4x2Q").pack
_pack_evict = struct.Struct("8Q3i4x").pack


def declare(L) -> None:
    """The prototypes of include/moe_decode_ops.h on the loaded library."""
    P = ctypes.POINTER
    protos = {
        "quant": [_vp, _i64, _i32, _i32, ctypes.c_float, _vp, _vp, _vp],
        "product_desc_check": [P(ProductDesc)],
        "product_args_check": [P(ProductDesc), P(ProductArgs), _i32],
        "product_plan": [P(ProductDesc), ctypes.c_int, P(_vp)],
                "product_destroy": [_vp],
        "cache_desc_check": [P(CacheDesc)],
        "append_check": [P(CacheDesc), P(AppendArgs), _i32, _i32],
        "attend_check": [P(CacheDesc), P(AttendArgs), _i32, _i32],
        "evict_check": [P(CacheDesc), P(EvictArgs), _i32],
        "cache_plan": [P(CacheDesc), ctypes.c_int, P(_vp)],
        "cache_destroy": [_vp],
        # the arguments as a pointer or as packed bytes
        "product_run": [_vp, _vp, _i32, _vp],
        "cache_append": [_vp, _vp, _i32, _i32, _vp],
        "cache_attend": [_vp, _vp, _i32, _i32, _vp],
        "cache_evict": [_vp, _vp, _i32, _vp],
    }
    for name, args in protos.items():
        f = getattr(L, "moe_decode_" + name)
        f.argtypes, f.restype = args, ctypes.c_int
    for name in ("product_workspace_bytes", "cache_workspace_bytes"):
        f = getattr(L, "moe_decode_" + name)
        f.argtypes, f.restype = [_vp], ctypes.c_size_t


def _need(ok: bool, what: str, why: str, *args) -> None:
    if not ok:
        raise MoeDecodeError(ERR_INVALID_ARG, "%s: %s" % (what, why % args))


def _tensor(what, name, t, dtypes, shape, device) -> int:
    """The address of a contiguous tensor of one of `dtypes` and `shape` on
    CUDA device `device`."""
    if t.dtype in dtypes and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    raise MoeDecodeError(ERR_INVALID_ARG, "%s: %s must be a contiguous %s tensor %s on device "
                         "%d, got %s %s strides %s on %s"
                         % (what, name, "/".join(str(d) for d in dtypes), list(shape), device,
                            t.dtype, list(t.shape), list(t.stride()), t.device))


def _rows(what, name, t, dtypes, shape, device) -> int:
    """As _tensor for at least shape[0] rows."""
    if t.dtype in dtypes and t.get_device() == device and t.is_contiguous():
        s = t.shape
        if s == shape or (len(s) == len(shape) and s[0] > shape[0] and s[1:] == shape[1:]):
            return t.data_ptr()
    return _tensor(what, name, t, dtypes, shape, device)


# torch and the types of the operators' tensors, set at the first use: the
# package itself loads without torch.
torch = None
_raw_stream = None  # device -> its current stream's handle
_CODES = _BYTES = _BF16 = _I32 = _F32 = ()


def _load_torch() -> None:
    global torch, _raw_stream, _CODES, _BYTES, _BF16, _I32, _F32
    if torch is None:
        import torch as t

        _CODES, _BYTES = (t.uint8, t.float8_e4m3fn), (t.uint8,)
        _BF16 = (t.bfloat16, t.int16)  # int16: bf16 bit patterns
        _I32, _F32 = (t.int32,), (t.float32,)
        # without the Stream object that torch.cuda.current_stream makes (1 us)
        _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream",
                              lambda d: t.cuda.current_stream(d).cuda_stream)
        torch = t


def _heads(what, name, t, T, heads, D, device):
    """(address, token stride) of a [>= T, heads, D] bf16 tensor whose tokens
    may be strided."""
    if t.dim() == 3 and t.dtype in _BF16 and t.get_device() == device:
        n, h, d = t.shape
        s0, s1, s2 = t.stride()
        if n >= T and h == heads and d == D and s2 == 1 and (s1 == D or heads == 1):
            # one token: its stride means nothing
            return t.data_ptr(), s0 if n > 1 else heads * D
    raise MoeDecodeError(ERR_INVALID_ARG, "%s: %s must be a bf16 tensor [%d, %d, %d] on device "
                         "%d with contiguous tokens, got %s %s strides %s on %s"
                         % (what, name, T, heads, D, device, t.dtype, list(t.shape),
                            list(t.stride()), t.device))


def _stream_of(stream, device: int) -> int:
    if stream is None:
        return _raw_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _done(rc: int, what: str) -> None:
    if rc:
        raise MoeDecodeError(rc, what)


def quant(x, codes, scales, limit=None, stream=None) -> None:
    """moe_decode_quant: codes [M, K] and scale bytes [M, K/128] of x [M, K]
    bf16 (rows may be strided), or with `limit` of the clamped SwiGLU of
    x [M, 2K]."""
    what = "moe_decode_quant"
    _load_torch()
    device = codes.get_device()
    _need(device >= 0, what, "tensors must be on a GPU")
    _need(codes.dim() == 2, what, "codes must be a matrix")
    _need(limit is None or limit > 0, what, "limit must be positive")
    M, K = codes.shape
    cols = K if limit is None else 2 * K
    if not (x.dtype in _BF16 and x.shape == (M, cols) and x.get_device() == device
            and x.stride(1) == 1):
        _need(False, what, "x must be a bf16 tensor [%d, %d] on the device of codes with "
              "contiguous rows", M, cols)
    pc = _tensor(what, "codes", codes, _CODES, (M, K), device)
    ps = _tensor(what, "scales", scales, _BYTES, (M, K // 128), device)
    if M == 0:
        return
    args = (x.data_ptr(), x.stride(0) if M > 1 else cols, M, K, limit or 0.0, pc, ps,
            _stream_of(stream, device))
    if device == torch.cuda.current_device():
        rc = lib().moe_decode_quant(*args)
    else:
        with torch.cuda.device(device):
            rc = lib().moe_decode_quant(*args)
    if rc:
        _done(rc, what)


def make_product_desc(N, K, max_rows, scale_fmt="fp32", out_fmt="bf16") -> ProductDesc:
    fmt = {"fp32": SCALE_FP32, "e8m0": SCALE_E8M0}.get(scale_fmt, scale_fmt)
    return ProductDesc(N, K, max_rows, fmt, {"bf16": OUT_BF16, "fp32": OUT_FP32}.get(out_fmt, out_fmt))


def product_desc_check(d: ProductDesc) -> int:
    return lib().moe_decode_product_desc_check(ctypes.byref(d))


def product_args_check(d: ProductDesc, a: ProductArgs, M: int) -> int:
    return lib().moe_decode_product_args_check(ctypes.byref(d), ctypes.byref(a), M)


class _PlanBase:
    _kind = ""

    def __init__(self, desc, device: int = 0):
        _load_torch()
        self.desc = desc
        self.device = device
        self._lib = lib()
        self._h = ctypes.c_void_p()
        what = "moe_decode_%s_plan" % self._kind
        _done(getattr(self._lib, what)(ctypes.byref(desc), device, ctypes.byref(self._h)), what)

    def close(self):
        if self._h:
            getattr(lib(), "moe_decode_%s_destroy" % self._kind)(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def workspace_bytes(self) -> int:
        return getattr(lib(), "moe_decode_%s_workspace_bytes" % self._kind)(self._h)


class ProductPlan(_PlanBase):
    """moe_decode_product_plan / _run / _destroy."""

    _kind = "product"

    def __init__(self, desc, device: int = 0):
        super().__init__(desc, device)
        d = self.desc
        self._N, self._K, self._M = d.n, d.k, d.max_rows
        self._scale = ((d.n + 127) // 128, d.k // 128)
        self._scale_types = _F32 if d.scale_fmt == SCALE_FP32 else _BYTES
        self._out_types = _F32 if d.out_fmt == OUT_FP32 else _BF16

    def run(self, M: int, *, codes, scales, w, w_scale, out, stream=None) -> None:
        """out [M, n] = (scales codes) (w_scale w)^T for the first M rows of
        codes, scales and out (whose rows may be strided)."""
        what, dev, N, K = "moe_decode_product_run", self.device, self._N, self._K
        if not 0 <= M <= self._M:
            _need(False, what, "M must be in [0, %d]", self._M)
        rows, cols = out.shape if out.dim() == 2 else (-1, -1)
        if not (rows >= M and cols == N and out.dtype in self._out_types
                and out.get_device() == dev and (out.stride(1) == 1 or N == 1)):
            _need(False, what, "out must be a %s tensor [%d, %d] on device %d with contiguous "
                  "rows", self._out_types[0], M, N, dev)
        a = _pack_product(_rows(what, "codes", codes, _CODES, (M, K), dev),
                          _rows(what, "scales", scales, _BYTES, (M, K // 128), dev),
                          _tensor(what, "w", w, _CODES, (N, K), dev),
                          _tensor(what, "w_scale", w_scale, self._scale_types, self._scale, dev),
                          out.data_ptr(), out.stride(0) if rows > 1 else N)
        if M == 0:
            return
        rc = self._lib.moe_decode_product_run(self._h, a, M, _stream_of(stream, dev))
        if rc:
            _done(rc, what)


def make_cache_desc(heads, kv_heads, head_dim, pages, max_batch, max_pages, max_q=1,
                    with_mass=True) -> CacheDesc:
    return CacheDesc(heads, kv_heads, head_dim, pages, max_batch, max_pages, max_q,
                     int(with_mass))


def cache_desc_check(d: CacheDesc) -> int:
    return lib().moe_decode_cache_desc_check(ctypes.byref(d))


def append_check(d: CacheDesc, a: AppendArgs, B: int, T: int) -> int:
    return lib().moe_decode_append_check(ctypes.byref(d), ctypes.byref(a), B, T)


def attend_check(d: CacheDesc, a: AttendArgs, B: int, T: int) -> int:
    return lib().moe_decode_attend_check(ctypes.byref(d), ctypes.byref(a), B, T)


def evict_check(d: CacheDesc, a: EvictArgs, B: int) -> int:
    return lib().moe_decode_evict_check(ctypes.byref(d), ctypes.byref(a), B)


class CachePlan(_PlanBase):
    """moe_decode_cache_plan and the runs on it: append, attend, evict.

    B sequences, T token rows; the first B rows of page_table and seq_lens and
    the first B + 1 of q_start are read."""

    _kind = "cache"

    def __init__(self, desc, device: int = 0):
        super().__init__(desc, device)
        d = self.desc
        self._heads, self._kv, self._D = d.heads, d.kv_heads, d.head_dim
        self._B, self._P = d.max_batch, d.max_pages
        self._scale = (d.pages, 2, d.kv_heads)
        self._pool = self._scale + (PAGE_TOKENS * d.head_dim,)

    def _cache(self, what, B, T, pool, pool_scale, page_table, seq_lens, q_start):
        dev = self.device
        if not (0 <= B <= self._B and T >= 0):
            _need(False, what, "B must be in [0, %d] and T not negative", self._B)
        return (_tensor(what, "pool", pool, _CODES, self._pool, dev),
                _tensor(what, "pool_scale", pool_scale, _BYTES, self._scale, dev),
                _rows(what, "page_table", page_table, _I32, (B, self._P), dev),
                _rows(what, "seq_lens", seq_lens, _I32, (B,), dev),
                _rows(what, "q_start", q_start, _I32, (B + 1,), dev))

    def append(self, B: int, T: int, *, k, v, pool, pool_scale, page_table, seq_lens, q_start,
               stream=None) -> None:
        """moe_decode_cache_append: K and V [T, kv_heads, head_dim] of the new
        tokens into their pages."""
        what, dev = "moe_decode_cache_append", self.device
        c = self._cache(what, B, T, pool, pool_scale, page_table, seq_lens, q_start)
        pk, sk = _heads(what, "k", k, T, self._kv, self._D, dev)
        pv, sv = _heads(what, "v", v, T, self._kv, self._D, dev)
        if B == 0 or T == 0:
            return
        rc = self._lib.moe_decode_cache_append(self._h, _pack_append(*c, pk, pv, sk, sv), B, T,
                                               _stream_of(stream, dev))
        if rc:
            _done(rc, what)

    def attend(self, B: int, T: int, *, q, pool, pool_scale, page_table, seq_lens, q_start, out,
               sm_scale, mass_in=None, mass_out=None, stream=None) -> None:
        """moe_decode_cache_attend: out [T, heads, head_dim] of the queries q
        over the cache, and with mass_out the pages' accumulated weight."""
        what, dev = "moe_decode_cache_attend", self.device
        c = self._cache(what, B, T, pool, pool_scale, page_table, seq_lens, q_start)
        pq, sq = _heads(what, "q", q, T, self._heads, self._D, dev)
        po, so = _heads(what, "out", out, T, self._heads, self._D, dev)
        mi = mo = 0
        if mass_in is not None:
            mi = _rows(what, "mass_in", mass_in, _F32, (B, self._P), dev)
        if mass_out is not None:
            mo = _rows(what, "mass_out", mass_out, _F32, (B, self._P), dev)
        if B == 0 or (T == 0 and not mo):
            return
        try:
            a = _pack_attend(*c, pq, sq, po, so, sm_scale, mi, mo)
        except OverflowError:
            _need(False, what, "sm_scale must be finite in 32 bits")
        rc = self._lib.moe_decode_cache_attend(self._h, a, B, T, _stream_of(stream, dev))
        if rc:
            _done(rc, what)

    def evict(self, B: int, keep: int, *, sink, recent, page_table, seq_lens, mass, out_table,
              out_lens, out_mass, freed, n_freed, stream=None) -> None:
        """moe_decode_cache_evict: the pages that each sequence keeps."""
        what, dev = "moe_decode_cache_evict", self.device
        if not 0 <= B <= self._B:
            _need(False, what, "B must be in [0, %d]", self._B)
        table, row = (B, self._P), (B,)
        p = (_rows(what, "page_table", page_table, _I32, table, dev),
             _rows(what, "seq_lens", seq_lens, _I32, row, dev),
             _rows(what, "mass", mass, _F32, table, dev),
             _rows(what, "out_table", out_table, _I32, table, dev),
             _rows(what, "out_lens", out_lens, _I32, row, dev),
             _rows(what, "out_mass", out_mass, _F32, table, dev),
             _rows(what, "freed", freed, _I32, table, dev),
             _rows(what, "n_freed", n_freed, _I32, row, dev))
        try:
            a = _pack_evict(*p, keep, sink, recent)
        except struct.error:
            _need(False, what, "keep, sink and recent must be integers of 32 bits")
        if B == 0:
            return
        rc = self._lib.moe_decode_cache_evict(self._h, a, B, _stream_of(stream, dev))
        if rc:
            _done(rc, what)
