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


def declare(L) -> None:
    """The prototypes of include/moe_decode_ops.h on the loaded library."""
    P = ctypes.POINTER
    protos = {
        "quant": [_vp, _i64, _i32, _i32, ctypes.c_float, _vp, _vp, _vp],
        "product_desc_check": [P(ProductDesc)],
        "product_args_check": [P(ProductDesc), P(ProductArgs), _i32],
        "product_plan": [P(ProductDesc), ctypes.c_int, P(_vp)],
        "product_run": [_vp, P(ProductArgs), _i32, _vp],
        "product_destroy": [_vp],
        "cache_desc_check": [P(CacheDesc)],
        "append_check": [P(CacheDesc), P(AppendArgs), _i32, _i32],
        "attend_check": [P(CacheDesc), P(AttendArgs), _i32, _i32],
        "evict_check": [P(CacheDesc), P(EvictArgs), _i32],
        "cache_plan": [P(CacheDesc), ctypes.c_int, P(_vp)],
        "cache_destroy": [_vp],
        "cache_append": [_vp, P(AppendArgs), _i32, _i32, _vp],
        "cache_attend": [_vp, P(AttendArgs), _i32, _i32, _vp],
        "cache_evict": [_vp, P(EvictArgs), _i32, _vp],
    }
    for name, args in protos.items():
        f = getattr(L, "moe_decode_" + name)
        f.argtypes, f.restype = args, ctypes.c_int
    for name in ("product_workspace_bytes", "cache_workspace_bytes"):
        f = getattr(L, "moe_decode_" + name)
        f.argtypes, f.restype = [_vp], ctypes.c_size_t


def _need(ok: bool, what: str, why: str) -> None:
    if not ok:
        raise MoeDecodeError(ERR_INVALID_ARG, "%s: %s" % (what, why))


def _tensor(what, name, t, dtypes, shape, device) -> int:
    """The address of a contiguous tensor of one of `dtypes` and `shape` on
    CUDA device `device`."""
    if t.get_device() != device or t.dtype not in dtypes or tuple(t.shape) != shape \
            or not t.is_contiguous():
        raise MoeDecodeError(ERR_INVALID_ARG, "%s: %s must be a contiguous %s tensor %s on device "
                             "%d, got %s %s on %s" % (what, name, "/".join(str(d) for d in dtypes),
                                                      list(shape), device, t.dtype,
                                                      list(t.shape), t.device))
    return t.data_ptr()


# torch and the types of the operators' tensors, set at the first use: the
# package itself loads without torch.
torch = None
_CODES = _BYTES = _BF16 = _I32 = _F32 = ()


def _load_torch() -> None:
    global torch, _CODES, _BYTES, _BF16, _I32, _F32
    if torch is None:
        import torch as t

        _CODES, _BYTES = (t.uint8, t.float8_e4m3fn), (t.uint8,)
        _BF16 = (t.bfloat16, t.int16)  # int16: bf16 bit patterns
        _I32, _F32 = (t.int32,), (t.float32,)
        torch = t


def _heads(what, name, t, T, heads, D, device):
    """(address, token stride) of a [>= T, heads, D] bf16 tensor whose tokens
    may be strided."""
    if t.get_device() != device or t.dtype not in _BF16 or t.dim() != 3 or t.shape[0] < T \
            or t.shape[1] != heads or t.shape[2] != D or t.stride(2) != 1 \
            or (heads > 1 and t.stride(1) != D):
        raise MoeDecodeError(ERR_INVALID_ARG, "%s: %s must be a bf16 tensor [%d, %d, %d] on device "
                             "%d with contiguous tokens, got %s %s strides %s on %s"
                             % (what, name, T, heads, D, device, t.dtype, list(t.shape),
                                list(t.stride()), t.device))
    # one token: its stride means nothing
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else heads * D


def _stream_of(stream, device: int) -> int:
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
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
    _need(codes.dim() == 2 and x.dim() == 2, what, "x and codes must be matrices")
    M, K = codes.shape
    cols = K if limit is None else 2 * K
    _need(limit is None or limit > 0, what, "limit must be positive")
    _need(x.get_device() == device and x.dtype in _BF16 and tuple(x.shape) == (M, cols)
          and (x.stride(1) == 1 or cols == 1), what,
          "x must be a bf16 tensor [%d, %d] on the device of codes with contiguous rows" % (M, cols))
    _need(device >= 0, what, "tensors must be on a GPU")
    pc = _tensor(what, "codes", codes, _CODES, (M, K), device)
    ps = _tensor(what, "scales", scales, _BYTES, (M, K // 128), device)
    if M == 0:
        return
    xs = x.stride(0) if M > 1 else cols
    L, s = lib(), _stream_of(stream, device)
    if device == torch.cuda.current_device():
        rc = L.moe_decode_quant(x.data_ptr(), xs, M, K, limit or 0.0, pc, ps, s)
    else:
        with torch.cuda.device(device):
            rc = L.moe_decode_quant(x.data_ptr(), xs, M, K, limit or 0.0, pc, ps, s)
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
        self._h = ctypes.c_void_p()
        what = "moe_decode_%s_plan" % self._kind
        _done(getattr(lib(), what)(ctypes.byref(desc), device, ctypes.byref(self._h)), what)

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

    def run(self, M: int, *, codes, scales, w, w_scale, out, stream=None) -> None:
        """out [M, n] = (scales codes) (w_scale w)^T for the first M rows of
        codes, scales and out (whose rows may be strided)."""
        what, d, dev = "moe_decode_product_run", self.desc, self.device
        N, K = d.n, d.k
        _need(0 <= M <= d.max_rows, what, "M must be in [0, %d]" % d.max_rows)
        want = torch.float32 if d.out_fmt == OUT_FP32 else torch.bfloat16
        _need(out.get_device() == dev and out.dim() == 2 and out.shape[0] >= M and out.shape[1] == N
              and (out.dtype == want or (want is torch.bfloat16 and out.dtype == torch.int16))
              and (out.stride(1) == 1 or N == 1),
              what, "out must be a %s tensor [%d, %d] on device %d with contiguous rows"
              % (want, M, N, dev))
        _need(codes.dim() == 2 and codes.shape[0] >= M and scales.dim() == 2
              and scales.shape[0] >= M, what, "codes and scales must have %d rows" % M)
        fmt = _F32 if d.scale_fmt == SCALE_FP32 else _BYTES
        a = ProductArgs(
            _tensor(what, "codes", codes, _CODES, (codes.shape[0], K), dev),
            _tensor(what, "scales", scales, _BYTES, (scales.shape[0], K // 128), dev),
            _tensor(what, "w", w, _CODES, (N, K), dev),
            _tensor(what, "w_scale", w_scale, fmt, ((N + 127) // 128, K // 128), dev),
            out.data_ptr(), out.stride(0) if out.shape[0] > 1 else N)
        if M == 0:
            return
        _done(lib().moe_decode_product_run(self._h, ctypes.byref(a), M, _stream_of(stream, dev)),
              what)


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

    def _cache(self, what, B, pool, pool_scale, page_table, seq_lens, q_start) -> Cache:
        d, dev = self.desc, self.device
        _need(0 <= B <= d.max_batch, what, "B must be in [0, %d]" % d.max_batch)
        _need(page_table.shape[0] >= B and seq_lens.shape[0] >= B and q_start.shape[0] >= B + 1,
              what, "page_table, seq_lens and q_start must cover %d sequences" % B)
        return Cache(
            _tensor(what, "pool", pool, _CODES, (d.pages, 2, d.kv_heads, 64 * d.head_dim), dev),
            _tensor(what, "pool_scale", pool_scale, _BYTES, (d.pages, 2, d.kv_heads), dev),
            _tensor(what, "page_table", page_table, _I32, (page_table.shape[0], d.max_pages), dev),
            _tensor(what, "seq_lens", seq_lens, _I32, (seq_lens.shape[0],), dev),
            _tensor(what, "q_start", q_start, _I32, (q_start.shape[0],), dev))

    def append(self, B: int, T: int, *, k, v, pool, pool_scale, page_table, seq_lens, q_start,
               stream=None) -> None:
        """moe_decode_cache_append: K and V [T, kv_heads, head_dim] of the new
        tokens into their pages."""
        what, d, dev = "moe_decode_cache_append", self.desc, self.device
        c = self._cache(what, B, pool, pool_scale, page_table, seq_lens, q_start)
        pk, sk = _heads(what, "k", k, T, d.kv_heads, d.head_dim, dev)
        pv, sv = _heads(what, "v", v, T, d.kv_heads, d.head_dim, dev)
        if B == 0 or T == 0:
            return
        a = AppendArgs(c, pk, pv, sk, sv)
        _done(lib().moe_decode_cache_append(self._h, ctypes.byref(a), B, T,
                                            _stream_of(stream, dev)), what)

    def attend(self, B: int, T: int, *, q, pool, pool_scale, page_table, seq_lens, q_start, out,
               sm_scale, mass_in=None, mass_out=None, stream=None) -> None:
        """moe_decode_cache_attend: out [T, heads, head_dim] of the queries q
        over the cache, and with mass_out the pages' accumulated weight."""
        what, d, dev = "moe_decode_cache_attend", self.desc, self.device
        c = self._cache(what, B, pool, pool_scale, page_table, seq_lens, q_start)
        pq, sq = _heads(what, "q", q, T, d.heads, d.head_dim, dev)
        po, so = _heads(what, "out", out, T, d.heads, d.head_dim, dev)
        mi = mo = None
        if mass_in is not None:
            _need(mass_in.shape[0] >= B, what, "mass_in must cover %d sequences" % B)
            mi = _tensor(what, "mass_in", mass_in, _F32, (mass_in.shape[0], d.max_pages), dev)
        if mass_out is not None:
            _need(mass_out.shape[0] >= B, what, "mass_out must cover %d sequences" % B)
            mo = _tensor(what, "mass_out", mass_out, _F32, (mass_out.shape[0], d.max_pages), dev)
        if B == 0 or (T == 0 and mo is None):
            return
        a = AttendArgs(c, pq, sq, po, so, sm_scale, mi, mo)
        _done(lib().moe_decode_cache_attend(self._h, ctypes.byref(a), B, T,
                                            _stream_of(stream, dev)), what)

    def evict(self, B: int, keep: int, *, sink, recent, page_table, seq_lens, mass, out_table,
              out_lens, out_mass, freed, n_freed, stream=None) -> None:
        """moe_decode_cache_evict: the pages that each sequence keeps."""
        what, d, dev = "moe_decode_cache_evict", self.desc, self.device
        _need(0 <= B <= d.max_batch, what, "B must be in [0, %d]" % d.max_batch)
        ptrs = []
        for name, t, dt, wide in (("page_table", page_table, _I32, True),
                                  ("seq_lens", seq_lens, _I32, False), ("mass", mass, _F32, True),
                                  ("out_table", out_table, _I32, True),
                                  ("out_lens", out_lens, _I32, False),
                                  ("out_mass", out_mass, _F32, True), ("freed", freed, _I32, True),
                                  ("n_freed", n_freed, _I32, False)):
            _need(t.shape[0] >= B, what, "%s must cover %d sequences" % (name, B))
            ptrs.append(_tensor(what, name, t, dt,
                                (t.shape[0], d.max_pages) if wide else (t.shape[0],), dev))
        if B == 0:
            return
        a = EvictArgs(*ptrs, keep, sink, recent)
        _done(lib().moe_decode_cache_evict(self._h, ctypes.byref(a), B, _stream_of(stream, dev)),
              what)
