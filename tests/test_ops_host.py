"""The refusals of the operators beside the MoE layer, on the host: every
check runs before any launch."""

import ctypes
import math

import pytest
import torch

import moe_decode_layer_sigmoid_amd as md

OK, BAD, UNS = md.OK, md.ERR_INVALID_ARG, md.ERR_UNSUPPORTED
P = 0x10000  # stands for an aligned device pointer; checks do not dereference


# ---- quantiser -----------------------------------------------------------------

@pytest.mark.parametrize("kw,code", [
    (dict(x=None), BAD), (dict(codes=None), BAD), (dict(scales=None), BAD), (dict(M=-1), BAD),
    (dict(K=0), BAD), (dict(limit=-1.0), BAD), (dict(limit=math.nan), BAD), (dict(limit=1e19, stride=512), BAD),
    (dict(M=(1 << 20) - 1, K=16512, stride=16512), UNS), (dict(M=(1 << 18) + 1, K=65536, stride=65536), UNS), (dict(x=P + 8), BAD),
    (dict(codes=P + 4), BAD), (dict(stride=255), BAD), (dict(stride=260), BAD),
    (dict(limit=7.0, stride=264), BAD), (dict(K=100, stride=256), UNS),
    (dict(K=65664, stride=65664), UNS), (dict(M=(1 << 20) + 1), UNS), (dict(M=0), OK),
])
def test_quant_refusals(kw, code):
    a = dict(x=P, stride=256, M=2, K=256, limit=0.0, codes=P, scales=P)
    a.update(kw)
    assert md.lib().moe_decode_quant(a["x"], a["stride"], a["M"], a["K"], a["limit"], a["codes"],
                                     a["scales"], None) == code


def test_quant_python_refusals():
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    with pytest.raises(md.MoeDecodeError):  # not on a GPU
        md.quant(x, torch.zeros(2, 256, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8))


# ---- product -------------------------------------------------------------------

@pytest.mark.parametrize("kw,code", [
    (dict(), OK), (dict(N=1, K=128, max_rows=1), OK), (dict(N=0), BAD), (dict(K=0), BAD),
    (dict(max_rows=0), BAD), (dict(scale_fmt=2), BAD), (dict(out_fmt=2), BAD), (dict(K=192), UNS),
    (dict(K=65664), UNS), (dict(N=(1 << 20) + 1), UNS), (dict(max_rows=(1 << 20) + 1), UNS),
])
def test_product_desc(kw, code):
    a = dict(N=1000, K=512, max_rows=16, scale_fmt="fp32", out_fmt="bf16")
    a.update(kw)
    assert md.product_desc_check(md.make_product_desc(**a)) == code


@pytest.mark.parametrize("kw,M,code", [
    ({}, 16, OK), ({}, 0, OK), ({}, -1, BAD), ({}, 17, BAD), (dict(codes=None), 1, BAD),
    (dict(scales=None), 1, BAD), (dict(w=None), 1, BAD), (dict(w_scale=None), 1, BAD),
    (dict(out=None), 1, BAD), (dict(codes=P + 8), 1, BAD), (dict(w=P + 8), 1, BAD),
    (dict(w_scale=P + 2), 1, BAD), (dict(out=P + 1), 1, BAD), (dict(out=P + 2), 1, OK),
    (dict(scales=P + 1), 1, OK), (dict(out_stride=999), 1, BAD),
])
def test_product_args(kw, M, code):
    a = dict(codes=P, scales=P, w=P, w_scale=P, out=P, out_stride=1000)
    a.update(kw)
    assert md.product_args_check(md.make_product_desc(1000, 512, 16), md.ProductArgs(**a), M) == code


def test_product_null():
    lib = md.lib()
    assert lib.moe_decode_product_run(None, None, 1, None) == BAD
    assert lib.moe_decode_product_destroy(None) == OK
    assert lib.moe_decode_product_workspace_bytes(None) == 0
    out = ctypes.c_void_p(1)
    assert lib.moe_decode_product_plan(None, 0, ctypes.byref(out)) == BAD and not out.value


# ---- cache ---------------------------------------------------------------------

GOOD = dict(heads=8, kv_heads=2, head_dim=128, pages=100, max_batch=4, max_pages=32, max_q=4)


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(head_dim=256), OK), (dict(heads=0), BAD), (dict(kv_heads=0), BAD),
    (dict(head_dim=0), BAD), (dict(pages=0), BAD), (dict(max_batch=0), BAD),
    (dict(max_pages=-1), BAD), (dict(max_q=0), BAD), (dict(with_mass=2), BAD),
    (dict(head_dim=96), UNS), (dict(head_dim=320), UNS), (dict(heads=9), UNS),
    (dict(heads=34), UNS), (dict(heads=129, kv_heads=129), UNS), (dict(max_batch=1025), UNS),
    (dict(max_pages=16385), UNS), (dict(max_q=257), UNS), (dict(pages=(1 << 24) + 1), UNS),
])
def test_cache_desc(kw, code):
    assert md.cache_desc_check(md.make_cache_desc(**{**GOOD, **kw})) == code


def cache(**kw):
    a = dict(pool=P, pool_scale=P, page_table=P, seq_lens=P, q_start=P)
    a.update(kw)
    return md.Cache(**a)


BAD_CACHES = [dict(pool=None), dict(pool=P + 8), dict(pool_scale=None), dict(page_table=None),
              dict(page_table=P + 2), dict(seq_lens=None), dict(q_start=None), dict(q_start=P + 1)]


def test_append_args():
    d = md.make_cache_desc(**GOOD)

    def check(B=4, T=6, c=None, **kw):
        a = dict(k=P, v=P, k_stride=256, v_stride=256)
        a.update(kw)
        return md.append_check(d, md.AppendArgs(c or cache(), **a), B, T)

    assert check() == OK and check(B=0) == OK and check(T=0) == OK and check(k_stride=264) == OK
    assert check(B=5) == BAD and check(B=-1) == BAD and check(T=-1) == BAD
    for kw in (dict(k=None), dict(v=None), dict(k=P + 8), dict(v=P + 2), dict(k_stride=255),
               dict(v_stride=128), dict(v_stride=260)):
        assert check(**kw) == BAD, kw
    for kw in BAD_CACHES:
        assert check(c=cache(**kw)) == BAD, kw


def test_attend_args():
    d = md.make_cache_desc(**GOOD)
    no_mass = md.make_cache_desc(**GOOD, with_mass=False)

    def check(B=4, T=6, c=None, desc=d, **kw):
        a = dict(q=P, q_stride=1024, out=2 * P, out_stride=1024, sm_scale=0.1)
        a.update(kw)
        return md.attend_check(desc, md.AttendArgs(c or cache(), **a), B, T)

    assert check() == OK and check(out_stride=1028) == OK and check(mass_out=P) == OK
    assert check(mass_out=P, mass_in=P) == OK
    for kw in (dict(B=5), dict(T=-1), dict(q=None), dict(out=None), dict(q=P + 8), dict(out=P + 4),
               dict(q_stride=1020), dict(q_stride=512), dict(out_stride=1026), dict(out=P),
               dict(sm_scale=math.inf), dict(sm_scale=math.nan), dict(mass_in=P),
               dict(mass_out=P + 2), dict(mass_out=P, desc=no_mass)):
        assert check(**kw) == BAD, kw
    for kw in BAD_CACHES:
        assert check(c=cache(**kw)) == BAD, kw


def test_evict_args():
    d = md.make_cache_desc(**GOOD)
    names = ["page_table", "seq_lens", "mass", "out_table", "out_lens", "out_mass", "freed", "n_freed"]

    def check(B=4, **kw):
        a = {n: P * (i + 1) for i, n in enumerate(names)}
        a.update(keep=8, sink=1, recent=2)
        a.update(kw)
        return md.evict_check(d, md.EvictArgs(**a), B)

    assert check() == OK and check(B=0) == OK
    assert check(out_table=P, out_lens=2 * P, out_mass=3 * P) == OK  # in place
    for n in names:
        assert check(**{n: None}) == BAD and check(**{n: P + 2}) == BAD, n
    for kw in (dict(B=5), dict(keep=0), dict(keep=2), dict(sink=-1), dict(recent=0),
               dict(sink=2 ** 31 - 1, recent=2), dict(freed=P), dict(n_freed=2 * P),
               dict(freed=8 * P)):
        assert check(**kw) == BAD, kw
    assert check(keep=3) == OK


def test_cache_null():
    lib = md.lib()
    for f in (lib.moe_decode_cache_append, lib.moe_decode_cache_attend):
        assert f(None, None, 1, 1, None) == BAD
    assert lib.moe_decode_cache_evict(None, None, 1, None) == BAD
    assert lib.moe_decode_cache_destroy(None) == OK
    assert lib.moe_decode_cache_workspace_bytes(None) == 0


def test_packed_arguments_are_the_structs():
    from moe_decode_layer_sigmoid_amd import ops

    def fields(s):
        for name, kind in s._fields_:
            v = getattr(s, name)
            if isinstance(v, ctypes.Structure):
                yield from fields(v)
            else:
                yield v

    for pack, kind, n in ((ops._pack_product, ops.ProductArgs, 6),
                          (ops._pack_append, ops.AppendArgs, 9),
                          (ops._pack_attend, ops.AttendArgs, 12),
                          (ops._pack_evict, ops.EvictArgs, 11)):
        b = pack(*range(1, n + 1))
        assert len(b) == ctypes.sizeof(kind)
        assert list(fields(kind.from_buffer_copy(b))) == list(range(1, n + 1))
