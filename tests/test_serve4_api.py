"""Refusals of the entry points on the 4-bit cache, of cg_read and of cg_rotate: every argument is
checked on the host before any device work (no GPU is touched here)."""
import ctypes

import numpy as np
import pytest

from fixed_rate_compression_amd import binding as cg
from test_serve_api import FAR, P, append, attend, attn, codec, evict, shape

K4 = cg.make_codec(cg.CG_BACKEND_KIVI, 4, 32)


def kivi(bits=4, block=32, residual=0):
    return cg.make_codec(cg.CG_BACKEND_KIVI, bits, block, residual)


@pytest.mark.parametrize("call", [attend, append, evict])
@pytest.mark.parametrize("kw,code", [
    (dict(co=kivi(bits=2)), cg.CG_E_UNSUPPORTED), (dict(co=kivi(bits=8)), cg.CG_E_UNSUPPORTED),
    (dict(co=kivi(block=64)), cg.CG_E_UNSUPPORTED), (dict(co=kivi(block=0)), cg.CG_E_UNSUPPORTED),
    (dict(co=kivi(residual=32)), cg.CG_E_UNSUPPORTED),
    (dict(co=K4, sh=shape(token_capacity=80)), cg.CG_E_SHAPE),
    (dict(co=K4, sh=shape(kv=1)), cg.CG_E_SHAPE),
    (dict(co=K4, sh=shape(head_dim=64)), cg.CG_E_UNSUPPORTED),
    (dict(co=K4, cap=2 * 2 * 2 * 2 * 64 * 64 - 1), cg.CG_E_SIZE),
    (dict(co=K4, mcap=2 * 2 * 2 * 2 * 64 * 32 - 1), cg.CG_E_SIZE),
    (dict(co=K4, pay=P + 8), cg.CG_E_INVAL),
    (dict(co=K4, meta=None), cg.CG_E_INVAL),
])
def test_refusals_of_4_bit_caches(call, kw, code):
    assert call(**kw) == code
    assert cg.cg_last_error()


def test_other_refusals_are_those_of_8_bits():
    assert attend(co=K4, at=attn(layer=2)) == cg.CG_E_SHAPE
    assert attend(co=K4, mass=P, wsb=16) == cg.CG_E_SIZE
    assert append(co=K4, tail=None) == cg.CG_E_INVAL
    assert append(co=K4, n=0, k=None, v=None, tail=None) == cg.CG_OK
    assert evict(co=K4, budget=3) == cg.CG_E_SHAPE
    # ranges that overlap by their true sizes: 2 * 8 fields * 2 blocks of 128 pairs
    fields, ranges = 16, 16 * 64 * 32
    assert evict(co=K4, mo=P + ranges - 16) == cg.CG_E_INVAL
    assert evict(co=K4, po=P + fields * 64 * 64 - 16) == cg.CG_E_INVAL


def test_tokens_need_not_fill_a_key_range():
    n = ctypes.c_size_t()
    r = ctypes.byref
    assert cg.lib().cg_attend_workspace_bytes(r(shape(tokens=33)), r(cg.make_gauge(0)), r(K4), r(attn()), 1, r(n)) == cg.CG_OK
    assert attend(co=K4, sh=shape(tokens=33), at=attn(n_queries=0), q=None, out=None) == cg.CG_OK


def read(sh=None, co=None, g=None, layer=0, n=4, pay=P, cap=FAR, meta=P, mcap=FAR, ln=None, st=None, k=FAR, v=2 * FAR, bs=0,
         rs=0):
    r = ctypes.byref
    return cg.lib().cg_read(r(sh or shape()), pay, cap, meta, mcap, r(g or cg.make_gauge(0)), r(co or K4), layer, n, ln, st,
                            k, v, bs, rs, None)


@pytest.mark.parametrize("co", [K4, codec()])
@pytest.mark.parametrize("kw,code", [
    (dict(sh=shape(kv=1)), cg.CG_E_SHAPE), (dict(g=cg.CgGauge(12, P)), cg.CG_E_SHAPE), (dict(layer=2), cg.CG_E_SHAPE),
    (dict(layer=-1), cg.CG_E_SHAPE), (dict(n=-1), cg.CG_E_SHAPE), (dict(n=(1 << 31) - 1, sh=shape(batch=64)), cg.CG_E_SHAPE),
    (dict(k=None, v=None), cg.CG_E_INVAL), (dict(k=FAR + 4), cg.CG_E_INVAL), (dict(v=2 * FAR + 8), cg.CG_E_INVAL),
    (dict(ln=P + 1), cg.CG_E_INVAL), (dict(st=P + 2), cg.CG_E_INVAL), (dict(bs=-256), cg.CG_E_INVAL),
    (dict(rs=257), cg.CG_E_INVAL), (dict(rs=128), cg.CG_E_INVAL), (dict(bs=256), cg.CG_E_INVAL),
    (dict(k=P), cg.CG_E_INVAL), (dict(v=P + 16), cg.CG_E_INVAL), (dict(v=FAR), cg.CG_E_INVAL),
    (dict(v=FAR + 256), cg.CG_E_INVAL), (dict(v=FAR + 512, rs=256), cg.CG_E_INVAL), (dict(v=FAR + 512, rs=384), cg.CG_E_INVAL),
    (dict(v=FAR - 16), cg.CG_E_INVAL), (dict(cap=1000), cg.CG_E_SIZE), (dict(mcap=8), cg.CG_E_SIZE), (dict(pay=None), cg.CG_E_INVAL),
    (dict(sh=shape(batch=1), n=3, v=FAR + 1024, rs=1 << 40, bs=0), None),
])
def test_read_refusals(co, kw, code):
    if code is None:
        return
    assert read(co=co, **kw) == code
    assert cg.cg_last_error()


def test_read_of_nothing():
    assert read(n=0, k=None, v=None) == cg.CG_OK
    assert read(sh=shape(tokens=0)) == cg.CG_OK
    assert read(sh=shape(tokens=0), k=None) == cg.CG_OK
    # keys beside values in the same rows, one row a sequence too
    assert read(sh=shape(tokens=0), v=FAR + 512, rs=512, bs=4 * 512) == cg.CG_OK
    assert read(sh=shape(tokens=0), n=1, v=FAR + 512, bs=512) == cg.CG_OK


def test_read_strides_that_reach_too_far():
    assert read(n=(1 << 25), sh=shape(batch=2), rs=1 << 40, bs=1 << 40) == cg.CG_E_INVAL
    assert read(sh=shape(batch=1 << 21, heads=1), cap=1 << 62, mcap=1 << 62, bs=1 << 40) == cg.CG_E_INVAL


def rotary(**kw):
    a = dict(dim=128, interleaved=0, axes=1, dealt=0, sections=(ctypes.c_int32 * 4)(), eps=1e-6, magnitude=1.0, freq=P,
             q_weight=P, k_weight=None)
    a.update(kw)
    if not isinstance(a["sections"], ctypes.Array):
        a["sections"] = (ctypes.c_int32 * 4)(*a["sections"])
    return cg.CgRotary(**a)


def rows(at, bs=0, rs=0):
    return None if at is None else ctypes.byref(cg.CgRows(at, bs, rs))


def rotate(sh=None, ro=None, q_heads=4, n=3, pos=None, ln=None, st=None, q=rows(FAR), k=rows(2 * FAR), qo=rows(3 * FAR),
           ko=rows(4 * FAR)):
    return cg.lib().cg_rotate(ctypes.byref(sh or shape()), ctypes.byref(ro or rotary()), q_heads, n, pos, ln, st, q, k, qo, ko,
                              None)


@pytest.mark.parametrize("kw,code", [
    (dict(sh=shape(head_dim=64)), cg.CG_E_UNSUPPORTED), (dict(sh=shape(dtype=7)), cg.CG_E_INVAL),
    (dict(ro=rotary(dim=24)), cg.CG_E_UNSUPPORTED), (dict(ro=rotary(dim=144)), cg.CG_E_UNSUPPORTED),
    (dict(ro=rotary(dim=-16)), cg.CG_E_UNSUPPORTED), (dict(ro=rotary(axes=0)), cg.CG_E_SHAPE),
    (dict(ro=rotary(axes=5)), cg.CG_E_SHAPE), (dict(ro=rotary(interleaved=2)), cg.CG_E_INVAL),
    (dict(ro=rotary(dealt=-1)), cg.CG_E_INVAL), (dict(ro=rotary(axes=2, sections=(32, 31)), pos=P), cg.CG_E_SHAPE),
    (dict(ro=rotary(axes=2, sections=(-1, 65)), pos=P), cg.CG_E_SHAPE),
    (dict(ro=rotary(axes=2, sections=(30, 34), dealt=1), pos=P), cg.CG_E_SHAPE),
    (dict(ro=rotary(axes=3, sections=(20, 22, 22), dealt=1), pos=P), cg.CG_E_SHAPE),
    (dict(ro=rotary(axes=2, sections=(32, 32))), cg.CG_E_INVAL),
    (dict(ro=rotary(freq=None)), cg.CG_E_INVAL), (dict(ro=rotary(freq=P + 2)), cg.CG_E_INVAL),
    (dict(ro=rotary(eps=-1.0)), cg.CG_E_INVAL), (dict(ro=rotary(eps=float("nan"))), cg.CG_E_INVAL),
    (dict(ro=rotary(magnitude=float("inf"))), cg.CG_E_INVAL), (dict(ro=rotary(q_weight=P + 4)), cg.CG_E_INVAL),
    (dict(pos=P + 1), cg.CG_E_INVAL), (dict(ln=P + 2), cg.CG_E_INVAL), (dict(st=P + 1), cg.CG_E_INVAL),
    (dict(n=-1), cg.CG_E_SHAPE), (dict(q_heads=0), cg.CG_E_SHAPE), (dict(q_heads=(1 << 31) - 1), cg.CG_E_SHAPE),
    (dict(n=(1 << 31) - 1), cg.CG_E_SHAPE), (dict(q=None), cg.CG_E_INVAL), (dict(ko=None), cg.CG_E_INVAL),
    (dict(q=None, qo=None, k=None, ko=None), cg.CG_E_INVAL), (dict(q=rows(0)), cg.CG_E_INVAL),
    (dict(q=rows(FAR + 8)), cg.CG_E_INVAL), (dict(qo=rows(3 * FAR, rs=516)), cg.CG_E_INVAL),
    (dict(qo=rows(3 * FAR, bs=-512)), cg.CG_E_INVAL), (dict(qo=rows(3 * FAR, rs=256)), cg.CG_E_INVAL),
    (dict(qo=rows(3 * FAR, bs=512)), cg.CG_E_INVAL),
    (dict(qo=rows(FAR + 16)), cg.CG_E_INVAL), (dict(qo=rows(2 * FAR)), cg.CG_E_INVAL), (dict(ko=rows(FAR)), cg.CG_E_INVAL),
    (dict(ko=rows(3 * FAR)), cg.CG_E_INVAL), (dict(qo=rows(FAR, rs=1024)), cg.CG_E_INVAL),
    (dict(q=rows(FAR, bs=3 * 1024, rs=1024), qo=rows(FAR, bs=3 * 1024, rs=1024), k=rows(FAR + 512, bs=3 * 1024, rs=1024),
          ko=rows(FAR + 512, bs=3 * 1024, rs=1024)), cg.CG_E_INVAL),      # keys begin inside the queries
])
def test_rotate_refusals(kw, code):
    assert rotate(**kw) == code
    assert cg.cg_last_error()


def test_rotate_nothing_and_nulls():
    assert rotate(n=0) == cg.CG_OK
    r = ctypes.byref
    L = cg.lib()
    assert L.cg_rotate(None, r(rotary()), 4, 3, None, None, None, rows(FAR), None, rows(P), None, None) == cg.CG_E_INVAL
    assert L.cg_rotate(r(shape()), None, 4, 3, None, None, None, rows(FAR), None, rows(P), None, None) == cg.CG_E_INVAL


def test_binding_checks():
    """What the C calls cannot see of a tensor is checked before them."""
    import torch
    sh, g = shape(layers=1), cg.make_gauge(0)
    pay, meta = torch.zeros(8 * 64 * 64, dtype=torch.uint8), torch.zeros(8 * 4 * 64 * 2)
    k = torch.zeros(2, 3, 2, 128, dtype=torch.bfloat16)
    for kw in (dict(k=k.float()), dict(k=k[:, :, :1]), dict(v=k[:1].expand(2, 3, 2, 128)), dict(k=k[:, :1].expand(2, 3, 2, 128)),
               dict(k=k.transpose(2, 3).contiguous().transpose(2, 3)), dict(v=torch.zeros(2, 3, 4, 128, dtype=k.dtype)[:, :, :2]),
               dict(lengths=torch.zeros(2)), dict(starts=torch.zeros(1, dtype=torch.int32)), dict(k=None, v=None)):
        a = dict(k=k, v=k.clone(), lengths=None, starts=None)
        a.update(kw)
        with pytest.raises(ValueError):
            cg.cg_read(sh, pay, meta, g, K4, 0, a["k"], a["v"], a["lengths"], a["starts"], stream=0)
    with pytest.raises(ValueError, match="host memory"):
        cg.cg_read(sh, pay, meta, g, K4, 0, k, k.clone(), stream=0)

    f, w = torch.zeros(64), torch.ones(128)
    for kw in (dict(freq=f.double()), dict(freq=f.view(8, 8)), dict(freq=f[::2]), dict(q_weight=w.half()), dict(sections=[13] * 5)):
        a = dict(freq=f, sections=None, q_weight=w)
        a.update(kw)
        with pytest.raises(ValueError):
            cg.make_rotary(a["freq"], a["sections"], q_weight=a["q_weight"])
    q = torch.zeros(2, 3, 4, 128, dtype=torch.bfloat16)
    ro = cg.make_rotary(f, q_weight=w)
    two = cg.make_rotary(f, [32, 32])
    pos = torch.zeros(2, 2, 3, dtype=torch.int32)
    for kw in (dict(q=q.float()), dict(q=q[:, :2]), dict(qo=q[:, :, :2]), dict(k=q), dict(k=k[:1]), dict(qo=q[:1].expand(2, 3, 4, 128)),
               dict(q=q.transpose(2, 3)), dict(q=None), dict(ko=None), dict(ro=cg.make_rotary(f, q_weight=w[:64].clone())),
               dict(ro=two, pos=pos[:1]), dict(ro=two, pos=pos.long()), dict(pos=pos), dict(ln=torch.zeros(2)),
               dict(st=torch.zeros(1, dtype=torch.int32)), dict(k=k.transpose(2, 3).contiguous().transpose(2, 3))):
        a = dict(ro=ro, q=q, k=k, qo=q.clone(), ko=k.clone(), pos=None, ln=None, st=None)
        a.update(kw)
        with pytest.raises(ValueError):
            cg.cg_rotate(sh, a["ro"], a["q"], a["k"], a["qo"], a["ko"], a["ln"], a["st"], a["pos"], stream=0)
    with pytest.raises(ValueError, match="host memory"):
        cg.cg_rotate(sh, ro, q, k, q.clone(), k.clone(), stream=0)
