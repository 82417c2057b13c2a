"""Refusals of the serving entry points: every argument is checked on the host
before any device work (no GPU is touched here)."""
import ctypes

import numpy as np
import pytest

from fixed_rate_compression_amd import binding as cg

P = 4096          # a 16-byte aligned address that is never dereferenced
FAR = 1 << 40


def shape(**kw):
    a = dict(layers=2, kv=2, batch=2, heads=2, tokens=64, token_capacity=64, head_dim=128, dtype=cg.CG_DTYPE_BF16)
    a.update(kw)
    return cg.CgShape(**a)


def codec(bits=8, block=32, backend=cg.CG_BACKEND_BLOCK_UNIFORM):
    return cg.make_codec(backend, bits, block)


def attn(**kw):
    a = dict(layer=0, q_heads=4, n_queries=1, causal=1, scale=0.1, lengths=None, starts=None, q_batch_stride=0,
             q_token_stride=0)
    a.update(kw)
    return cg.CgAttn(**a)


def attend(sh=None, co=None, at=None, g=None, pay=P, cap=FAR, meta=P, mcap=FAR, q=P, out=FAR, lse=None, mass=None,
           ws=P, wsb=FAR):
    sh, co, at, g = sh or shape(), co or codec(), at or attn(), g or cg.make_gauge(0)
    r = ctypes.byref
    return cg.lib().cg_attend(r(sh), pay, cap, meta, mcap, r(g), r(co), r(at), q, out, lse, mass, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(sh=shape(kv=1)), cg.CG_E_SHAPE),
    (dict(sh=shape(head_dim=64)), cg.CG_E_UNSUPPORTED),
    (dict(sh=shape(tokens=65)), cg.CG_E_SHAPE),
    (dict(sh=shape(token_capacity=1 << 31, tokens=4)), cg.CG_E_SHAPE),
    (dict(co=codec(bits=4)), cg.CG_E_UNSUPPORTED),
    (dict(co=codec(block=48)), cg.CG_E_UNSUPPORTED),
    (dict(co=cg.make_codec(cg.CG_BACKEND_ZFP, 8)), cg.CG_E_UNSUPPORTED),
    (dict(co=cg.make_codec(cg.CG_BACKEND_KIVI, 8, 32)), cg.CG_E_UNSUPPORTED),
    (dict(g=cg.CgGauge(16, None)), cg.CG_E_INVAL),
    (dict(g=cg.CgGauge(64, P)), cg.CG_E_UNSUPPORTED),
    (dict(pay=None), cg.CG_E_INVAL),
    (dict(pay=P + 8), cg.CG_E_INVAL),
    (dict(meta=None), cg.CG_E_INVAL),
    (dict(cap=2 * 2 * 2 * 2 * 64 * 128 - 1), cg.CG_E_SIZE),
    (dict(mcap=2 * 2 * 2 * 2 * 2 * 8 - 1), cg.CG_E_SIZE),
    (dict(at=attn(layer=2)), cg.CG_E_SHAPE),
    (dict(at=attn(layer=-1)), cg.CG_E_SHAPE),
    (dict(at=attn(q_heads=3)), cg.CG_E_SHAPE),
    (dict(at=attn(q_heads=0)), cg.CG_E_SHAPE),
    (dict(at=attn(n_queries=-1)), cg.CG_E_SHAPE),
    (dict(at=attn(n_queries=1 << 30)), cg.CG_E_SHAPE),
    (dict(at=attn(causal=2)), cg.CG_E_INVAL),
    (dict(at=attn(scale=float("nan"))), cg.CG_E_INVAL),
    (dict(at=attn(scale=float("inf"))), cg.CG_E_INVAL),
    (dict(at=attn(lengths=P + 2)), cg.CG_E_INVAL),
    (dict(at=attn(q_token_stride=516)), cg.CG_E_INVAL),
    (dict(at=attn(q_batch_stride=-512)), cg.CG_E_INVAL),
    (dict(q=None), cg.CG_E_INVAL),
    (dict(q=P + 2), cg.CG_E_INVAL),
    (dict(out=FAR + 8), cg.CG_E_INVAL),
    (dict(out=P), cg.CG_E_INVAL),
    (dict(q=P, out=P + 1024, at=attn(q_batch_stride=2048)), cg.CG_E_INVAL),
    (dict(lse=P + 1), cg.CG_E_INVAL),
    (dict(mass=P + 1), cg.CG_E_INVAL),
    (dict(mass=P, ws=None), cg.CG_E_SIZE),
    (dict(mass=P, wsb=16), cg.CG_E_SIZE),
])
def test_attend_refusals(kw, code):
    assert attend(**kw) == code
    assert cg.cg_last_error()


def test_attend_nulls_and_nothing_to_do():
    L, r, g = cg.lib(), ctypes.byref, cg.make_gauge(0)
    sh, co, at = shape(), codec(), attn()
    n = ctypes.c_size_t()
    assert L.cg_attend(None, P, FAR, P, FAR, r(g), r(co), r(at), P, FAR, None, None, P, FAR, None) == cg.CG_E_INVAL
    assert L.cg_attend(r(sh), P, FAR, P, FAR, None, r(co), r(at), P, FAR, None, None, P, FAR, None) == cg.CG_E_INVAL
    assert L.cg_attend(r(sh), P, FAR, P, FAR, r(g), r(co), None, P, FAR, None, None, P, FAR, None) == cg.CG_E_INVAL
    assert L.cg_attend_workspace_bytes(r(sh), r(g), r(co), r(at), 0, None) == cg.CG_E_INVAL
    assert attend(at=attn(n_queries=0), q=None, out=None) == cg.CG_OK
    assert L.cg_attend_workspace_bytes(r(sh), r(g), r(co), r(attn(n_queries=0)), 1, r(n)) == cg.CG_OK
    # the workspace grows with the tokens' bound and never needs lengths
    sizes = []
    for T in (64, 4096, 65536):
        assert L.cg_attend_workspace_bytes(r(shape(tokens=T, token_capacity=T)), r(g), r(co), r(at), 1, r(n)) == cg.CG_OK
        sizes.append(n.value)
    assert sizes[0] < sizes[1] < sizes[2]


def append(sh=None, co=None, g=None, layer=0, n=1, k=P, v=P, bs=0, rs=0, ln=None, st=None, tail=FAR, pay=P, cap=FAR,
           meta=P, mcap=FAR):
    r = ctypes.byref
    return cg.lib().cg_append(r(sh or shape()), r(g or cg.make_gauge(0)), r(co or codec()), layer, n, k, v, bs, rs, ln,
                              st, tail, pay, cap, meta, mcap, None)


@pytest.mark.parametrize("kw,code", [
    (dict(sh=shape(kv=1)), cg.CG_E_SHAPE), (dict(co=codec(bits=6)), cg.CG_E_UNSUPPORTED),
    (dict(g=cg.CgGauge(12, P)), cg.CG_E_SHAPE), (dict(layer=2), cg.CG_E_SHAPE), (dict(n=-1), cg.CG_E_SHAPE),
    (dict(n=(1 << 31) - 1, sh=shape(batch=64)), cg.CG_E_SHAPE), (dict(k=None), cg.CG_E_INVAL),
    (dict(v=P + 4), cg.CG_E_INVAL), (dict(tail=None), cg.CG_E_INVAL), (dict(tail=P), cg.CG_E_INVAL),
    (dict(bs=-256), cg.CG_E_INVAL), (dict(rs=257), cg.CG_E_INVAL), (dict(ln=P + 1), cg.CG_E_INVAL),
    (dict(st=P + 2), cg.CG_E_INVAL), (dict(cap=1000), cg.CG_E_SIZE), (dict(mcap=8), cg.CG_E_SIZE),
    (dict(pay=None), cg.CG_E_INVAL),
])
def test_append_refusals(kw, code):
    assert append(**kw) == code


def test_append_of_nothing():
    assert append(n=0, k=None, v=None, tail=None) == cg.CG_OK


def evict(sh=None, co=None, budget=2, sink=0, recent=1, mass=P, pay=P, cap=FAR, meta=P, mcap=FAR, ln=None, osh=None,
          po=FAR, pcap=FAR, mo=FAR, omcap=FAR, wo=FAR, kept=FAR, lo=FAR):
    r = ctypes.byref
    return cg.lib().cg_evict(r(sh or shape()), r(co or codec()), budget, sink, recent, mass, pay, cap, meta, mcap, ln,
                             r(osh or shape()), po, pcap, mo, omcap, wo, kept, lo, None)


@pytest.mark.parametrize("kw,code", [
    (dict(co=codec(bits=4)), cg.CG_E_UNSUPPORTED), (dict(osh=shape(layers=1)), cg.CG_E_SHAPE),
    (dict(osh=shape(batch=1)), cg.CG_E_SHAPE), (dict(osh=shape(heads=1)), cg.CG_E_SHAPE),
    (dict(budget=3), cg.CG_E_SHAPE), (dict(budget=0), cg.CG_E_SHAPE), (dict(recent=0), cg.CG_E_SHAPE),
    (dict(sink=-1), cg.CG_E_SHAPE), (dict(sink=2), cg.CG_E_SHAPE),
    (dict(sink=(1 << 31) - 1, recent=(1 << 31) - 1), cg.CG_E_SHAPE),
    (dict(mass=None), cg.CG_E_INVAL), (dict(kept=None), cg.CG_E_INVAL), (dict(lo=None), cg.CG_E_INVAL),
    (dict(wo=None), cg.CG_E_INVAL), (dict(mass=P + 1), cg.CG_E_INVAL), (dict(po=P + 16), cg.CG_E_INVAL),
    (dict(mo=P + 16), cg.CG_E_INVAL), (dict(wo=P + 4), cg.CG_E_INVAL), (dict(po=P), cg.CG_E_INVAL),
    (dict(po=P, mo=P, wo=P, osh=shape(token_capacity=128)), cg.CG_E_INVAL),
    (dict(ln=FAR + 4), cg.CG_E_INVAL), (dict(pcap=100), cg.CG_E_SIZE), (dict(omcap=8), cg.CG_E_SIZE),
    (dict(po=None), cg.CG_E_INVAL),
])
def test_evict_refusals(kw, code):
    assert evict(**kw) == code


def test_binding_checks_types_and_sizes():
    """What the C call cannot see of a tensor is checked before it."""
    import torch
    sh, co, g = shape(layers=1), codec(), cg.make_gauge(0)
    pay, meta = torch.zeros(2 * 2 * 2 * 64 * 128, dtype=torch.uint8), torch.zeros(2 * 2 * 2 * 2 * 2)
    q = torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16)
    at = attn()
    for kw in (dict(q=q.float()), dict(q=q[:, :, :2]), dict(q=q.expand(2, 1, 4, 128)[:, :, :, :64]),
               dict(out=torch.zeros(8)), dict(out=q[:1].clone()), dict(lse=torch.zeros(7)),
               dict(lse=torch.zeros(8, dtype=torch.float64)), dict(mass=torch.zeros(7)),
               dict(q=q[:1].expand(2, 1, 4, 128))):
        a = dict(q=q, out=q.clone(), lse=None, mass=None)
        a.update(kw)
        with pytest.raises(ValueError):
            cg.cg_attend(sh, pay, meta, g, co, at, a["q"], a["out"], a["lse"], a["mass"], None, stream=0)
    with pytest.raises(ValueError):
        cg.make_attn(0, 4, 1, 0.1, lengths=torch.zeros(2, dtype=torch.int64))
    k = torch.zeros(2, 1, 2, 128, dtype=torch.bfloat16)
    tail = torch.zeros(1, 2, 2, 2, 32, 128, dtype=torch.bfloat16)
    for kw in (dict(k=k.float()), dict(k=k[:, :, :1]), dict(v=k[:1].expand(2, 1, 2, 128)), dict(tail=tail[:, :1].clone()),
               dict(k=k.transpose(2, 3).contiguous().transpose(2, 3)), dict(lengths=torch.zeros(2, dtype=torch.int64)),
               dict(lengths=torch.zeros(1, dtype=torch.int32))):
        a = dict(k=k, v=k.clone(), tail=tail, lengths=None)
        a.update(kw)
        with pytest.raises(ValueError):
            cg.cg_append(sh, g, co, 0, 1, a["k"], a["v"], a["tail"], pay, meta, a["lengths"], stream=0)
    w, kept, ln = torch.zeros(8), torch.zeros(8, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for kw in (dict(mass=w[:7]), dict(kept=kept[:7]), dict(kept=kept.long()), dict(lo=ln[:1]), dict(wo=w.double())):
        a = dict(mass=w, kept=kept, lo=ln, wo=w.clone())
        a.update(kw)
        with pytest.raises(ValueError):
            cg.cg_evict(sh, co, 2, 0, 1, a["mass"], pay, meta, sh, pay.clone(), meta.clone(), a["wo"], a["kept"],
                        a["lo"], ln.clone(), stream=0)


def test_host_tensors_are_refused():
    """A tensor in host memory never reaches a kernel."""
    import torch

    sh, co, g = shape(), codec(), cg.make_gauge(0)
    pay, meta = torch.zeros(16 * 64 * 128, dtype=torch.uint8), torch.zeros(16 * 2 * 2)
    q = torch.zeros((2, 1, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="host memory"):
        cg.cg_attend(sh, pay, meta, g, co, attn(), q, torch.zeros_like(q), stream=0)
    k, tail = torch.zeros((2, 1, 2, 128), dtype=torch.bfloat16), torch.zeros(2 * 2 * 2 * 2 * 32 * 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="host memory"):
        cg.cg_append(sh, g, co, 0, 1, k, k, tail, pay, meta, stream=0)
    mass, kept, ln = torch.zeros((2, 2, 2, 2)), torch.zeros((2, 2, 2, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="host memory"):
        cg.cg_evict(sh, co, 1, 0, 1, mass, pay, meta, sh, pay, meta, mass, kept, ln, stream=0)


def test_small_arrays_are_refused():
    """Lengths, starts and gauges that hold less than a call reads of them."""
    import torch

    sh, co = shape(), codec()
    pay, meta = torch.zeros(16 * 64 * 128, dtype=torch.uint8), torch.zeros(16 * 2 * 2)
    q = torch.zeros((2, 1, 4, 128), dtype=torch.bfloat16)
    one, g = torch.zeros(1, dtype=torch.int32), cg.make_gauge(0)
    for kw in (dict(lengths=one), dict(starts=one)):
        with pytest.raises(ValueError, match=next(iter(kw))):
            cg.cg_attend(sh, pay, meta, g, co, cg.make_attn(0, 4, 1, 0.1, **kw), q, torch.zeros_like(q), stream=0)
    k, tail = torch.zeros((2, 1, 2, 128), dtype=torch.bfloat16), torch.zeros(2 * 2 * 2 * 2 * 32 * 128, dtype=torch.bfloat16)
    for G in (torch.zeros(2 * 2 * 2 * 128 * 16 - 1), torch.zeros(2 * 2 * 2 * 128 * 16, dtype=torch.float64)):
        g = cg.make_gauge(16, G)
        with pytest.raises(ValueError, match="gauge"):
            cg.cg_attend(sh, pay, meta, g, co, cg.make_attn(0, 4, 1, 0.1), q, torch.zeros_like(q), stream=0)
        with pytest.raises(ValueError, match="gauge"):
            cg.cg_append(sh, g, co, 0, 1, k, k, tail, pay, meta, stream=0)


def test_strides_that_reach_too_far_are_refused():
    far = 1 << 40
    assert attend(at=attn(n_queries=1 << 21, q_token_stride=far)) == cg.CG_E_INVAL
    r = ctypes.byref
    assert cg.lib().cg_append(r(shape()), r(cg.make_gauge(0)), r(codec()), 0, 1 << 21, P, P, 0, far, None, None, FAR, P,
                              FAR, P, FAR, None) == cg.CG_E_INVAL


@pytest.mark.parametrize("tokens", [64, 2048, 4096, 32768])
@pytest.mark.parametrize("batch,n", [(1, 1), (2, 1), (64, 1), (8, 20), (3, 300)])
def test_workspace_does_not_depend_on_the_arrays(tokens, batch, n):
    """A size asked for without lengths serves calls with them."""
    sh = shape(batch=batch, heads=8, tokens=tokens, token_capacity=tokens)
    need = [cg.cg_attend_workspace_bytes(sh, cg.make_gauge(0), codec(), attn(q_heads=32, n_queries=n, lengths=a, starts=b), m)
            for m in (False, True) for a in (None, P) for b in (None, P)]
    assert len(set(need[:4])) == 1 and len(set(need[4:])) == 1


def test_strides_of_single_rows_are_free():
    """One sequence, or one row a sequence: torch leaves any stride there, and k and v may
    differ in it (a rotated key beside a slice of a fused projection)."""
    import torch

    wide = torch.zeros((2, 1, 6, 128), dtype=torch.bfloat16)
    tails = torch.zeros(2 * 2 * 2 * 2 * 32 * 128, dtype=torch.bfloat16)
    for batch, n, k, v in ((1, 1, wide[:1, :, 2:4].contiguous(), wide[:1, :, 4:6]),
                           (1, 2, wide[:, 0, 2:4].unsqueeze(0), wide.transpose(0, 1)[:, :, 4:6]),
                           (2, 1, wide[:, :, 2:4], wide.as_strided((2, 1, 2, 128), (768, 128, 128, 1), 512))):
        sh = shape(batch=batch)
        pay, meta = torch.zeros(8 * batch * 64 * 128, dtype=torch.uint8), torch.zeros(8 * batch * 2 * 2)
        # past the checks of the strides: what is left to refuse is that these are in host memory
        with pytest.raises(ValueError, match="host memory"):
            cg.cg_append(sh, cg.make_gauge(0), codec(), 0, n, k, v, tails, pay, meta, stream=0)
    k = wide[:, :, 2:4].contiguous()
    pay, meta = torch.zeros(16 * 64 * 128, dtype=torch.uint8), torch.zeros(16 * 2 * 2)
    with pytest.raises(ValueError, match="strides"):            # two sequences that do lie apart differently
        cg.cg_append(shape(), cg.make_gauge(0), codec(), 0, 1, k, wide[:, :, 4:6], tails, pay, meta, stream=0)


@pytest.mark.parametrize("scale", [2.5e38, -2.5e38, 3.4e38])
def test_scales_whose_factor_is_not_finite_are_refused(scale):
    """Scores are formed in units of log2: scale log2(e) has to be an fp32 number."""
    assert np.isfinite(np.float32(scale))
    assert attend(at=attn(scale=scale, n_queries=0)) == cg.CG_E_INVAL
    assert attend(at=attn(scale=scale / 2, n_queries=0)) == cg.CG_OK


@pytest.mark.parametrize("batch,heads,q_heads,capacity,block,n", [
    (64, 8, 32, 131072, 32, 2000), (64, 8, 32, 131072, 16, 2000), (128, 8, 8, 131072, 64, 300),
    (64, 8, 2048, 65536, 32, 9), (8, 8, 32, 131072, 32, 2000), (1, 8, 32, 131072, 32, 4096), (2, 4, 16, 8192, 64, 700),
    (256, 8, 32, 65536, 32, 16)])
def test_workspace_of_the_block_weights_is_what_the_header_says(batch, heads, q_heads, capacity, block, n):
    """8 bytes a row and 32 tokens of the capacity; past 64 rows a KV head queries go in turn
    above 1 GiB, 128 rows (or a query's) at least."""
    sh = shape(layers=1, batch=batch, heads=heads, tokens=capacity, token_capacity=capacity)
    at = attn(q_heads=q_heads, n_queries=n)
    need = cg.cg_attend_workspace_bytes(sh, cg.make_gauge(0), codec(block=block), at, True)
    ratio, entries = q_heads // heads, capacity // min(block, 32)
    each = 8 * batch * heads * entries
    rows = n * ratio
    if rows > 64:
        rows = min(rows, max((1 << 30) // each, 128, ratio))
    # the parts of split rows and the rows' log-sums come on top: 512 + 8 + 4 bytes a row and split
    splits = max(1, 768 // (batch * heads)) if rows <= 64 else 512
    rest = batch * heads * rows * 524 * splits + 4 * 256 + 8 * batch
    assert each * min(rows, 64) <= need <= each * rows + rest


def test_workspace_of_the_block_weights_past_the_limit():
    sh = shape(layers=1, batch=64, heads=8, tokens=131072, token_capacity=131072)
    need = cg.cg_attend_workspace_bytes(sh, cg.make_gauge(0), codec(), attn(q_heads=32, n_queries=2048), True)
    assert need == 512 * 4096 * 1024 + 512 * 128 * 4      # 2 GiB of sums, 128 rows at a time
