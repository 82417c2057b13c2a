"""cg_read on the GPU: rows of a layer of both serving caches against the oracle's decoded values and
inverse gauge, each sequence from its own position, other memory left alone."""
import numpy as np
import pytest

import oracle
from fixed_rate_compression_amd import binding as cg
from gpu_util import D, check_decoded, empty_u8, gauges_for, to_dev, to_host
from serve4_util import random_cache4
from serve_util import random_cache

pytestmark = pytest.mark.gpu
FILL = 7.0


def torch():
    return __import__("torch")


class Cache:
    def __init__(self, seed, bits, L=1, B=2, H=2, cap=256, T=None, block=32, g=16, bf16=True):
        rng = np.random.default_rng(seed)
        self.bits, self.B, self.H, self.cap, self.block, self.g, self.bf16 = bits, B, H, cap, block, g, bf16
        self.pay, self.meta = random_cache4(rng, L, B, H, cap) if bits == 4 else random_cache(rng, L, B, H, cap, block)
        self.G = gauges_for(seed + 1, L, 2, H, g)
        self.shape = cg.make_shape(L, 2, B, H, cap if T is None else T, cap, D, cg.CG_DTYPE_BF16 if bf16 else cg.CG_DTYPE_F32)
        self.codec = cg.make_codec(cg.CG_BACKEND_KIVI, 4, 32) if bits == 4 else cg.make_codec(cg.CG_BACKEND_BLOCK_UNIFORM, 8, block)
        self.gauge = cg.make_gauge(g, to_dev(np.ascontiguousarray(self.G)) if g else None)
        self.payd, self.metad = to_dev(self.pay), to_dev(self.meta)
        self.dtype = torch().bfloat16 if bf16 else torch().float32

    def values(self, layer, kind, b, h):
        """Gauged values in the decoder's fp32 operations."""
        at = (layer, kind, b, h)
        if self.bits == 4:
            code = oracle.serving4.codes(self.pay[at]).astype(np.float32)
            t, c = np.arange(self.cap)[:, None], np.arange(D)[None]
            m = self.meta[at][t // 32 * D + c if kind == 0 else t * 4 + c // 32]
            return m[..., 0] + m[..., 1] * code
        m = np.repeat(self.meta[at], self.block, axis=0)
        return m[:, :1] + m[:, 1:] * self.pay[at].astype(np.float32)

    def read(self, n, lengths=None, starts=None, layer=0, k=None, v=None):
        t = torch()
        dev = lambda x: None if x is None else t.tensor(x, dtype=t.int32, device="cuda")
        if k is None and v is None:
            k, v = (t.full((self.B, n, self.H, D), FILL, dtype=self.dtype, device="cuda") for _ in range(2))
        cg.cg_read(self.shape, self.payd, self.metad, self.gauge, self.codec, layer, k, v, dev(lengths), dev(starts))
        return k, v

    def check(self, got, n, lengths=None, starts=None, layer=0):
        lengths = lengths or [self.shape.tokens] * self.B
        for kind, x in enumerate(got):
            if x is None:
                continue
            x = to_host(x)
            for b in range(self.B):
                T = min(max(lengths[b], 0), self.shape.tokens)
                p0 = T - n if starts is None else starts[b]
                lo, hi = max(p0, 0), min(p0 + n, T)
                fill = oracle.from_f32(np.full((1, D), FILL, np.float32), x.dtype)[0, 0]
                for h in range(self.H):
                    rows = x[b, :, h]
                    there = np.zeros(n, bool)
                    there[max(lo - p0, 0):max(hi - p0, 0)] = True
                    assert np.all(rows[~there] == fill), (kind, b, h)
                    if there.any():
                        G = None if self.G is None else self.G[layer, kind, h]
                        self.rows(rows[there], self.values(layer, kind, b, h)[lo:hi], G, (kind, b, h))

    def rows(self, got, y, G, where):
        if self.g == 128 and self.bf16:  # fmaf chains here, not the full-head decoders' products
            ref = oracle.from_f32(oracle.gauge_inverse(y, G, 128), got.dtype)
            assert np.array_equal(got, ref), where
        else:
            check_decoded(np.ascontiguousarray(got), np.ascontiguousarray(y), G, self.g, where)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("g", [0, 8, 16, 32, 128])
def test_rows_of_both_caches(bits, bf16, g):
    c = Cache(10 + g, bits, g=g, bf16=bf16)
    c.check(c.read(256), 256)
    c.check(c.read(100, [256, 131], [77, 100]), 100, [256, 131], [77, 100])


@pytest.mark.parametrize("block", [16, 64])
def test_blocks_of_the_8_bit_cache(block):
    c = Cache(30 + block, 8, block=block)
    c.check(c.read(129, [256, 200], [50, 71]), 129, [256, 200], [50, 71])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 97, 200])
def test_lengths_and_positions(bits, n):
    """Every way a strip of rows can lie over the blocks; rows before the first and behind the last."""
    for starts, lengths in (([0, 31, 100], [224, 224, 150]), ([-5, 220, 33], [224, 224, 33]), ([-300, 224, 1], [3, 224, 0]), (None, [224, n, 5])):
        c = Cache(40 + n, bits, B=3, H=1, cap=256, T=224)
        c.check(c.read(n, lengths, starts), n, lengths, starts)


def test_lengths_far_outside():
    c = Cache(50, 4, B=4, T=200)
    ln, st = [1 << 30, -(1 << 31), 200, 200], [190, 0, (1 << 31) - 1, -(1 << 31)]
    c.check(c.read(64, ln, st), 64, ln, st)


@pytest.mark.parametrize("bits", [4, 8])
def test_layers_strides_and_one_kind(bits):
    """Rows as parts of wider ones, keys beside values; a layer of several; keys or values alone."""
    t = torch()
    c = Cache(60, bits, L=3, H=2)
    for n in (1, 70):
        wide = t.full((2, n, 9, D), FILL, dtype=c.dtype, device="cuda")
        k, v = wide[:, :, 3:5], wide[:, :, 5:7]
        c.read(n, None, [9, 100], layer=1, k=k, v=v)
        c.check((k, v), n, None, [9, 100], layer=1)
        assert bool((wide[:, :, :3] == FILL).all()) and bool((wide[:, :, 7:] == FILL).all())
        for kind in (0, 1):
            x = t.full((2, n, 2, D), FILL, dtype=c.dtype, device="cuda")
            c.read(n, layer=2, **{"kv"[kind]: x})
            c.check((None, x) if kind else (x, None), n, layer=2)


@pytest.mark.parametrize("bits", [4, 8])
def test_rows_that_are_not_numbers_stay_alone(bits):
    """Ranges behind the end are not looked at; a token's NaN range reaches its own row."""
    t = torch()
    c = Cache(70, bits, B=1, H=1)
    want = [x.clone() for x in c.read(256, [131], [0])]
    if bits == 4:
        c.metad[0, 0, 0, 0, -(-131 // 32) * D:] = float("nan")
        c.metad[0, 1, 0, 0, 4 * 131:] = float("nan")
    else:
        c.metad[0, :, 0, 0, -(-131 // 32):] = float("nan")
    for x, y in zip(c.read(256, [131], [0]), want):
        assert t.equal(x, y)
    if bits == 4:
        c.metad[0, 1, 0, 0, 4 * 50 + 1] = float("nan")
        k, v = c.read(256, [131], [0])
        assert bool(t.isnan(v[0, 50, 0, 32:64]).all())
        v[0, 50] = want[1][0, 50]
        assert t.equal(v, want[1]) and t.equal(k, want[0])


def test_reads_what_cg_decode_decodes():
    t = torch()
    for bits, g, bf16 in ((4, 16, True), (8, 32, True), (4, 8, False), (8, 0, True)):
        c = Cache(80 + g, bits, B=2, H=3, g=g, bf16=bf16)
        dec = t.empty((2, 2, 3, 256, D), dtype=c.dtype, device="cuda")
        cg.cg_decode(c.shape, c.payd.view(-1), c.metad.view(-1), c.gauge, c.codec, 0, 256, dec)
        k, v = c.read(256)
        assert t.equal(k, dec[0].transpose(1, 2)) and t.equal(v, dec[1].transpose(1, 2)), (bits, g)


def test_captured_read():
    t = torch()
    c = Cache(90, 4)
    ln, st = (t.zeros(2, dtype=t.int32, device="cuda") for _ in range(2))
    k, v = (t.empty((2, 65, 2, D), dtype=c.dtype, device="cuda") for _ in range(2))
    def call():
        cg.cg_read(c.shape, c.payd, c.metad, c.gauge, c.codec, 0, k, v, ln, st)
    call()
    gr = t.cuda.CUDAGraph()
    with t.cuda.graph(gr):
        call()
    for lengths, starts in (([256, 100], [100, 60]), ([30, 256], [0, 191]), ([0, 0], [0, 0])):
        ln.copy_(t.tensor(lengths, dtype=t.int32))
        st.copy_(t.tensor(starts, dtype=t.int32))
        k.fill_(FILL)
        v.fill_(FILL)
        gr.replay()
        c.check((k, v), 65, lengths, starts)


def test_offsets_past_32_bits():
    t = torch()
    cap, H = 1 << 22, 8
    small = Cache(95, 4, B=1, H=H, cap=64)
    pay = t.zeros((2, 2, 1, H, cap, D // 2), dtype=t.uint8, device="cuda")
    meta = t.zeros((2, 2, 1, H, 4 * cap, 2), device="cuda")
    pay[1, :, :, :, cap - 64:], meta[1, :, :, :, 4 * (cap - 64):] = small.payd[0], small.metad[0]
    shape = cg.make_shape(2, 2, 1, H, cap, cap, D, cg.CG_DTYPE_BF16)
    G = t.cat([t.zeros_like(to_dev(small.G)), to_dev(small.G)])
    k, v = (t.empty((1, 64, H, D), dtype=t.bfloat16, device="cuda") for _ in range(2))
    cg.cg_read(shape, pay, meta, cg.make_gauge(16, G), small.codec, 1, k, v)
    small.check((k, v), 64)
