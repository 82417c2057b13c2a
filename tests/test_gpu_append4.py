"""cg_append into the 4-bit cache on the GPU: codes, ranges and raw rows against the
oracle's gauge and quantizer bit for bit, whatever the way the rows arrived."""
import numpy as np
import pytest

import oracle
from fixed_rate_compression_amd import binding as cg
from gpu_util import D, empty_u8, to_dev, to_host
from serve4_util import GROUP
from test_gpu_append import FILL, Filled

pytestmark = pytest.mark.gpu


def torch():
    return __import__("torch")


class Filled4(Filled):
    def __init__(self, seed, lengths, **kw):
        super().__init__(seed, lengths, block=GROUP, **kw)
        t = torch()
        L, B, H = self.L, self.B, self.H
        self.codec = cg.make_codec(cg.CG_BACKEND_KIVI, 4, GROUP)
        self.pay = t.full((L, 2, B, H, self.cap, D // 2), FILL, dtype=t.uint8, device="cuda")
        self.meta = t.full((L, 2, B, H, 4 * self.cap, 2), 5.0, device="cuda")

    def check(self, layer=0, lengths=None):
        pay, meta, tail = to_host(self.pay), to_host(self.meta), to_host(self.tail)
        for kind in (0, 1):
            for b, T in enumerate(lengths or self.lengths):
                for h in range(self.H):
                    raw = self.xh[kind, b, :T, h]
                    xg = oracle.gauge_forward(oracle.to_f32(raw), None if self.G is None else self.G[layer, kind, h], self.g)
                    code, m = oracle.serving4.quantize(xg, kind)
                    at = (layer, kind, b, h)
                    assert np.array_equal(pay[at][:T], code), at
                    assert np.all(pay[at][T:] == FILL), at
                    assert np.array_equal(meta[at][:len(m)].view(np.uint32), m.view(np.uint32)), at
                    assert np.all(meta[at][len(m):] == 5.0), at
                    if T:
                        lo = (T - 1) // GROUP * GROUP
                        assert np.array_equal(tail[at][:T - lo], raw[lo:]), at


@pytest.mark.parametrize("g", [0, 8, 16, 32, 128])
@pytest.mark.parametrize("bf16", [True, False])
def test_right_padded_prompts(g, bf16):
    f = Filled4(g, [150, 1, 0, 64, 65, 32, 33], g=g, bf16=bf16)
    f.put(f.x[0], f.x[1], 150, f.lengths, [0] * 7)
    f.check()


def test_left_padded_prompts():
    f = Filled4(40, [100, 3, 0, 33])
    t = torch()
    x = t.full_like(f.x, float("nan"))
    for b, T in enumerate(f.lengths):
        x[:, b, 100 - T:] = f.x[:, b, :T]
    f.put(x[0], x[1], 100, f.lengths)
    f.check()


@pytest.mark.parametrize("steps", [[1] * 40, [7, 1, 25, 64, 2, 1, 130], [63, 1, 1, 63, 65]])
@pytest.mark.parametrize("bf16", [True, False])
def test_token_by_token_and_in_pieces(steps, bf16):
    """However the rows arrive, every state of the cache is that of its rows."""
    t = torch()
    total = sum(steps)
    f = Filled4(60, [total, total - 5, total - 17], bf16=bf16, H=1)
    at = [0, -5, -17]          # two sequences begin later than the first
    for k, n in enumerate(steps):
        at = [p + n for p in at]
        ln = [max(p, 0) for p in at]
        new = t.full((2, 3, n, 1, D), float("nan"), dtype=f.x.dtype, device="cuda")
        for b, p in enumerate(at):
            lo = max(p - n, 0)
            if p > lo:
                new[:, b, n - (p - lo):] = f.x[:, b, lo:p]
        f.put(new[0], new[1], n, ln)
        if k % 9 == 0 or k + 1 == len(steps):
            f.check(lengths=ln)


def test_rows_of_the_last_block_again():
    """Rows may begin at one of the last block's: those behind the new ones are taken as not there."""
    f = Filled4(70, [60])
    f.put(f.x[0], f.x[1], 60, [60], [0])
    f.put(f.x[0][:, 40:45], f.x[1][:, 40:45], 5, [45], [40])
    pay, meta = to_host(f.pay), to_host(f.meta)
    for kind in (0, 1):
        xg = oracle.gauge_forward(oracle.to_f32(f.xh[kind, 0, :45, 0]), f.G[0, kind, 0], f.g)
        code, m = oracle.serving4.quantize(xg, kind)
        assert np.array_equal(pay[0, kind, 0, 0][:45], code)
        assert np.array_equal(meta[0, kind, 0, 0][:len(m)], m)


@pytest.mark.parametrize("g", [0, 8, 16, 32])
@pytest.mark.parametrize("bf16", [True, False])
def test_whole_blocks_equal_cg_encode(g, bf16):
    t = torch()
    f = Filled4(80 + g, [128, 128], g=g, bf16=bf16)
    f.put(f.x[0], f.x[1], 128, f.lengths)
    kv = f.x.transpose(2, 3).contiguous()
    pb, mb, _ = cg.cg_encoded_bytes(f.shape, f.codec)
    pay, meta = empty_u8(pb), t.zeros(mb // 4, device="cuda")
    cg.cg_encode(f.shape, kv, f.gauge, f.codec, 0, 128, pay, meta)
    assert t.equal(pay, f.pay.view(-1)) and t.equal(meta, f.meta.view(-1))


def test_layers_and_strided_rows():
    """Rows as parts of a fused projection's output; only layer 1 changes."""
    t = torch()
    f = Filled4(90, [50, 20], L=3, H=2)
    wide = t.zeros((2, 50, 8, D), dtype=f.x.dtype, device="cuda")
    wide[:, :, 4:6], wide[:, :, 6:8] = f.x[0], f.x[1]
    f.put(wide[:, :, 4:6], wide[:, :, 6:8], 50, f.lengths, [0, 0], layer=1)
    f.check(layer=1)
    for l in (0, 2):
        assert bool((f.pay[l] == FILL).all()) and bool((f.meta[l] == 5.0).all()) and not f.tail[l].any()


def test_positions_outside_write_nothing():
    f = Filled4(95, [40, 40, 40])
    f.put(f.x[0, :, :4], f.x[1, :, :4], 4, [0, 1 << 30, -3], [5, f.cap, -9])
    assert bool((f.pay == FILL).all()) and bool((f.meta == 5.0).all()) and not f.tail.any()
    # beyond the capacity: the rows that fit
    f = Filled4(96, [64], cap=64)
    f.put(f.x[0], f.x[1], 64, [1 << 30], [0])
    f.check()


def test_captured_append():
    """A recorded append follows lengths on the device."""
    t = torch()
    f = Filled4(97, [70, 40], H=1)
    ln = t.zeros(2, dtype=t.int32, device="cuda")
    k, v = f.x[0, :, :1].clone(), f.x[1, :, :1].clone()
    def call():
        cg.cg_append(f.shape, f.gauge, f.codec, 0, 1, k, v, f.tail, f.pay, f.meta, ln)
    call()
    gr = t.cuda.CUDAGraph()
    with t.cuda.graph(gr):
        call()
    for i in range(70):
        ln.copy_(t.tensor([i + 1, min(i + 1, 40)], dtype=t.int32))
        k.copy_(f.x[0, :, i:i + 1])
        v.copy_(f.x[1, :, i:i + 1])
        if i >= 40:                     # the second sequence's last row once more
            k[1], v[1] = f.x[0, 1, 39:40], f.x[1, 1, 39:40]
        gr.replay()
        if i % 20 == 3:
            f.check(lengths=[i + 1, min(i + 1, 40)])
    f.check()


def test_constant_and_extreme_rows():
    """A channel that is constant over a block, tokens of equal values, magnitudes near the ends of fp32."""
    t = torch()
    f = Filled4(98, [70], g=0, bf16=False)
    f.x[:, :, :, :, 3] = 1.5
    f.x[:, :, 10, :, :] = -2.0
    f.x[:, :, 20, :, 64:] *= 1e30
    f.x[:, :, 21, :, :] *= 1e-35
    f.xh = to_host(f.x)
    f.put(f.x[0], f.x[1], 70, f.lengths, [0])
    f.check()
