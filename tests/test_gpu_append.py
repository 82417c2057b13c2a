"""cg_append on the GPU: codes, ranges and raw rows against the oracle's gauge
and quantizer bit for bit, whatever the way the rows arrived."""
import numpy as np
import pytest

import oracle
from fixed_rate_compression_amd import binding as cg
from gpu_util import D, empty_u8, gauges_for, to_dev, to_host

pytestmark = pytest.mark.gpu
FILL = 77        # codes nobody wrote


def torch():
    return __import__("torch")


class Filled:
    """An empty cache and the rows each sequence is to hold."""

    def __init__(self, seed, lengths, L=1, H=2, cap=None, block=32, g=16, bf16=True):
        t = torch()
        rng = np.random.default_rng(seed)
        self.B, self.H, self.L, self.block, self.g, self.bf16 = len(lengths), H, L, block, g, bf16
        self.lengths = lengths
        T = max(max(lengths), 1)
        self.cap = cap or -(-T // block) * block
        x = rng.standard_normal((2, self.B, T, H, D)).astype(np.float32) * np.exp(rng.standard_normal((2, 1, 1, H, D)))
        self.xh = oracle.f32_to_bf16(x.astype(np.float32)) if bf16 else x.astype(np.float32)
        self.x = to_dev(self.xh)
        self.G = gauges_for(seed + 1, L, 2, H, g)
        self.gauge = cg.make_gauge(g, to_dev(np.ascontiguousarray(self.G)) if g else None)
        self.shape = cg.make_shape(L, 2, self.B, H, self.cap, self.cap, D, cg.CG_DTYPE_BF16 if bf16 else cg.CG_DTYPE_F32)
        self.codec = cg.make_codec(cg.CG_BACKEND_BLOCK_UNIFORM, 8, block)
        self.pay = t.full((L, 2, self.B, H, self.cap, D), FILL, dtype=t.uint8, device="cuda")
        self.meta = t.full((L, 2, self.B, H, self.cap // block, 2), 5.0, device="cuda")
        self.tail = t.zeros((L, 2, self.B, H, block, D), dtype=self.x.dtype, device="cuda")

    def put(self, k, v, n, lengths, starts=None, layer=0):
        t = torch()
        ln = t.tensor(lengths, dtype=t.int32, device="cuda")
        st = None if starts is None else t.tensor(starts, dtype=t.int32, device="cuda")
        cg.cg_append(self.shape, self.gauge, self.codec, layer, n, k, v, self.tail, self.pay, self.meta, ln, st)

    def check(self, layer=0, lengths=None):
        pay, meta, tail = to_host(self.pay), to_host(self.meta), to_host(self.tail)
        for kind in (0, 1):
            for b, T in enumerate(lengths or self.lengths):
                for h in range(self.H):
                    raw = self.xh[kind, b, :T, h]
                    xg = oracle.gauge_forward(oracle.to_f32(raw), None if self.G is None else self.G[layer, kind, h], self.g)
                    codes, m = oracle.serving.quantize(xg, self.block)
                    at = (layer, kind, b, h)
                    assert np.array_equal(pay[at][:T], codes), at
                    assert np.all(pay[at][T:] == FILL), at
                    assert np.array_equal(meta[at][:len(m)].view(np.uint32), m.view(np.uint32)), at
                    assert np.all(meta[at][len(m):] == 5.0), at
                    if T:
                        lo = (T - 1) // self.block * self.block
                        assert np.array_equal(tail[at][:T - lo], raw[lo:]), at


@pytest.mark.parametrize("g", [0, 8, 16, 32, 128])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("block", [16, 32, 64])
def test_right_padded_prompts(g, bf16, block):
    f = Filled(g + block, [150, 1, 0, 64, 65], block=block, g=g, bf16=bf16)
    f.put(f.x[0], f.x[1], 150, f.lengths, [0] * 5)
    f.check()


@pytest.mark.parametrize("block", [16, 32, 64])
def test_left_padded_prompts(block):
    f = Filled(40 + block, [100, 3, 0, 33], block=block)
    t = torch()
    x = t.full_like(f.x, float("nan"))
    for b, T in enumerate(f.lengths):
        x[:, b, 100 - T:] = f.x[:, b, :T]
    f.put(x[0], x[1], 100, f.lengths)
    f.check()


@pytest.mark.parametrize("steps", [[1] * 40, [7, 1, 25, 64, 2, 1, 130], [63, 1, 1, 63, 65]])
@pytest.mark.parametrize("block", [16, 32, 64])
@pytest.mark.parametrize("bf16", [True, False])
def test_token_by_token_and_in_pieces(steps, block, bf16):
    """However the rows arrive, every state of the cache is that of its rows."""
    total = sum(steps)
    f = Filled(60 + block, [total, total - 5, total - 17], block=block, bf16=bf16, H=1)
    at = [0, -5, -17]          # two sequences begin later than the first
    for k, n in enumerate(steps):
        at = [p + n for p in at]
        ln = [max(p, 0) for p in at]
        t = torch()
        new = t.full((2, 3, n, 1, D), float("nan"), dtype=f.x.dtype, device="cuda")
        for b, p in enumerate(at):
            lo = max(p - n, 0)
            if p > lo:
                new[:, b, n - (p - lo):] = f.x[:, b, lo:p]
        f.put(new[0], new[1], n, ln)
        if k % 9 == 0 or k + 1 == len(steps):
            f.check(lengths=ln)


@pytest.mark.parametrize("g", [0, 8, 16, 32])
@pytest.mark.parametrize("bf16", [True, False])
def test_whole_blocks_equal_cg_encode(g, bf16):
    t = torch()
    f = Filled(80 + g, [128, 128], block=32, g=g, bf16=bf16)
    f.put(f.x[0], f.x[1], 128, f.lengths)
    kv = f.x.transpose(2, 3).contiguous()
    pb, mb, _ = cg.cg_encoded_bytes(f.shape, f.codec)
    pay, meta = empty_u8(pb), t.zeros(mb // 4, device="cuda")
    cg.cg_encode(f.shape, kv, f.gauge, f.codec, 0, 128, pay, meta)
    assert t.equal(pay, f.pay.view(-1)) and t.equal(meta, f.meta.view(-1))


def test_layers_and_strided_rows():
    """Rows as parts of a fused projection's output; only layer 1 changes."""
    t = torch()
    f = Filled(90, [50, 20], L=3, H=2)
    wide = t.zeros((2, 50, 8, D), dtype=f.x.dtype, device="cuda")
    wide[:, :, 4:6], wide[:, :, 6:8] = f.x[0], f.x[1]
    f.put(wide[:, :, 4:6], wide[:, :, 6:8], 50, f.lengths, [0, 0], layer=1)
    f.check(layer=1)
    for l in (0, 2):
        assert bool((f.pay[l] == FILL).all()) and bool((f.meta[l] == 5.0).all()) and not f.tail[l].any()


def test_positions_outside_write_nothing():
    f = Filled(95, [40, 40, 40])
    f.put(f.x[0, :, :4], f.x[1, :, :4], 4, [0, 1 << 30, -3], [5, f.cap, -9])
    assert bool((f.pay == FILL).all()) and bool((f.meta == 5.0).all()) and not f.tail.any()
    # beyond the capacity: the rows that fit
    f = Filled(96, [64], cap=64)
    f.put(f.x[0], f.x[1], 64, [1 << 30], [0])
    f.check()


def test_captured_append():
    t = torch()
    f = Filled(97, [48, 30], H=1)
    k, v = t.zeros((2, 1, 1, D), dtype=f.x.dtype, device="cuda"), t.zeros((2, 1, 1, D), dtype=f.x.dtype, device="cuda")
    ln = t.zeros(2, dtype=t.int32, device="cuda")

    def call():
        cg.cg_append(f.shape, f.gauge, f.codec, 0, 1, k, v, f.tail, f.pay, f.meta, ln)

    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        call()
    for i in range(48):
        n = [i + 1, min(i + 1, 30)]
        ln.copy_(t.tensor(n, dtype=t.int32))
        for b in range(2):
            k[b, 0], v[b, 0] = f.x[0, b, n[b] - 1], f.x[1, b, n[b] - 1]
        g.replay()
    t.cuda.synchronize()
    f.check()


@pytest.mark.parametrize("block", [16, 32])
def test_new_rows_are_the_last(block):
    """Rows of the last block are written again; lengths past the new rows' end bring none back."""
    f = Filled(99 + block, [41, 35], block=block)
    t = torch()
    old = t.randn(f.x.shape, device="cuda").to(f.x.dtype)
    f.put(old[0], old[1], 41, [41, 41], [0, 0])
    f.put(f.x[0, :, :32], f.x[1, :, :32], 32, [32, 32], [0, 0])
    new = t.stack([f.x[:, 0, 32:35], f.x[:, 1, 32:35]], 1)     # positions 32 .. 34 of both
    f.put(new[0], new[1], 3, [41, 39], [32, 32])
    pay, meta = f.pay.clone(), f.meta.clone()
    f.put(new[0], new[1], 3, [35, 35], [32, 32])
    assert t.equal(pay, f.pay) and t.equal(meta, f.meta)
    f.pay[:, :, :, :, 35:] = FILL
    f.meta[:, :, :, :, 35 // block + 1:] = 5.0
    f.check(lengths=[35, 35])


def test_single_rows_that_lie_differently():
    """One row of one sequence: k and v may come from tensors of unlike strides."""
    t = torch()
    f, z = (Filled(120, [40]) for _ in range(2))
    f.put(f.x[0], f.x[1], 40, [40])
    wide = t.zeros((1, 40, 6, D), dtype=z.x.dtype, device="cuda")
    wide[:, :, 4:6] = z.x[1]
    for i in range(40):
        z.put(z.x[0, :, i:i + 1].contiguous(), wide[:, i:i + 1, 4:6], 1, [i + 1])
    z.check()
    assert t.equal(f.tail[:, :, :, :, :8], z.tail[:, :, :, :, :8]) and t.equal(f.pay, z.pay)
