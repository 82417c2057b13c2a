"""The 4-bit serving cache as a decoder uses it: heads normed and rotated, ragged prompts,
single and drafted tokens, rows read back, evictions, every layer, against the same run on plain
arrays (fp64 attention over codes that the oracle quantized)."""
import numpy as np
import pytest

import oracle
from fixed_rate_compression_amd import binding as cg
from fixed_rate_compression_amd.serving import ServingCache
from gpu_util import D, check_decoded, gauges_for, to_dev, to_host
from serve4_util import GROUP

pytestmark = pytest.mark.gpu


def torch():
    return __import__("torch")


class Plain4:
    """The cache on the host: per (layer, kind, sequence, head) the raw rows of every block, oldest first."""

    def __init__(self, L, B, H, cap, G, g):
        self.dims, self.G, self.g, self.cap = (L, B, H), G, g, cap
        self.len = [0] * B
        self.blocks = {}
        self.mass, self.mass_tol = np.zeros((L, B, H, cap // GROUP)), np.zeros((L, B, H, cap // GROUP))

    def append(self, l, kind, b, h, rows):
        bl = self.blocks.setdefault((l, kind, b, h), [])
        if bl and len(bl[-1]) < GROUP:
            rows = np.concatenate([bl.pop(), rows], 0)
        bl.extend(rows[lo:lo + GROUP] for lo in range(0, len(rows), GROUP))

    def arrays(self, l):
        L, B, H = self.dims
        pay = np.zeros((1, 2, B, H, self.cap, D // 2), np.uint8)
        meta = np.zeros((1, 2, B, H, 4 * self.cap, 2), np.float32)
        for kind in (0, 1):
            for b in range(B):
                for h in range(H):
                    for i, raw in enumerate(self.blocks.get((l, kind, b, h), [])):
                        xg = oracle.gauge_forward(oracle.to_f32(raw), None if self.G is None else self.G[l, kind, h], self.g)
                        c, m = oracle.serving4.quantize(xg, kind)
                        pay[0, kind, b, h, i * GROUP:i * GROUP + len(c)] = c
                        meta[0, kind, b, h, i * D:i * D + len(m)] = m
        return pay, meta

    def evict(self, budget, sink, recent, mass):
        L, B, H = self.dims
        kept = np.full((L, B, H, budget), -1, np.int32)
        for b in range(B):
            n = -(-self.len[b] // GROUP)
            for l in range(L):
                for h in range(H):
                    keep = oracle.serving.keep_blocks(mass[l, b, h], self.len[b], GROUP, budget, sink, recent)
                    kept[l, b, h, :len(keep)] = keep
                    for kind in (0, 1):
                        bl = self.blocks.get((l, kind, b, h), [])
                        self.blocks[(l, kind, b, h)] = [bl[i] for i in keep]
                    for x in (self.mass, self.mass_tol):
                        v = np.zeros(self.cap // GROUP)
                        v[:len(keep)] = x[l, b, h][keep]
                        x[l, b, h] = v
            if n > budget:
                self.len[b] -= (n - budget) * GROUP
        return kept


@pytest.mark.parametrize("bf16,g,R", [(True, 16, 4), (False, 32, 1), (True, 128, 3), (True, 0, 8)])
def test_a_run_of_prompts_tokens_reads_and_evictions(bf16, g, R):
    t = torch()
    L, B, H, cap = 2, 3, 2, 320
    rng = np.random.default_rng(7 + g)
    G = gauges_for(8 + g, L, 2, H, g)
    gauge = cg.make_gauge(g, to_dev(np.ascontiguousarray(G)) if g else None)
    cache = ServingCache(L, B, H, H * R, cap, gauge, GROUP, cg.CG_DTYPE_BF16 if bf16 else cg.CG_DTYPE_F32, with_mass=True,
                         bits=4)
    ref = Plain4(L, B, H, cap, G, g)
    sc = np.float64(np.float32(D ** -0.5))
    freq = (1e4 ** (-np.arange(64) / 64)).astype(np.float32)
    w = (1 + 0.2 * rng.standard_normal((2, D))).astype(np.float32)
    rotary = cg.make_rotary(to_dev(freq), q_weight=to_dev(w[0]), k_weight=to_dev(w[1]))
    half = 2.0 ** -8 if bf16 else 2.0 ** -24

    def rounds_to(x, want, tol):
        assert np.all(np.abs(oracle.to_f32(x).astype(np.float64) - want) <= tol + half * (np.abs(want) + tol))

    def step(n, valid=None):
        starts = list(ref.len)
        cnt = [n] * B if valid is None else valid
        cache.begin(n, None if valid is None else t.tensor(valid, dtype=t.int32, device="cuda"))
        for b in range(B):
            ref.len[b] += cnt[b]
        there = np.arange(n)[None] < np.array(cnt)[:, None]
        pos = (np.array(starts)[:, None] + np.arange(n))[None]
        for l in range(L):
            # a fused projection's rows: queries and keys turned where they lie
            x = rng.standard_normal((B, n, (R + 2) * H, D)).astype(np.float32) * np.exp(0.5 * rng.standard_normal(((R + 2) * H, D)))
            x = oracle.f32_to_bf16(x.astype(np.float32)) if bf16 else x.astype(np.float32)
            qkv = to_dev(x)
            q, k, v = qkv[:, :, :R * H], qkv[:, :, R * H:(R + 1) * H], qkv[:, :, (R + 1) * H:]
            cache.rotate(q, k, rotary)
            for y, s, ww in ((q, slice(0, R * H), w[0]), (k, slice(R * H, (R + 1) * H), w[1])):
                want, tol = oracle.serving4.rotate(oracle.to_f32(x[:, :, s]), ww, 1e-6, freq, pos, False)
                rounds_to(to_host(y)[there], want[there], tol[there])
            qh, kh, vh = to_host(q), to_host(k), to_host(v)     # as rotated
            cache.append(l, k, v)
            for kind, y in ((0, kh), (1, vh)):
                for b in range(B):
                    for h in range(H):
                        if cnt[b]:
                            ref.append(l, kind, b, h, y[b, :cnt[b], h])
            out = cache.attend(l, q)
            pay, meta = ref.arrays(l)
            Gl = None if G is None else G[l:l + 1]
            r = oracle.serving4.attend(oracle.to_f32(qh).astype(np.float64), pay, meta, Gl, 0, sc, True, ref.len, starts,
                                       fp32=not bf16)
            rounds_to(to_host(out), r["out"], r["out_tol"])
            ref.mass[l] += r["mass"]
            ref.mass_tol[l] += r["mass_tol"] + 2.0 ** -22 * ref.mass[l]
            back = cache.read(l, 40)
            for kind in (0, 1):
                y = to_host(back[kind])
                for b in range(B):
                    lo = max(ref.len[b] - 40, 0)
                    m = ref.len[b] - lo
                    assert not y[b, :40 - m].any()
                    for h in range(H):
                        if not m or (g == 128 and bf16):
                            continue
                        at = (0, kind, b, h)
                        tt, c = np.arange(lo, ref.len[b])[:, None], np.arange(D)[None]
                        mm = meta[at][tt // GROUP * D + c if kind == 0 else tt * 4 + c // GROUP]
                        yg = mm[..., 0] + mm[..., 1] * oracle.serving4.codes(pay[at][lo:ref.len[b]]).astype(np.float32)
                        check_decoded(np.ascontiguousarray(y[b, 40 - m:, h]), yg, None if G is None else G[l, kind, h], g)
        assert cache.lengths.tolist() == ref.len
        assert np.all(np.abs(to_host(cache.mass) - ref.mass) <= ref.mass_tol + 1e-7)

    step(100, [100, 37, 0])        # right-padded prompts, one sequence still empty
    step(20, [20, 20, 15])
    for _ in range(3):
        step(1)
    step(5)                        # drafted tokens
    mass = to_host(cache.mass)     # the choice turns on the weights as they are
    kept = to_host(cache.evict(3, 1, 1))
    assert np.array_equal(kept, ref.evict(3, 1, 1, mass))
    assert cache.lengths.tolist() == ref.len
    for _ in range(GROUP + 3):     # past the end of the block that was open
        step(1)
    mass = to_host(cache.mass)
    kept = to_host(cache.evict(2, 0, 1))
    assert np.array_equal(kept, ref.evict(2, 0, 1, mass)) and (kept[:, 0] >= 0).all()
    step(33)
    step(1)


def test_a_recorded_step_is_replayed_as_the_cache_grows():
    """Rotation, append and attention of every layer in one graph; two caches share the recorded arrays' sizes, not
    their workspaces."""
    t = torch()
    L, B, H, R, cap = 2, 2, 2, 4, 256
    gauge = cg.make_gauge(16, to_dev(gauges_for(31, L, 2, H, 16)))
    rotary = cg.make_rotary(to_dev((1e4 ** (-np.arange(32) / 32)).astype(np.float32)))
    gen = t.Generator("cuda").manual_seed(5)
    caches = [ServingCache(L, B, H, H * R, cap, gauge, with_mass=True, bits=4) for _ in range(2)]
    rows = t.zeros((L, B, 1, (R + 2) * H, D), dtype=t.bfloat16, device="cuda")
    turned = [t.zeros_like(rows) for _ in range(2)]
    outs = [t.zeros((L, B, 1, H * R, D), dtype=t.bfloat16, device="cuda") for _ in range(2)]
    prompt = t.randn((2, L, B, 50, H, D), generator=gen, device="cuda").bfloat16()
    valid = t.tensor([50, 13], dtype=t.int32, device="cuda")
    for c in caches:
        c.begin(50, valid)
        for l in range(L):
            c.append(l, prompt[0, l], prompt[1, l])

    def step(c, y, o):
        c.begin(1)
        y.copy_(rows)
        for l in range(L):
            q, k, v = y[l][:, :, :R * H], y[l][:, :, R * H:(R + 1) * H], y[l][:, :, (R + 1) * H:]
            c.rotate(q, k, rotary)
            c.append(l, k, v)
            c.attend(l, q, out=o[l])

    def fill():
        rows.copy_(t.randn(rows.shape, generator=gen, device="cuda"))

    fill()
    for c, y, o in zip(caches, turned, outs):
        step(c, y, o)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step(caches[0], turned[0], outs[0])
    for i in range(40):
        fill()
        graph.replay()
        step(caches[1], turned[1], outs[1])
        t.cuda.synchronize()
        assert t.equal(outs[0], outs[1]) and t.equal(turned[0], turned[1]), i
    for a, b in ((caches[0].payload, caches[1].payload), (caches[0].meta, caches[1].meta), (caches[0].mass, caches[1].mass),
                 (caches[0].lengths, caches[1].lengths)):
        assert t.equal(a, b)


def test_from_8_bits_to_4():
    """A cache's rows move to another format through cg_read and cg_append."""
    t = torch()
    L, B, H = 2, 2, 2
    gauge = cg.make_gauge(8, to_dev(gauges_for(41, L, 2, H, 8)))
    a, b = (ServingCache(L, B, H, H, 128, gauge, bits=x) for x in (8, 4))
    x = t.randn((2, B, 70, H, D), device="cuda").bfloat16()
    valid = t.tensor([70, 33], dtype=t.int32, device="cuda")
    zero = t.zeros(B, dtype=t.int32, device="cuda")
    a.begin(70, valid)
    b.begin(70, valid)
    for l in range(L):
        a.append(l, x[0], x[1])
        k, v = a.read(l, 70, zero)
        b.append(l, k, v)
        k4, v4 = b.read(l, 70, zero)
        for y, z in ((k, k4), (v, v4)):
            assert not z[1, 33:].any()
            # a 4-bit value is off by half a step, 1 / 30 of its range of 32 (at most about 9 here)
            assert float((y.float() - z.float()).abs().max()) < 1.0 and not t.equal(y, z)


def test_refusals():
    gauge = cg.make_gauge(0)
    with pytest.raises(ValueError):
        ServingCache(1, 1, 1, 1, 128, gauge, bits=2)
    with pytest.raises(ValueError):
        ServingCache(1, 1, 1, 1, 100, gauge, bits=4)
    with pytest.raises(cg.CodecGaugeError):
        ServingCache(1, 1, 1, 1, 128, gauge, block_tokens=16, bits=4)
