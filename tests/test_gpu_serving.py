"""The serving cache as a decoder uses it: ragged prompts, single tokens, drafted
tokens, evictions, every layer, against the same run on plain arrays (fp64
attention over codes that the oracle quantized)."""
import numpy as np
import pytest

import oracle
from fixed_rate_compression_amd import binding as cg
from fixed_rate_compression_amd.serving import ServingCache
from gpu_util import D, gauges_for, to_dev, to_host

pytestmark = pytest.mark.gpu


def torch():
    return __import__("torch")


class Plain:
    """The cache on the host: per (layer, kind, sequence, head) a list of blocks (codes, range), the last one's raw rows."""

    def __init__(self, L, B, H, cap, block, G, g):
        self.dims, self.block, self.G, self.g, self.cap = (L, B, H), block, G, g, cap
        self.len = [0] * B
        self.blocks = {}
        self.raw = {}
        self.mass = np.zeros((L, B, H, cap // block))
        self.mass_tol = np.zeros_like(self.mass)

    def append(self, l, kind, b, h, rows):
        at = (l, kind, b, h)
        bl, raw = self.blocks.setdefault(at, []), self.raw.get(at)
        if raw is not None and len(raw) < self.block and bl:
            bl.pop()
            rows = np.concatenate([raw, rows], 0)
        for lo in range(0, len(rows), self.block):
            part = rows[lo:lo + self.block]
            xg = oracle.gauge_forward(oracle.to_f32(part), None if self.G is None else self.G[l, kind, h], self.g)
            codes, m = oracle.serving.quantize(xg, self.block)
            bl.append((codes, m[0]))
            self.raw[at] = part

    def arrays(self, l):
        L, B, H = self.dims
        pay = np.zeros((1, 2, B, H, self.cap, D), np.uint8)
        meta = np.zeros((1, 2, B, H, self.cap // self.block, 2), np.float32)
        for kind in (0, 1):
            for b in range(B):
                for h in range(H):
                    for i, (c, m) in enumerate(self.blocks.get((l, kind, b, h), [])):
                        pay[0, kind, b, h, i * self.block:i * self.block + len(c)] = c
                        meta[0, kind, b, h, i] = m
        return pay, meta

    def evict(self, budget, sink, recent, mass):
        L, B, H = self.dims
        kept = np.full((L, B, H, budget), -1, np.int32)
        for b in range(B):
            n = -(-self.len[b] // self.block)
            for l in range(L):
                for h in range(H):
                    keep = oracle.serving.keep_blocks(mass[l, b, h], self.len[b], self.block, budget, sink, recent)
                    kept[l, b, h, :len(keep)] = keep
                    for kind in (0, 1):
                        bl = self.blocks.get((l, kind, b, h), [])
                        self.blocks[(l, kind, b, h)] = [bl[i] for i in keep]
                    for x in (self.mass, self.mass_tol):
                        v = np.zeros(self.cap // self.block)
                        v[:len(keep)] = x[l, b, h][keep]
                        x[l, b, h] = v
            if n > budget:
                self.len[b] -= (n - budget) * self.block
        return kept


@pytest.mark.parametrize("bf16,g,block,R", [(True, 16, 16, 4), (False, 32, 32, 1), (True, 128, 64, 3), (True, 0, 32, 8)])
def test_a_run_of_prompts_tokens_and_evictions(bf16, g, block, R):
    t = torch()
    L, B, H, cap = 2, 3, 2, 320
    rng = np.random.default_rng(7 + g)
    G = gauges_for(8 + g, L, 2, H, g)
    gauge = cg.make_gauge(g, to_dev(np.ascontiguousarray(G)) if g else None)
    cache = ServingCache(L, B, H, H * R, cap, gauge, block, cg.CG_DTYPE_BF16 if bf16 else cg.CG_DTYPE_F32, with_mass=True)
    ref = Plain(L, B, H, cap, block, G, g)
    sc = np.float64(np.float32(D ** -0.5))

    def step(n, valid=None):
        starts = list(ref.len)
        cnt = [n] * B if valid is None else valid
        cache.begin(n, None if valid is None else t.tensor(valid, dtype=t.int32, device="cuda"))
        for b in range(B):
            ref.len[b] += cnt[b]
        for l in range(L):
            x = rng.standard_normal((2, B, n, H, D)).astype(np.float32) * np.exp(0.5 * rng.standard_normal((2, 1, 1, H, D)))
            x = oracle.f32_to_bf16(x.astype(np.float32)) if bf16 else x.astype(np.float32)
            q = rng.standard_normal((B, n, H * R, D)).astype(np.float32)
            q = oracle.f32_to_bf16(q) if bf16 else q
            cache.append(l, to_dev(x[0]), to_dev(x[1]))
            for kind in (0, 1):
                for b in range(B):
                    for h in range(H):
                        if cnt[b]:
                            ref.append(l, kind, b, h, x[kind, b, :cnt[b], h])
            out = cache.attend(l, to_dev(q))
            pay, meta = ref.arrays(l)
            r = oracle.serving.attend(oracle.to_f32(q).astype(np.float64), pay, meta, None if G is None else G[l:l + 1], 0,
                                      block, sc, True, ref.len, starts, fp32=not bf16)
            o = oracle.to_f32(to_host(out)).astype(np.float64)
            half = 2.0 ** -8 if bf16 else 2.0 ** -24
            assert np.all(np.abs(o - r["out"]) <= r["out_tol"] + half * (np.abs(r["out"]) + r["out_tol"])), (n, l)
            ref.mass[l] += r["mass"]
            ref.mass_tol[l] += r["mass_tol"] + 2.0 ** -22 * ref.mass[l]
        assert cache.lengths.tolist() == ref.len
        assert np.all(np.abs(to_host(cache.mass) - ref.mass) <= ref.mass_tol + 1e-7)

    step(100, [100, 37, 0])        # right-padded prompts, one sequence still empty
    step(20, [20, 20, 15])
    for _ in range(3):
        step(1)
    step(5)                        # drafted tokens
    mass = to_host(cache.mass)     # the choice turns on the weights as they are
    kept = to_host(cache.evict(5, 1, 2))
    assert np.array_equal(kept, ref.evict(5, 1, 2, mass))
    assert cache.lengths.tolist() == ref.len
    for _ in range(block + 3):     # past the end of the block that was open
        step(1)
    mass = to_host(cache.mass)
    kept = to_host(cache.evict(2, 0, 1))
    assert np.array_equal(kept, ref.evict(2, 0, 1, mass)) and (kept[:, 0] >= 0).all()
    step(33)
    step(1)


def test_a_recorded_step_is_replayed_as_the_cache_grows():
    t = torch()
    L, B, H, R, block, cap = 2, 2, 2, 4, 16, 256
    gauge = cg.make_gauge(16, to_dev(gauges_for(31, L, 2, H, 16)))
    gen = t.Generator("cuda").manual_seed(5)
    caches = [ServingCache(L, B, H, H * R, cap, gauge, block, with_mass=True) for _ in range(2)]
    k, v = (t.zeros((L, B, 1, H, D), dtype=t.bfloat16, device="cuda") for _ in range(2))
    q = t.zeros((L, B, 1, H * R, D), dtype=t.bfloat16, device="cuda")
    outs = [t.zeros((L, B, 1, H * R, D), dtype=t.bfloat16, device="cuda") for _ in range(2)]
    prompt = t.randn((2, L, B, 50, H, D), generator=gen, device="cuda").bfloat16()
    valid = t.tensor([50, 13], dtype=t.int32, device="cuda")
    for c in caches:
        c.begin(50, valid)
        for l in range(L):
            c.append(l, prompt[0, l], prompt[1, l])

    def step(c, o):
        c.begin(1)
        for l in range(L):
            c.append(l, k[l], v[l])
            c.attend(l, q[l], out=o[l])

    def fill():
        for x in (k, v, q):
            x.copy_(t.randn(x.shape, generator=gen, device="cuda"))

    fill()
    for c, o in zip(caches, outs):
        step(c, o)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step(caches[0], outs[0])
    for i in range(40):
        fill()
        graph.replay()
        step(caches[1], outs[1])
        t.cuda.synchronize()
        assert t.equal(outs[0], outs[1]), i
    for a, b in ((caches[0].payload, caches[1].payload), (caches[0].mass, caches[1].mass),
                 (caches[0].lengths, caches[1].lengths)):
        assert t.equal(a, b)


def test_refusals():
    gauge = cg.make_gauge(0)
    with pytest.raises(ValueError):
        ServingCache(1, 1, 1, 1, 100, gauge, 32)
    c = ServingCache(1, 1, 1, 2, 64, gauge, 32)
    with pytest.raises(ValueError):
        c.begin(65)
    with pytest.raises(ValueError):
        c.begin(-1)
    c.begin(64)
    with pytest.raises(ValueError):
        c.begin(1)
    with pytest.raises(ValueError):
        c.evict(1)


def test_an_eviction_ends_the_step():
    """Positions change: rows of the step before are refused, the next step goes on."""
    t = torch()
    c = ServingCache(1, 1, 1, 2, 64, cg.make_gauge(0), 16, with_mass=True)
    k = t.ones((1, 40, 1, D), dtype=t.bfloat16, device="cuda")
    q = t.ones((1, 40, 2, D), dtype=t.bfloat16, device="cuda")
    c.begin(40)
    c.append(0, k, k)
    c.attend(0, q)
    c.evict(2)
    assert c.lengths.tolist() == [24]
    with pytest.raises(ValueError):
        c.append(0, k, k)
    with pytest.raises(ValueError):
        c.attend(0, q)
    with pytest.raises(ValueError):
        c.begin(40)                # the host's bound: a sequence of 32 rows would have kept them all
    c.begin(32)
    c.append(0, k[:, :32], k[:, :32])
    assert bool((c.attend(0, q[:, :32]) == 1).all()) and c.lengths.tolist() == [56]


def test_workspaces_do_not_pile_up():
    """Prompts of many lengths share one workspace that grows; an older one outlives what recorded it."""
    t = torch()
    c = ServingCache(1, 2, 2, 8, 4096, cg.make_gauge(0), 32, with_mass=True)
    k = t.randn((2, 40, 2, D), device="cuda").bfloat16()
    q = t.randn((2, 40, 8, D), device="cuda").bfloat16()
    outs = []
    for n in list(range(40, 0, -1)) + list(range(1, 41)):
        c.begin(n)
        c.append(0, k[:, :n], k[:, :n])
        outs.append(c.attend(0, q[:, :n]))
    assert len(c._work) <= 3
    assert all(bool(t.isfinite(o.float()).all()) for o in outs)


def test_a_refused_step_leaves_the_cache_as_it_was():
    """Counts of valid rows that are not there for every sequence, or are no whole numbers on
    the GPU, are refused before the step begins."""
    t = torch()
    c = ServingCache(1, 3, 1, 2, 64, cg.make_gauge(0), 32)
    c.begin(20, t.tensor([20, 5, 0], dtype=t.int32, device="cuda"))
    for bad in (t.tensor([4], dtype=t.int32, device="cuda"), t.tensor([1, 2], dtype=t.int32, device="cuda"),
                t.tensor([1, 2, 3], dtype=t.int32), t.tensor([1.0, 2.0, 3.0], device="cuda"), [1, 2, 3]):
        with pytest.raises(ValueError):
            c.begin(40, bad)
        assert (c.n, c.most) == (20, 20) and c.lengths.tolist() == [20, 5, 0] and c.starts.tolist() == [0, 0, 0]
    c.begin(44, t.tensor([44, -3, 90], dtype=t.int64, device="cuda"))
    assert c.lengths.tolist() == [64, 5, 44] and c.starts.tolist() == [20, 5, 0]


def test_a_layers_rows_go_in_once_a_step():
    """Rows put in again after they have passed the end of a block would be encoded beside the
    raw rows of a later one: refused, and the cache is as it was."""
    t = torch()
    c, want = (ServingCache(2, 1, 1, 2, 64, cg.make_gauge(0), 16) for _ in range(2))
    k = t.randn((1, 30, 1, D), device="cuda", generator=t.Generator("cuda").manual_seed(3)).bfloat16()
    for x in (c, want):
        for lo, n in ((0, 10), (10, 20)):
            x.begin(n)
            for layer in range(2):
                x.append(layer, k[:, lo:lo + n], k[:, lo:lo + n])
            if x is c:
                with pytest.raises(ValueError):
                    x.append(1, k[:, lo:lo + n], k[:, lo:lo + n])
    assert t.equal(c.payload, want.payload) and t.equal(c.meta, want.meta) and t.equal(c.tail, want.tail)
    c.begin(1)
    with pytest.raises(ValueError):
        c.append(0, k[:, :2], k[:, :2])      # a refused call has put nothing in
    c.append(0, k[:, :1], k[:, :1])


def test_buffers_are_made_where_the_cache_lies(monkeypatch):
    """Workspaces and results name the cache's GPU, not the current one: a workspace made
    elsewhere by a call that is refused for it would be kept and refused from then on."""
    t = torch()
    c = ServingCache(1, 1, 1, 2, 64, cg.make_gauge(0), 16, with_mass=True)
    k = t.zeros((1, 20, 1, D), dtype=t.bfloat16, device="cuda")
    made, empty = [], t.empty

    def record(*a, **kw):
        made.append(t.device(kw["device"]))
        return empty(*a, **kw)

    monkeypatch.setattr(t, "empty", record)
    c.begin(20)
    c.append(0, k, k)
    c.attend(0, t.zeros((1, 20, 2, D), dtype=t.bfloat16, device="cuda"))
    c.evict(2)
    assert len(made) >= 3 and all(d == c.payload.device for d in made), made      # "cuda" alone is the current one
