"""Positions of a serving cache's rows: every row that a sequence has had counts, also after evictions, so that new
queries and keys are turned against the kept keys as they would be without one."""
import numpy as np
import pytest

import oracle
from fixed_rate_compression_amd import binding as cg
from fixed_rate_compression_amd.serving import ServingCache
from gpu_util import D, gauges_for, to_dev, to_host
from serve4_util import GROUP
from test_gpu_serving4 import Plain4

pytestmark = pytest.mark.gpu


def torch():
    return __import__("torch")


@pytest.mark.parametrize("bf16,g,R", [(True, 16, 4), (False, 32, 1), (True, 128, 3), (True, 0, 8)])
def test_a_run_of_prompts_tokens_and_evictions(bf16, g, R):
    """The 4-bit cache, layer by layer, against plain arrays and positions that the test counts for itself."""
    t = torch()
    L, B, H, cap = 2, 3, 2, 320
    rng = np.random.default_rng(27 + g)
    G = gauges_for(28 + g, L, 2, H, g)
    cache = ServingCache(L, B, H, H * R, cap, cg.make_gauge(g, to_dev(np.ascontiguousarray(G)) if g else None), GROUP,
                         cg.CG_DTYPE_BF16 if bf16 else cg.CG_DTYPE_F32, with_mass=True, bits=4)
    ref, seen = Plain4(L, B, H, cap, G, g), np.zeros(B, np.int64)
    freq = (1e4 ** (-np.arange(64) / 64)).astype(np.float32)
    w = (1 + 0.2 * rng.standard_normal((2, D))).astype(np.float32)
    rotary = cg.make_rotary(to_dev(freq), q_weight=to_dev(w[0]), k_weight=to_dev(w[1]))
    half = 2.0 ** -8 if bf16 else 2.0 ** -24

    def rounds_to(x, want, tol):
        assert np.all(np.abs(oracle.to_f32(x).astype(np.float64) - want) <= tol + half * (np.abs(want) + tol))

    def step(n, valid=None):
        starts, cnt = list(ref.len), np.array([n] * B if valid is None else valid)
        cache.begin(n, None if valid is None else t.tensor(valid, dtype=t.int32, device="cuda"))
        for b in range(B):
            ref.len[b] += int(cnt[b])
        there = np.arange(n)[None] < cnt[:, None]
        pos = (seen[:, None] + np.arange(n))[None]
        seen[:] += cnt
        for l in range(L):
            x = rng.standard_normal((B, n, (R + 2) * H, D)).astype(np.float32)
            x = oracle.f32_to_bf16(x) if bf16 else x
            qkv = to_dev(x)
            q, k, v = qkv[:, :, :R * H], qkv[:, :, R * H:(R + 1) * H], qkv[:, :, (R + 1) * H:]
            cache.rotate(q, k, rotary)
            for y, s, ww in ((q, slice(0, R * H), w[0]), (k, slice(R * H, (R + 1) * H), w[1])):
                want, tol = oracle.serving4.rotate(oracle.to_f32(x[:, :, s]), ww, 1e-6, freq, pos, False)
                rounds_to(to_host(y)[there], want[there], tol[there])
                assert np.array_equal(to_host(y)[~there], x[:, :, s][~there])
            qh, kh, vh = to_host(q), to_host(k), to_host(v)
            cache.append(l, k, v)
            for kind, y in ((0, kh), (1, vh)):
                for b in range(B):
                    for h in range(H):
                        if cnt[b]:
                            ref.append(l, kind, b, h, y[b, :cnt[b], h])
            out = cache.attend(l, q)
            pay, meta = ref.arrays(l)
            r = oracle.serving4.attend(oracle.to_f32(qh).astype(np.float64), pay, meta, None if G is None else G[l:l + 1], 0,
                                       np.float64(np.float32(D ** -0.5)), True, ref.len, starts, fp32=not bf16)
            rounds_to(to_host(out), r["out"], r["out_tol"])
        assert cache.lengths.tolist() == ref.len

    def evict(*how):
        mass = to_host(cache.mass)
        assert np.array_equal(to_host(cache.evict(*how)), ref.evict(*how, mass))
        assert cache.lengths.tolist() == ref.len and (cache.gone + cache.lengths).tolist() == seen.tolist()

    step(100, [100, 37, 0])
    step(20, [20, 20, 15])
    step(1)
    evict(3, 1, 1)
    assert cache.gone.tolist() == [32, 0, 0]
    for _ in range(4):
        step(1)
    step(40, [40, 3, 0])
    evict(2, 0, 1)
    evict(1, 0, 1)                 # twice, with no step between
    step(33)
    step(1)


@pytest.mark.parametrize("bits", [4, 8])
def test_weights_of_the_kept_keys_are_those_without_an_eviction(bits):
    """A query after an eviction gives each kept key the score that it gives it in a cache that keeps all."""
    t = torch()
    H, R, T, n = 1, 2, 256, 3
    gen = t.Generator("cuda").manual_seed(40)
    rotary = cg.make_rotary(to_dev((1e4 ** (-np.arange(64) / 64)).astype(np.float32)))
    caches = [ServingCache(1, 1, H, R, 320, cg.make_gauge(0), GROUP, cg.CG_DTYPE_F32, with_mass=True, bits=bits) for _ in range(2)]
    rows = [t.randn((1, m, R + 2 * H, D), generator=gen, device="cuda") for m in (T, n)]
    res = []
    for c, drop in zip(caches, (False, True)):
        for i, x in enumerate(rows):
            x = x.clone()
            q, k, v = x[:, :, :R], x[:, :, R:R + H], x[:, :, R + H:]
            c.begin(x.shape[1])
            c.rotate(q, k, rotary)
            c.append(0, k, v)
            lse = t.empty((1, x.shape[1], R), device="cuda")
            out = c.attend(0, q, lse=lse)
            if i == 0 and drop:
                kept = c.evict(4, 1, 1)[0, 0, 0].tolist()
        res.append((q, k, v, out, lse))
    for x, y in zip(res[0][:3], res[1][:3]):
        assert t.equal(x, y)                                  # turned alike
    # the kept keys as both caches hold them, and the plain attention of the query over them
    at = [32 * b + i for b in kept for i in range(32)] + list(range(T, T + n))
    k, v = (x[0, :, 0].double().cpu() for x in caches[0].read(0, T + n, t.zeros(1, dtype=t.int32, device="cuda")))
    k2, v2 = (x[0, :, 0].double().cpu() for x in caches[1].read(0, len(at), t.zeros(1, dtype=t.int32, device="cuda")))
    assert t.equal(k[at], k2) and t.equal(v[at], v2)
    q = res[1][0][0].double().cpu()
    for i in range(n):
        vis = len(at) - n + i + 1
        s = t.matmul(q[i], k2[:vis].t().contiguous()) * np.float64(np.float32(D ** -0.5))
        # scores of a few units: 2^-17 of a value is ample above fp32's and the codes' 2^-20
        assert float((res[1][3][0, i].double().cpu() - t.matmul(t.softmax(s, -1), v2[:vis])).abs().max()) < 2.0 ** -15
        assert float((res[1][4][0, i].double().cpu() - t.logsumexp(s, -1)).abs().max()) < 2.0 ** -15


@pytest.mark.parametrize("bits", [4, 8])
def test_a_recorded_step_counts_on_after_evictions(bits):
    t = torch()
    L, B, H, R, cap = 2, 2, 2, 4, 256
    gauge = cg.make_gauge(16, to_dev(gauges_for(51, L, 2, H, 16)))
    freq = (1e4 ** (-np.arange(64) / 64)).astype(np.float32)
    rotary = cg.make_rotary(to_dev(freq))
    gen = t.Generator("cuda").manual_seed(52)
    c = ServingCache(L, B, H, H * R, cap, gauge, with_mass=True, bits=bits)
    rows = t.zeros((L, B, 1, (R + 2) * H, D), dtype=t.bfloat16, device="cuda")
    turned, outs = t.zeros_like(rows), t.zeros((L, B, 1, H * R, D), dtype=t.bfloat16, device="cuda")
    seen = np.array([150, 70])
    prompt = t.randn((2, L, B, 150, H, D), generator=gen, device="cuda").bfloat16()
    c.begin(150, t.tensor(seen, dtype=t.int32, device="cuda"))
    for l in range(L):
        c.append(l, prompt[0, l], prompt[1, l])

    def step():
        c.begin(1)
        turned.copy_(rows)
        for l in range(L):
            q, k, v = turned[l].split((R * H, H, H), 2)
            c.rotate(q, k, rotary)
            c.append(l, k, v)
            c.attend(l, q, out=outs[l])

    def check():
        for l in range(L):
            want, tol = oracle.serving4.rotate(oracle.to_f32(to_host(rows[l])), None, 0.0, freq, seen[None, :, None], False)
            got = oracle.to_f32(to_host(turned[l])).astype(np.float64)[:, :, :(R + 1) * H]
            want, tol = want[:, :, :(R + 1) * H], tol[:, :, :(R + 1) * H]
            assert np.all(np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol))

    step()
    check()
    seen += 1
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step()
    for i in range(12):
        rows.copy_(t.randn(rows.shape, generator=gen, device="cuda"))
        graph.replay()
        t.cuda.synchronize()
        check()
        seen += 1
        assert (c.gone + c.lengths).tolist() == seen.tolist()
        if i in (3, 7):
            c.evict(4 if i == 3 else 2, 1, 1)
    assert c.gone.tolist() != [0, 0]


def test_rotation_belongs_to_a_step():
    """Before the first step, after an eviction and for other numbers of rows it is refused, and nothing is turned."""
    t = torch()
    c = ServingCache(1, 1, 1, 2, 128, cg.make_gauge(0), with_mass=True, bits=4)
    rotary = cg.make_rotary(to_dev(np.ones(64, np.float32)))
    x = t.ones((1, 40, 3, D), dtype=t.bfloat16, device="cuda")
    q, k, v = x[:, :, :2], x[:, :, 2:], t.ones((1, 40, 1, D), dtype=t.bfloat16, device="cuda")

    def refused(n):
        for a, b in ((q[:, :n], k[:, :n]), (q[:, :n], None), (None, k[:, :n])):
            with pytest.raises(ValueError):
                c.rotate(a, b, rotary)
        with pytest.raises(ValueError):
            c.rotate(q[:, :n], k[:, :n], rotary, positions=t.zeros((1, 1, n), dtype=t.int32, device="cuda"))
        assert bool((x == 1).all())

    refused(1)
    with pytest.raises(ValueError):
        c.rotate(None, None, rotary)
    c.begin(40)
    refused(39)
    c.append(0, k.contiguous(), v)
    c.attend(0, q)
    c.evict(1, 0, 1)
    refused(40)
    c.begin(1)
    refused(40)
    y = c.rotate(q[:, :1], None, rotary, q_out=t.empty_like(q[:, :1]))
    assert y[1] is None and not bool((y[0] == 1).any())
