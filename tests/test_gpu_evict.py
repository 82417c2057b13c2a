"""cg_evict on the GPU against a plain sort: kept blocks, moved bytes, weights
and lengths, into another cache and in place."""
import numpy as np
import pytest

import oracle
from fixed_rate_compression_amd import binding as cg
from gpu_util import D, to_dev, to_host
from serve_util import random_cache

pytestmark = pytest.mark.gpu


def torch():
    return __import__("torch")


def run(seed, L, B, H, cap, block, budget, sink, recent, lengths, mass=None, out_cap=None, in_place=False):
    t = torch()
    rng = np.random.default_rng(seed)
    nb = cap // block
    pay, meta = random_cache(rng, L, B, H, cap, block)
    if mass is None:
        mass = rng.exponential(1.0, (L, B, H, nb)).astype(np.float32)
    shape = cg.make_shape(L, 2, B, H, cap, cap, D)
    codec = cg.make_codec(cg.CG_BACKEND_BLOCK_UNIFORM, 8, block)
    oc = cap if in_place else out_cap or budget * block
    out_shape = cg.make_shape(L, 2, B, H, oc, oc, D)
    pd, md, wd = to_dev(pay), to_dev(meta), to_dev(mass)
    ln = t.tensor(lengths, dtype=t.int32, device="cuda") if lengths else None
    if in_place:
        po, mo, wo, lo = pd, md, wd, ln
        base_p, base_m = pay, meta
    else:
        po = t.full((L, 2, B, H, oc, D), 9, dtype=t.uint8, device="cuda")
        mo = t.full((L, 2, B, H, oc // block, 2), 9.0, device="cuda")
        wo = t.full((L, B, H, oc // block), 9.0, device="cuda")
        lo = t.full((B,), 9, dtype=t.int32, device="cuda")
        base_p, base_m = to_host(po).copy(), to_host(mo).copy()
    kept = t.full((L, B, H, budget), 9, dtype=t.int32, device="cuda")
    cg.cg_evict(shape, codec, budget, sink, recent, wd, pd, md, out_shape, po, mo, wo, kept, lo, ln)
    t.cuda.synchronize()
    got_p, got_m, got_w, got_k, got_l = (to_host(x) for x in (po, mo, wo, kept, lo))
    for b in range(B):
        T = min(max(lengths[b], 0), cap) if lengths else cap
        n = -(-T // block)
        assert got_l[b] == (T - (n - budget) * block if n > budget else T), b
        for l in range(L):
            for h in range(H):
                keep = oracle.serving.keep_blocks(mass[l, b, h], T, block, budget, sink, recent)
                k = len(keep)
                at = (l, b, h)
                assert got_k[at].tolist() == keep + [-1] * (budget - k), at
                assert np.array_equal(got_w[at][:k], mass[at][keep], equal_nan=True) and not got_w[at][k:].any(), at
                for kind in (0, 1):
                    f = (l, kind, b, h)
                    src = pay[f].reshape(nb, block * D)
                    dst = got_p[f].reshape(-1, block * D)
                    assert np.array_equal(dst[:k], src[keep]), f
                    assert np.array_equal(got_m[f][:k], meta[f][keep]), f
                    assert np.array_equal(dst[k:], base_p[f].reshape(-1, block * D)[k:]), f
                    assert np.array_equal(got_m[f][k:], base_m[f][k:]), f


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("block", [16, 32, 64])
@pytest.mark.parametrize("nb,budget,sink,recent", [(40, 13, 2, 3), (7, 1, 0, 1), (9, 9, 1, 1), (5, 30, 4, 4), (130, 128, 0, 2),
                                                  (2100, 700, 1, 5), (33, 6, 2, 4)])
def test_against_a_sort(block, nb, budget, sink, recent, in_place):
    cap = nb * block
    if in_place and budget > nb:
        cap = budget * block
    big = nb > 1000
    run(nb + block, 1 if big else 2, 2, 1 if big else 2, cap, block, budget, sink, recent,
        [nb * block, max(1, nb * block // 2 - 5)], in_place=in_place)


def test_lengths_at_their_ends():
    run(1, 1, 5, 1, 320, 32, 4, 1, 2, [0, 1, 320, 129, 128])
    run(2, 1, 3, 1, 320, 32, 4, 1, 2, [1 << 30, -4, 33])
    run(3, 2, 1, 3, 320, 32, 4, 1, 2, None, out_cap=640)


@pytest.mark.parametrize("in_place", [False, True])
def test_ties_signs_and_nan(in_place):
    rng = np.random.default_rng(4)
    m = rng.integers(-2, 3, (1, 2, 2, 300)).astype(np.float32)
    m[0, 0, 0, ::7] = -0.0
    m[0, 1, 0, ::5] = np.nan
    m[0, 1, 1, ::3] = np.inf
    m[0, 1, 1, 1::3] = -np.inf
    run(5, 1, 2, 2, 300 * 16, 16, 90, 1, 2, [300 * 16, 300 * 16 - 9], mass=m, in_place=in_place)
    run(6, 1, 1, 1, 300 * 16, 16, 50, 0, 1, [4800], mass=np.zeros((1, 1, 1, 300), np.float32), in_place=in_place)
    run(7, 1, 1, 1, 300 * 16, 16, 250, 0, 1, [4800], mass=np.full((1, 1, 1, 300), np.nan, np.float32), in_place=in_place)


def test_neighbouring_weights():
    """Weights that differ in the last bit are told apart."""
    m = (np.float32(1.0).view(np.uint32) + np.random.default_rng(8).permutation(500).astype(np.uint32)).view(np.float32)
    run(9, 1, 1, 1, 500 * 16, 16, 100, 0, 1, [8000], mass=m.reshape(1, 1, 1, 500))


def test_captured_in_place():
    """A recorded eviction replayed: the second finds nothing to evict."""
    t = torch()
    rng = np.random.default_rng(10)
    pay, meta = random_cache(rng, 1, 2, 2, 640, 32)
    mass = rng.exponential(1.0, (1, 2, 2, 20)).astype(np.float32)
    shape, codec = cg.make_shape(1, 2, 2, 2, 640, 640, D), cg.make_codec(cg.CG_BACKEND_BLOCK_UNIFORM, 8, 32)
    pd, md, wd = to_dev(pay), to_dev(meta), to_dev(mass)
    ln = t.tensor([640, 100], dtype=t.int32, device="cuda")
    kept = t.zeros((1, 2, 2, 6), dtype=t.int32, device="cuda")
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        cg.cg_evict(shape, codec, 6, 1, 1, wd, pd, md, shape, pd, md, wd, kept, ln, ln)
    g.replay()
    t.cuda.synchronize()
    assert ln.tolist() == [192, 100]
    k0 = kept.clone()
    p0 = pd.clone()
    for h in range(2):
        assert k0[0, 0, h].tolist() == oracle.serving.keep_blocks(mass[0, 0, h], 640, 32, 6, 1, 1)
    g.replay()
    t.cuda.synchronize()
    assert ln.tolist() == [192, 100] and t.equal(p0, pd)
    assert kept[0, 0, 0].tolist() == list(range(6))


@pytest.mark.parametrize("nb", [1, 64, 255, 256, 257, 1023, 1025, 4096, 4097, 8193, 9001])
@pytest.mark.parametrize("kind", ["ties", "spread", "nan"])
def test_every_number_of_blocks(nb, kind):
    """The forms of the selection, at both sides of their borders."""
    rng = np.random.default_rng(nb)
    m = {"ties": rng.integers(0, 4, (1, 1, 3, nb)), "spread": np.exp(rng.uniform(-80, 80, (1, 1, 3, nb))),
         "nan": np.where(rng.random((1, 1, 3, nb)) < 0.6, np.nan, rng.integers(-2, 2, (1, 1, 3, nb)))}[kind].astype(np.float32)
    budget = max(1, nb // 3)
    run(nb, 1, 1, 3, nb * 16, 16, budget, min(2, budget - 1), 1, [nb * 16 - 7], mass=m, in_place=nb % 2 == 0)
    run(nb + 1, 1, 1, 3, nb * 16, 16, max(1, nb - 1), 0, 1, [nb * 16], mass=m, in_place=nb % 2 == 1)
