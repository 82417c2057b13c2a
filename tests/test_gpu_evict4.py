"""cg_evict on the 4-bit cache against a plain sort: kept blocks, moved codes and ranges,
weights and lengths, into another cache and in place."""
import numpy as np
import pytest

import oracle
from fixed_rate_compression_amd import binding as cg
from gpu_util import D, to_dev, to_host
from serve4_util import GROUP, random_cache4

pytestmark = pytest.mark.gpu


def run(seed, L, B, H, nb, budget, sink, recent, lengths, mass=None, out_nb=None, in_place=False):
    t = __import__("torch")
    rng = np.random.default_rng(seed)
    cap = nb * GROUP
    pay, meta = random_cache4(rng, L, B, H, cap)
    if mass is None:
        mass = rng.exponential(1.0, (L, B, H, nb)).astype(np.float32)
    shape = cg.make_shape(L, 2, B, H, cap, cap, D)
    codec = cg.make_codec(cg.CG_BACKEND_KIVI, 4, GROUP)
    oc = cap if in_place else (out_nb or budget) * GROUP
    out_shape = cg.make_shape(L, 2, B, H, oc, oc, D)
    pd, md, wd = to_dev(pay), to_dev(meta), to_dev(mass)
    ln = t.tensor(lengths, dtype=t.int32, device="cuda") if lengths else None
    if in_place:
        po, mo, wo, lo = pd, md, wd, ln
        base_p, base_m = pay, meta
    else:
        po = t.full((L, 2, B, H, oc, D // 2), 9, dtype=t.uint8, device="cuda")
        mo = t.full((L, 2, B, H, 4 * oc, 2), 9.0, device="cuda")
        wo = t.full((L, B, H, oc // GROUP), 9.0, device="cuda")
        lo = t.full((B,), 9, dtype=t.int32, device="cuda")
        base_p, base_m = to_host(po).copy(), to_host(mo).copy()
    kept = t.full((L, B, H, budget), 9, dtype=t.int32, device="cuda")
    cg.cg_evict(shape, codec, budget, sink, recent, wd, pd, md, out_shape, po, mo, wo, kept, lo, ln)
    got_p, got_m, got_w, got_k, got_l = (to_host(x) for x in (po, mo, wo, kept, lo))
    for b in range(B):
        T = min(max(lengths[b], 0), cap) if lengths else cap
        n = -(-T // GROUP)
        assert got_l[b] == (T - (n - budget) * GROUP if n > budget else T), b
        for l in range(L):
            for h in range(H):
                keep = oracle.serving.keep_blocks(mass[l, b, h], T, GROUP, budget, sink, recent)
                k, at = len(keep), (l, b, h)
                assert got_k[at].tolist() == keep + [-1] * (budget - k), at
                assert np.array_equal(got_w[at][:k], mass[at][keep]) and not got_w[at][k:].any(), at
                for kind in (0, 1):
                    f = (l, kind, b, h)
                    for src, dst, base in ((pay, got_p, base_p), (meta, got_m, base_m)):
                        s, d, e = src[f].reshape(nb, -1), dst[f].reshape(oc // GROUP, -1), base[f].reshape(oc // GROUP, -1)
                        assert np.array_equal(d[:k], s[keep]) and np.array_equal(d[k:], e[k:]), f


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("nb,budget,sink,recent", [(40, 13, 2, 3), (7, 1, 0, 1), (9, 9, 1, 1), (5, 30, 4, 4), (300, 290, 0, 2),
                                                  (1100, 300, 1, 5), (33, 6, 2, 4)])
def test_against_a_sort(nb, budget, sink, recent, in_place):
    total = max(nb, budget) if in_place else nb
    big = nb > 200
    run(nb, 1 if big else 2, 2, 1 if big else 2, total, budget, sink, recent,
        [nb * GROUP, max(1, nb * GROUP // 2 - 5)], in_place=in_place)


def test_lengths_at_their_ends():
    run(1, 1, 5, 1, 10, 4, 1, 2, [0, 1, 320, 129, 128])
    run(2, 1, 3, 1, 10, 4, 1, 2, [1 << 30, -4, 33])
    run(3, 2, 1, 3, 10, 4, 1, 2, None, out_nb=20)


@pytest.mark.parametrize("in_place", [False, True])
def test_ties(in_place):
    m = np.random.default_rng(4).integers(0, 3, (1, 2, 2, 300)).astype(np.float32)
    run(5, 1, 2, 2, 300, 90, 1, 2, [300 * GROUP, 300 * GROUP - 9], mass=m, in_place=in_place)
