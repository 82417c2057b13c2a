"""The fp64 serving definitions against independent routines (torch on the CPU,
brute force): test infrastructure."""
import numpy as np
import torch

import oracle
from serve_util import Case


def test_attend_reference_against_torch_softmax():
    for causal in (True, False):
        c = Case(1, L=2, layer=1, B=2, H=2, R=3, n=4, T=37, block=16, g=16, lengths=[37, 20], causal=causal)
        ref = c.reference()
        q = torch.from_numpy(oracle.to_f32(c.qh)).double()
        for b, T in enumerate(c.lengths):
            for h in range(2):
                kv = []
                for kind in (0, 1):
                    mm = torch.from_numpy(c.meta[1, kind, b, h]).double().repeat_interleave(16, 0)
                    x = mm[:, :1] + mm[:, 1:] * torch.from_numpy(c.pay[1, kind, b, h]).double()
                    M = torch.block_diag(*torch.from_numpy(c.G[1, kind, h]).double())
                    kv.append((x @ M)[:T])                 # decoded rows: x = G^T x'
                for j in range(3):
                    s = (q[b, :, h * 3 + j] @ kv[0].T) * float(np.float32(c.scale))
                    if causal:
                        s = s.masked_fill(torch.arange(T)[None] > torch.arange(T - 4, T)[:, None], -np.inf)
                    o = torch.softmax(s, -1) @ kv[1]
                    assert np.allclose(ref["out"][b, :, h * 3 + j], o.numpy(), rtol=0, atol=1e-12)
                    assert np.allclose(ref["lse"][b, :, h * 3 + j], torch.logsumexp(s, -1).numpy(), atol=1e-12)
        assert np.allclose(ref["mass"].sum(-1), 3 * 4, atol=1e-10)


def test_padding_rows_see_nothing():
    c = Case(2, B=3, n=4, T=32, block=16, lengths=[2, 0, 9], starts=[0, 0, 7])
    ref = c.reference()
    assert np.array_equal(np.isneginf(ref["lse"][:, :, 0]),
                          [[False, False, True, True], [True] * 4, [False, False, True, True]])
    assert not ref["out"][0, 2:].any() and not ref["out"][1].any()


def test_quantize_matches_the_encoders_definition():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((70, 128)).astype(np.float32)
    x[32:48] = 1.25
    codes, meta = oracle.serving.quantize(x, 16)
    for k in range(5):
        y = x[16 * k:16 * k + 16]
        dec = meta[k, 0] + meta[k, 1] * codes[16 * k:16 * k + 16].astype(np.float64)
        assert np.max(np.abs(dec - y)) <= (y.max() - y.min()) / 255 * 0.5001 + 1e-6
    assert meta[2, 1] == 0 and not codes[32:48].any()


def test_keep_blocks_brute_force():
    rng = np.random.default_rng(4)
    for _ in range(50):
        n, block = int(rng.integers(1, 40)), 16
        sink, recent = int(rng.integers(0, 3)), int(rng.integers(1, 4))
        budget = sink + recent + int(rng.integers(0, 10))
        w = rng.integers(0, 5, n).astype(np.float32)
        got = oracle.serving.keep_blocks(w, n * block - 3, block, budget, sink, recent)
        assert got == sorted(set(got)) and len(got) == min(n, budget)
        if n > budget:
            assert set(range(sink)) <= set(got) and set(range(n - recent, n)) <= set(got)
            mid = [i for i in got if sink <= i < n - recent]
            for i in mid:
                for j in range(sink, n - recent):
                    if j not in mid:
                        assert (w[i], -i) > (w[j], -j)


def test_bounds_of_queries_in_one_part():
    """Attention of queries whose gauged channels are rounded to fp16, formed in 64 bits, stays
    within the one-part bound."""
    for seed, g, qscale in ((5, 16, 1.0), (6, 128, 8.0), (7, 8, 0.01)):
        c = Case(seed, B=1, H=1, R=2, n=5, T=90, block=16, g=g, qscale=qscale)
        ref = c.reference(one_part=True)
        K, V = (np.repeat(c.meta[0, kind, 0, 0], 16, 0)[:90].astype(np.float64) for kind in (0, 1))
        K, V = (m[:, :1] + m[:, 1:] * c.pay[0, kind, 0, 0, :90] for kind, m in ((0, K), (1, V)))
        GK, GV = (oracle.serving.dense(c.G[0, kind, 0]) for kind in (0, 1))
        worst = 0.0
        for i in range(5):
            for j in range(2):
                x = GK @ oracle.to_f32(c.qh)[0, i, j].astype(np.float64)
                up = 2.0 ** (13 - np.floor(np.log2(np.abs(x).max())))
                x = (x * up).astype(np.float16).astype(np.float64) / up
                s = (K[:86 + i] @ x) * np.float64(np.float32(c.scale))
                p = np.exp(s - s.max())
                err = np.abs((p / p.sum()) @ V[:86 + i] @ GV - ref["out"][0, i, j])
                assert np.all(err <= ref["out_tol"][0, i, j])
                worst = max(worst, float((err / ref["out_tol"][0, i, j]).max()))
        assert worst > 0                    # the rounding was there
