"""The fp64 definitions of the 4-bit serving operators against independent routines (torch on the CPU,
complex numbers, the C part of the oracle): test infrastructure."""
import numpy as np
import torch

import oracle
from serve4_util import Case4


def test_attend_reference_against_torch_softmax():
    for causal in (True, False):
        c = Case4(1, L=2, layer=1, B=2, H=2, R=3, n=4, T=67, g=16, lengths=[67, 20], causal=causal)
        ref = c.reference()
        q = torch.from_numpy(oracle.to_f32(c.qh)).double()
        for b, T in enumerate(c.lengths):
            for h in range(2):
                kv = []
                for kind in (0, 1):
                    byte = torch.from_numpy(c.pay[1, kind, b, h])
                    code = torch.stack([byte % 16, byte // 16], -1).double().flatten(1)
                    m = torch.from_numpy(c.meta[1, kind, b, h]).double()
                    if kind == 0:
                        m = m.view(-1, 1, 128, 2).expand(-1, 32, 128, 2).reshape(-1, 128, 2)
                    else:
                        m = m.view(-1, 4, 1, 2).expand(-1, 4, 32, 2).reshape(-1, 128, 2)
                    M = torch.block_diag(*torch.from_numpy(c.G[1, kind, h]).double())
                    kv.append(((m[..., 0] + m[..., 1] * code) @ M)[:T])                 # decoded rows: x = G^T x'
                for j in range(3):
                    s = (q[b, :, h * 3 + j] @ kv[0].T) * float(np.float32(c.scale))
                    if causal:
                        s = s.masked_fill(torch.arange(T)[None] > torch.arange(T - 4, T)[:, None], -np.inf)
                    o = torch.softmax(s, -1) @ kv[1]
                    assert np.allclose(ref["out"][b, :, h * 3 + j], o.numpy(), rtol=0, atol=1e-11)
                    assert np.allclose(ref["lse"][b, :, h * 3 + j], torch.logsumexp(s, -1).numpy(), atol=1e-11)
        assert np.allclose(ref["mass"].sum(-1), 3 * 4, atol=1e-10)


def test_quantizer_is_the_encoders():
    """Whole blocks: the C quantizer's bytes and ranges; parts of one: their own ranges."""
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((96, 128)) * np.exp(rng.standard_normal(128))).astype(np.float32)
    x[32:64, 5] = 1.25
    x[40] = -3.0
    for kind in (0, 1):
        pay, meta, _ = oracle.kivi_encode_field(x, kind, 32, 4, 0)
        p, m = oracle.serving4.quantize(x, kind)
        assert np.array_equal(p.reshape(-1), pay) and np.array_equal(m, meta)
        dec = oracle.kivi_decode_field(pay, meta, np.zeros((0, 128), np.float32), 96, 128, kind, 32, 4, 0)
        full = np.zeros((4 * 96, 2), np.float32)
        full[:len(m)] = m
        assert np.allclose(oracle.serving4.decoded(p, full, kind, 96), dec, rtol=1e-6, atol=1e-6)
        for T in (1, 31, 33, 70):
            p2, m2 = oracle.serving4.quantize(x[:T], kind)
            assert p2.shape == (T, 64) and len(m2) == (-(-T // 32) * 128 if kind == 0 else 4 * T)
            whole = T // 32 * 32
            assert np.array_equal(p2[:whole], p[:whole]) and np.array_equal(m2[:whole * 4], m[:whole * 4])


def test_codes_and_bytes():
    rng = np.random.default_rng(4)
    c = rng.integers(0, 16, (5, 128)).astype(np.uint8)
    b = oracle.serving4.packed(c)
    assert np.array_equal(oracle.serving4.codes(b), c)
    assert np.array_equal(oracle.unpack_codes(b.reshape(-1), 5 * 128, 4), c.reshape(-1))


def test_rotation_is_a_turn():
    """Complex products; lengths stay, scores depend on the distance alone, an axis turns its own pairs."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((2, 3, 2, 128))
    freq = (1e4 ** (-np.arange(64) / 64)).astype(np.float32)
    pos = rng.integers(0, 1000, (1, 2, 3))
    for il in (False, True):
        y, _ = oracle.serving4.rotate(x, None, 0.0, freq, pos, il)
        a = np.arange(64) * 2 if il else np.arange(64)
        b = a + 1 if il else a + 64
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[0][:, :, None, None] * freq.astype(np.float64))
        assert np.allclose(y[..., a], z.real) and np.allclose(y[..., b], z.imag)
        s = [float((oracle.serving4.rotate(x[:1, :1], None, 0.0, freq, np.full((1, 1, 1), p + 7), il)[0] *
                    oracle.serving4.rotate(x[1:, :1], None, 0.0, freq, np.full((1, 1, 1), p), il)[0]).sum()) for p in (0, 100)]
        assert abs(s[0] - s[1]) < 1e-9
    w = 1 + 0.1 * rng.standard_normal(128)
    y, _ = oracle.serving4.rotate(x, w, 0.0, freq[:0], pos, False)
    assert np.allclose((y / w) @ np.ones(128), (x / np.sqrt((x * x).mean(-1, keepdims=True))) @ np.ones(128))
    p2 = np.stack([pos[0], np.zeros_like(pos[0])])
    for dealt, still in ((False, np.arange(32, 64)), (True, np.arange(1, 64, 2))):
        y, _ = oracle.serving4.rotate(x, None, 0.0, freq, p2, False, [32, 32], dealt)
        assert np.array_equal(y[..., still], x[..., still]) and np.array_equal(y[..., still + 64], x[..., still + 64])
        moved = np.setdiff1d(np.arange(64), still)
        assert not np.any(np.isclose(y[..., moved[:5]], x[..., moved[:5]], atol=1e-9)[pos[0] > 0])
