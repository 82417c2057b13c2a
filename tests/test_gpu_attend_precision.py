"""What cg_attend keeps of its operands, where a coarser form of them would give another
answer: small channels of a query beside a large one."""
import numpy as np
import pytest

import oracle
from gpu_util import to_host
from serve_util import D, Case

pytestmark = pytest.mark.gpu

FORMS = [(200, 1), (300, 1), (3000, 1), (3000, 12), (300, 20), (3000, 20)]   # four and eight waves, splits, many rows


@pytest.mark.parametrize("T,n", FORMS)
def test_small_channels_of_a_query(T, n):
    """One channel of 1 on keys of value 0 beside one of 2^-22 .. 2^-20 on keys of up to 2^20: a
    channel below 2^-11 of the row's largest keeps 12 bits (half a step of fp16), so a score
    of at most 1 is off by 2^-12, and a log-sum by that and its own rounding."""
    rng = np.random.default_rng(T + n)
    c = Case(900 + n, T=T, n=n, B=1, H=2, R=4, g=0, block=32, bf16=False, scale=1.0)
    c.meta[0, 0, ..., 1] = 2.0 ** 13
    c.meta[0, 0, ..., 0] = -128 * 2.0 ** 13
    c.pay[0, 0] = 128
    c.pay[0, 0, ..., 5] = rng.integers(0, 256, c.pay[0, 0, ..., 5].shape)
    c.qh[...] = 0
    c.qh[..., 0] = 1.0
    c.qh[..., 5] = rng.uniform(2.0 ** -22, 2.0 ** -20, c.qh.shape[:-1])
    c.qh[0, 0, 0, 5] = 2.0 ** -21
    ref = c.reference()
    c.device()
    for mass in (False, True):
        got = to_host(c.run(lse=True, mass=mass)[1]).astype(np.float64)
        assert np.all(np.abs(got - ref["lse"]) <= 2.0 ** -12 + 2.0 ** -20), float(np.abs(got - ref["lse"]).max())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T,n", FORMS)
def test_values_of_zero_beside_wide_ranges(T, n, block, causal):
    """Channels whose cached values are all 0, in blocks whose range reaches far to one side of 0
    for other channels: every product is with 0, so any weights give 0 exactly."""
    rng = np.random.default_rng(T + n + block)
    c = Case(920 + n, T=T, n=n, B=1, H=2, R=4, g=0, block=block, bf16=False, causal=causal)
    zero = rng.integers(0, 256, c.meta[0, 1, ..., 0].shape)              # the code of 0 in each block
    zero[..., ::5] = 0
    zero[..., 1::5] = 255
    step = np.exp2(rng.integers(-6, 7, zero.shape)).astype(np.float32)
    c.meta[0, 1, ..., 0], c.meta[0, 1, ..., 1] = -step * zero, step      # exact
    at = np.repeat(zero, block, -1)[..., None]
    c.pay[0, 1] = np.where(np.arange(D) % 3 == 0, at, c.pay[0, 1])
    c.device()
    for lse, mass in ((False, False), (True, True)):
        out = to_host(c.run(lse=lse, mass=mass)[0])
        assert not out[..., ::3].any(), float(np.abs(out[..., ::3]).max())
        assert out[..., 1::3].all()


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T,n", FORMS)
def test_keys_of_zero_beside_wide_ranges(T, n, block):
    """Keys of 0 in blocks whose range reaches far: scores are 0 exactly, the log-sum that of the
    number of visible tokens: 2^-22 of it for log2 and its factor, 2^-22 for a power of two and
    its reciprocal that each weight may carry (a unit in the last place each)."""
    rng = np.random.default_rng(T + n + block + 1)
    c = Case(940 + n, T=T, n=n, B=1, H=2, R=4, g=0, block=block, bf16=False, scale=1000.0)
    zero = rng.integers(0, 256, c.meta[0, 0, ..., 0].shape)
    step = np.exp2(rng.integers(-3, 4, zero.shape)).astype(np.float32)
    c.meta[0, 0, ..., 0], c.meta[0, 0, ..., 1] = -step * zero, step
    c.pay[0, 0] = np.repeat(zero, block, -1)[..., None]
    c.device()
    want = np.log(np.arange(T - n + 1, T + 1, dtype=np.float64))[None, :, None]
    for mass in (False, True):
        got = to_host(c.run(lse=True, mass=mass)[1]).astype(np.float64)
        assert np.all(np.abs(got - want) <= 2.0 ** -22 * want + 2.0 ** -22), float(np.abs(got - want).max())


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,n", FORMS)
@pytest.mark.parametrize("e", [-100, -90, 90, 116])
def test_powers_of_two_between_queries_and_keys(e, T, n, bf16):
    """Queries 2^e times as large on keys 2^e times as small: the same products and the same
    roundings, so the same bits.  (2^-13 of a row's largest channel times scale log2(e), 2^-120
    at -100, is a normal number; at -112 it would have 17 bits.)"""
    t = __import__("torch")
    c = Case(960 + n, T=T, n=n, B=1, H=2, R=4, block=32, bf16=bf16, spread=0.5, scale=2.0 ** -8)
    c.meta[:, 0] *= 2.0 ** 5
    c.device()
    kinds = ((False, False), (True, False), (True, True))
    want = [c.run(lse=a, mass=b) for a, b in kinds]
    c.q = (c.q.float() * 2.0 ** e).to(c.q.dtype)
    c.metad[:, 0] *= 2.0 ** -e
    for (a, b), w in zip(kinds, want):
        for x, y in zip(c.run(lse=a, mass=b), w):
            assert x is None or t.equal(x, y), (a, b)
