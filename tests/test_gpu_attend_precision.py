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
