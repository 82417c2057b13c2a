"""cg_attend over 4-bit blocks whose tokens are of very unlike magnitudes, with the block's largest value on
both sides of powers of two: rows that see the small tokens alone get them as precisely as others theirs."""
import numpy as np
import pytest

from gpu_util import D
from serve4_util import GROUP, Case4
from test_gpu_attend4 import check_all

pytestmark = pytest.mark.gpu


def rising(n, R, bf16, top):
    """A prompt of n tokens whose values rise by 2^20 over a block to `top`; scores of about 0.01 (their error,
    which grows with them, would hide the values')."""
    c = Case4(600 + n, B=1, H=1, R=R, T=n, n=n, g=0, bf16=bf16, qscale=0.01)
    a = top * np.exp2(np.arange(c.cap) % GROUP * (20 / (GROUP - 1)) - 20)
    a = np.repeat(a, D // GROUP)
    c.meta[:, 1, ..., 0], c.meta[:, 1, ..., 1] = -a, a / 7.5
    return c


@pytest.mark.parametrize("top", [0.124, 0.126, 0.13, 1.0, 255.0, 257.0, 3e-6, 7e4])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("n,R", [(12, 4), (40, 4), (65, 1)])
def test_tokens_of_unlike_magnitude(n, R, bf16, top):
    check_all(rising(n, R, bf16, top).device(), top)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("n,T", [(1, 1), (5, 1), (20, 1), (70, 1), (12, 12), (40, 40), (1, 300), (40, 300), (1, 9000), (40, 9000)])
@pytest.mark.parametrize("alike", [True, False])
def test_values_beside_the_largest_number(n, T, alike, bf16):
    """Values of 2^127 and more, of which all weigh alike or one token has all the weight: sums of them would pass
    fp32, their averages do not; through waves, splits and merges."""
    c = Case4(640 + n, B=1, H=1, T=T, n=n, g=0, bf16=bf16, qscale=0.01 if alike else 1.0, causal=T == n)
    c.meta[:, 1, ..., 0], c.meta[:, 1, ..., 1] = 1.71e38, 5e36
    c.meta[:, 1, ..., 0::3, 0] = -2.46e38
    if not alike:      # the others' keys are far below the one's
        c.pay[:, 0] = 0x77
        c.pay[:, 0, :, :, T // 2] = 0xff
        c.meta[:, 0, ..., 0], c.meta[:, 0, ..., 1] = -20.0, 8 / 3.0
        c.qh = c.qh & 0x7fff if bf16 else np.abs(c.qh)
    c.device()
    check_all(c, (n, T))
