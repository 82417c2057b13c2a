"""Block weights are added to what stands there: two calls' in one array are the sum of each call's own."""
import numpy as np
import pytest

from fixed_rate_compression_amd import binding as cg
from gpu_util import empty_u8, to_host
from serve4_util import Case4
from serve_util import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [Case4, Case])
@pytest.mark.parametrize("n,T,lengths", [(1, 900, None), (1, 9000, [9000, 40]), (12, 900, None), (12, 9000, [9000, 40]),
                                         (40, 900, None), (40, 9000, [9000, 40])])
def test_two_calls_in_one_array(kind, n, T, lengths):
    """Few rows and many, in one split and in several, other layers left as they are."""
    t = __import__("torch")
    c = kind(800 + n, L=2, layer=1, T=T, n=n, lengths=lengths).device()
    L, B, H, R, _, _, block, g = c.dims
    at = c.attn()
    other = t.randn_like(c.q.float()).to(c.q.dtype)
    ws = empty_u8(cg.cg_attend_workspace_bytes(c.shape, c.gauge, c.codec, at, True))
    start = t.rand((L, B, H, c.cap // block), device="cuda") + 0.5

    def call(q, mass):
        cg.cg_attend(c.shape, c.payd, c.metad, c.gauge, c.codec, at, q, t.empty_like(c.q), None, mass, ws)
        return mass

    one, two = (to_host(call(q, t.zeros_like(start))).astype(np.float64) for q in (c.q, other))
    both = to_host(call(other, call(c.q, start.clone()))).astype(np.float64)
    first = to_host(start).astype(np.float64)
    assert np.array_equal(both[0], first[0]) and one[1].sum() > B * H * R * n * 0.5
    # two fp32 additions to each block, and each call's own sum of a block in fp32
    assert np.all(np.abs(both - (first + one + two)) <= 3 * 2.0 ** -24 * (first + one + two))
    assert np.abs(one - two).max() > 1e-3
