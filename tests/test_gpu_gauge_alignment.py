"""Gauge matrices aligned as floats are, no further: a view that begins at any float gives the bits of one that begins
at an allocation."""
import pytest

from fixed_rate_compression_amd import binding as cg
from serve4_util import GROUP
from test_gpu_append import Filled
from test_gpu_append4 import Filled4
from test_gpu_attend4 import Case4
from test_gpu_read import Cache

pytestmark = pytest.mark.gpu


def moved(gauge, by):
    """The gauge's matrices `by` floats behind an allocation's start."""
    t = __import__("torch")
    G = gauge._keep
    whole = t.full((G.numel() + 4,), float("nan"), device="cuda")
    view = whole[by:by + G.numel()].view(G.shape)
    view.copy_(G)
    assert view.data_ptr() % 16 == 4 * by
    return cg.make_gauge(gauge.group, view)


@pytest.mark.parametrize("by", [1, 2, 3])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("g", [8, 16, 32, 128])
def test_appended_rows(g, bf16, by):
    for f in (Filled4(700 + g, [100, 33], bf16=bf16, g=g), Filled(701 + g, [100, 33], block=GROUP, bf16=bf16, g=g)):
        f.gauge = moved(f.gauge, by)
        f.put(f.x[0], f.x[1], 100, f.lengths, [0, 0])
        f.check()


@pytest.mark.parametrize("g", [8, 16, 32, 128])
def test_attention_and_rows_read_back(g):
    t = __import__("torch")
    for n in (1, 40):
        c = Case4(710 + g, T=100, n=n, g=g).device()
        want = c.run()
        c.gauge = moved(c.gauge, 1)
        for x, y in zip(c.run(), want):
            assert t.equal(x, y)
    for bits in (4, 8):
        c = Cache(711 + g, bits, g=g)
        want = c.read(70)
        c.gauge = moved(c.gauge, 3)
        for x, y in zip(c.read(70), want):
            assert t.equal(x, y)
