"""Layouts of a step's rows: tokens first ([n][batch][width]), sequences with room behind them; queries and keys
turned where they lie, rows read into keys and values side by side, appended from there."""
import numpy as np
import pytest

from fixed_rate_compression_amd import binding as cg
from fixed_rate_compression_amd.serving import ServingCache
from gpu_util import D, gauges_for, to_dev
from test_gpu_read import FILL, Cache
from test_gpu_rotate import Rot

pytestmark = pytest.mark.gpu
LAYOUTS = ["tokens first", "room behind a sequence", "room behind all sequences of a token"]


def torch():
    return __import__("torch")


def array(layout, B, n, heads, fill, dtype):
    """An array of `fill` and its view [B, n, heads, 128]."""
    t = torch()
    if layout == LAYOUTS[0]:
        a = t.full((n, B, heads, D), fill, dtype=dtype, device="cuda")
        return a, a.transpose(0, 1)
    if layout == LAYOUTS[1]:
        a = t.full((B, n * heads * D + 64), fill, dtype=dtype, device="cuda")
        return a, a[:, : n * heads * D].unflatten(1, (n, heads, D))
    a = t.full((n, B * heads * D + 64), fill, dtype=dtype, device="cuda")
    return a, a[:, : B * heads * D].unflatten(1, (B, heads, D)).transpose(0, 1)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("B,n", [(3, 6), (1, 5), (4, 1)])
def test_rotation_in_place(B, n, layout, bf16):
    r = Rot(90, B=B, n=n, Hq=6, H=2, bf16=bf16)
    whole, rows = array(layout, B, n, 11, 5.0, r.q.dtype)
    q, k = rows[:, :, :6], rows[:, :, 6:8]
    q.copy_(r.q)
    k.copy_(r.k)
    r.run(q, k, q, k)
    r.check((q, k))
    q.fill_(5.0)
    k.fill_(5.0)
    assert bool((whole == 5.0).all())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n", [1, 70])
def test_rows_read_side_by_side(n, layout, bits):
    c = Cache(95, bits, B=3, H=2)
    whole, rows = array(layout, 3, n, 5, FILL, c.dtype)
    k, v = rows[:, :, :2], rows[:, :, 2:4]
    lengths = [256, 40, 0]
    got = c.read(n, lengths, k=k, v=v)
    c.check([x.contiguous() for x in got], n, lengths)
    k.fill_(FILL)
    v.fill_(FILL)
    assert bool((whole == FILL).all())


@pytest.mark.parametrize("layout", LAYOUTS)
def test_a_step_on_a_fused_projection(layout):
    """Rotation, append, attention and reading back on such rows give the bits that dense ones give."""
    t = torch()
    B, n, H, R = 2, 40, 2, 4
    gauge = cg.make_gauge(16, to_dev(np.ascontiguousarray(gauges_for(96, 1, 2, H, 16))))
    rotary = cg.make_rotary(to_dev((1e4 ** (-np.arange(64) / 64)).astype(np.float32)))
    x = t.randn((B, n, (R + 2) * H, D), generator=t.Generator("cuda").manual_seed(97), device="cuda").bfloat16()
    res = []
    for rows in (x.clone(), array(layout, B, n, (R + 2) * H, 0.0, x.dtype)[1]):
        rows.copy_(x)
        q, k, v = (y.contiguous() if rows.is_contiguous() else y for y in rows.split((R * H, H, H), 2))
        c = ServingCache(1, B, H, R * H, 64, gauge, bits=4)
        c.begin(n)
        c.rotate(q, k, rotary)
        c.append(0, k, v)
        res.append((q.contiguous(), c.attend(0, q), *c.read(0, n), c.payload, c.meta))
    for a, b in zip(*res):
        assert t.equal(a, b)
