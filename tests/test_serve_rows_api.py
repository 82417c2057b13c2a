"""Where rows may lie that cg_read and cg_rotate write: layouts of which rows share memory are refused, the
others are not (checked on the host; no GPU is touched here)."""
import random

import pytest

from fixed_rate_compression_amd import binding as cg
from test_serve4_api import FAR, K4, read, rotate, rows, shape

W, WQ = 2 * 128, 4 * 128  # elements of a row of keys, of queries


@pytest.mark.parametrize("bs,rs", [(8, W + 8), (8, W), (W - 8, 2 * W), (W - 8, 1 << 20), (8, 8), (W, 8), (1 << 20, W - 8)])
def test_rows_that_lie_in_one_another(bs, rs):
    """The second sequence's rows begin inside the first's, between them the next token's."""
    for v in (None, 2 * FAR):
        assert read(sh=shape(tokens=0), n=3, bs=bs, rs=rs, v=v) == cg.CG_E_INVAL
        assert "overlap" in cg.cg_last_error()
    assert rotate(ko=rows(4 * FAR, bs, rs)) == cg.CG_E_INVAL
    assert rotate(qo=rows(3 * FAR, 2 * bs, 2 * rs)) == cg.CG_E_INVAL
    assert rotate(q=None, qo=None, k=rows(FAR, bs, rs), ko=rows(FAR, bs, rs)) == cg.CG_E_INVAL
    assert "overlap" in cg.cg_last_error()


def test_one_row_a_sequence_and_one_sequence():
    sh = shape(tokens=0)
    assert read(sh=sh, n=1, bs=W - 8, v=None) == cg.CG_E_INVAL
    assert read(sh=sh, n=1, bs=W, v=None) == cg.CG_OK
    assert read(sh=sh, n=1, bs=W, rs=8, v=None) == cg.CG_OK          # a stride that no row uses
    one = shape(tokens=0, batch=1)
    assert read(sh=one, n=3, rs=W - 8, bs=1 << 20, v=None) == cg.CG_E_INVAL
    assert read(sh=one, n=3, rs=W, bs=8, v=None) == cg.CG_OK


@pytest.mark.parametrize("co", [K4, cg.make_codec(cg.CG_BACKEND_BLOCK_UNIFORM, 8, 32)])
def test_layouts_that_lie_apart(co):
    for bs, rs in ((3 * W, W), (W, 2 * W), (W + 64, 2 * W + 128), (3 * W + 64, W)):
        assert read(sh=shape(tokens=0), co=co, n=3, bs=bs, rs=rs, v=None) == cg.CG_OK, (bs, rs)


def marks(at, bs, rs, batch, n, w):
    return {at + b * bs + i * rs + e for b in range(batch) for i in range(n) for e in range(0, w, 8)}


def test_keys_and_values_in_the_same_rows():
    """k_out and v_out laid out alike in one array, against their elements counted one by one: sequences or
    tokens first, rows and sequences with room behind them, one row or sequence."""
    rng = random.Random(5)
    seen = {cg.CG_OK: 0, cg.CG_E_INVAL: 0}
    for _ in range(4000):
        batch, n, w = rng.randint(1, 4), rng.randint(1, 5), 128
        inner = w * rng.randint(1, 3) + 8 * rng.choice([0, 0, 1, 5, 16])
        by_row = rng.random() < 0.5
        outer = inner * ((n if by_row else batch) - 1) + w + 8 * rng.choice([0, 0, 1, 7, 16, 48, rng.randint(0, 200)])
        rs, bs = (inner, outer) if by_row else (outer, inner)
        d = 8 * rng.randint(-60, 60) if rng.random() < 0.5 else rng.choice([-1, 1]) * (
            inner * rng.randint(0, n + 1) + outer * rng.randint(0, batch + 1) + 8 * rng.randint(-17, 17))
        at = 1 << 30
        apart = not (marks(at, bs, rs, batch, n, w) & marks(at + d, bs, rs, batch, n, w))
        got = read(sh=shape(tokens=0, batch=batch, heads=1), n=n, bs=bs, rs=rs, k=FAR + 2 * at, v=FAR + 2 * (at + d))
        assert got == (cg.CG_OK if apart else cg.CG_E_INVAL), (batch, n, bs, rs, d)
        seen[got] += 1
    assert min(seen.values()) > 500


def test_far_strides():
    sh = shape(tokens=0)
    for bs, rs in ((1 << 40, W), (W, 1 << 40), (1 << 40, 1 << 20), (1 << 20, 1 << 40)):
        side = cg.CG_OK if min(bs, rs) > W else cg.CG_E_INVAL   # room beside a row, or the next one
        for d, code in ((W, side), (W + 8, side), (4 * W, cg.CG_OK), (8 - W, cg.CG_E_INVAL)):
            assert read(sh=sh, n=3, bs=bs, rs=rs, k=FAR, v=FAR + 2 * d) == code, (bs, rs, d)
    most = (1 << 31) // 64
    assert read(sh=shape(tokens=0, batch=1), n=most, rs=2 * W, k=FAR, v=FAR + 2 * W) == cg.CG_OK
    assert read(sh=shape(tokens=0, batch=1), n=most, rs=2 * W, k=FAR, v=FAR + 2 * W + 16) == cg.CG_E_INVAL


def test_queries_and_keys_that_share_memory():
    """In place in layouts that are not [batch][n][width]: parts of one another are refused as before."""
    T = (WQ + W) // 2  # time-major rows of fewer elements than both
    for bs, rs in ((T, 2 * T), (2 * T, T), (WQ + W - 8, 2 * (WQ + W)), (3 * (WQ + W) + 64, WQ + W - 8)):
        a, b = rows(FAR, bs, rs), rows(FAR + 2 * WQ, bs, rs)
        assert rotate(q=a, qo=a, k=b, ko=b) == cg.CG_E_INVAL
    a, b = rows(FAR, WQ + W, 2 * (WQ + W)), rows(FAR + 2 * WQ - 16, WQ + W, 2 * (WQ + W))
    assert rotate(q=a, qo=a, k=b, ko=b) == cg.CG_E_INVAL
