"""Where rows may lie that cg_read and cg_rotate write: layouts of which rows share memory are refused, the
others are not (checked on the host; no GPU is touched here)."""
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
