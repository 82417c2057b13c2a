"""The merge of splits and its inverse gauge, over every gauge group and both storage
types: a workgroup to a row (few and many splits, equal and dealt by length) and, past
4096 rows, sixteen rows to a workgroup."""
import numpy as np
import pytest

from serve_util import FEW, Case, check, check_outputs, form

pytestmark = pytest.mark.gpu

GROUPS = [0, 8, 16, 32, 128]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("g", GROUPS)
@pytest.mark.parametrize("T,n,lo,hi", [
    (1100, 1, 2, 8),          # a few splits
    (9001, 2, 32, 64),        # more than a wave's first four a group of lanes
    (20000, 1, 64, 128),
    (40000, 1, 128, 1024),    # more than a wave holds two of
    (3000, 11, 2, 32),        # several row tiles
    (2100, 30, 2, 32),        # many rows
])
def test_a_workgroup_to_a_row(T, n, lo, hi, g, bf16):
    H, R = 2, 3
    c = Case(700 + T, B=1, H=H, R=R, n=n, T=T, block=64, g=g, bf16=bf16).device()
    for mass in (False, True):
        rows, few, splits = form(c, mass)
        assert few == (rows <= FEW) and lo <= splits <= hi and H * rows <= 4096, (few, splits)
    check_outputs(c)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("g", GROUPS)
def test_splits_dealt_by_length(g, bf16):
    lengths = [5000, 37, 0, 1200, 256, 4999, 31]
    c = Case(710, B=7, H=2, R=3, n=2, T=6016, block=32, lengths=lengths, g=g, bf16=bf16).device()
    check_outputs(c)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("g", GROUPS)
def test_sixteen_rows_to_a_workgroup(g, bf16):
    """4100 rows of a prompt's last chunk: the last workgroup of a head has two rows."""
    H, R, n = 2, 2, 1025
    c = Case(720, B=1, H=H, R=R, n=n, T=1100, block=32, g=g, bf16=bf16).device()
    rows, few, splits = form(c, True)
    assert not few and splits > 1 and H * rows > 4096 and rows % 16 == 2
    check_outputs(c)


@pytest.mark.parametrize("g", GROUPS)
def test_sixteen_rows_to_a_workgroup_of_dealt_splits(g):
    """Few rows of many heads and sequences, some in one split: their rows are left alone."""
    rng = np.random.default_rng(730)
    lengths = rng.integers(1, 700, 58).tolist()
    lengths[7] = 2500
    c = Case(730, B=58, H=3, R=11, n=3, T=2500, lengths=lengths, g=g).device()
    ref = c.reference()
    check(c, c.run(), ref)
    check(c, c.run(lse=False, mass=False), ref)
