"""NaN and infinity in queries and in blocks' ranges: they reach the rows that see
them, and no other row's value."""
import numpy as np
import pytest

import oracle
from gpu_util import to_host
from serve_util import Case, check

pytestmark = pytest.mark.gpu

# one row tile with eight waves / with splits, a few tiles, many rows without and with splits
FORMS = [dict(T=300, n=2), dict(T=3000, n=2, H=1, B=1), dict(T=700, n=10), dict(T=300, n=40),
         dict(T=9001, n=20, H=1, B=1)]


def compare(c, got, ref, bad):
    """Rows `bad` [B, n, Hq] have no number for out, the others lie within the bounds."""
    out, lse, mass = got
    o, ls = oracle.to_f32(to_host(out)), to_host(lse).copy()
    assert not np.isfinite(o[bad]).any()
    t = __import__("torch")
    clean = out.clone()
    where = t.from_numpy(bad).cuda()
    clean[where] = t.from_numpy(ref["out"][bad]).cuda().to(clean.dtype)
    lse = t.where(where, t.from_numpy(ref["lse"]).float().cuda(), lse)
    check(c, (clean, lse, None), ref)
    return ls


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite(form, bf16, value):
    c = Case(800 + form, bf16=bf16, **FORMS[form])
    ref = c.reference()
    c.device()
    L, B, H, R, n, T, block, g = c.dims
    c.q[0, n - 1, 1, 5] = value
    got = c.run()
    bad = np.zeros(c.q.shape[:3], bool)
    bad[0, n - 1, 1] = True
    ls = compare(c, got, ref, bad)
    assert np.isnan(ls[bad]).all()
    m = to_host(got[2])[0].astype(np.float64)
    assert np.isnan(m[0, 0]).all()
    m[0, 0] = ref["mass"][0, 0]
    assert np.all(np.abs(m - ref["mass"]) <= ref["mass_tol"])
    # and without the optional outputs (another variant of many rows)
    plain = c.run(lse=False, mass=False)[0]
    compare(c, (plain, got[1], None), ref, bad)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("kind,at,value", [(0, 0, "nan"), (0, 1, "nan"), (1, 0, "nan"), (1, 1, "nan"), (1, 1, "inf")])
def test_a_range_that_is_not_finite(form, bf16, block, kind, at, value):
    """The block of the last position: queries before it must not notice."""
    c = Case(830 + form, bf16=bf16, block=block, **FORMS[form])
    L, B, H, R, n, T, _, g = c.dims
    if T % block == 0 or (T - 1) % block > n - 2:    # some queries before the last block, some in it
        c.lengths = [T - (T - 1) % block + n // 2 - 1 if (T - 1) % block > n - 2 else T - block + n // 2] * B
    ref = c.reference()
    last = [(x - 1) // block for x in c.lengths]
    pos = np.array([[x - n + i for i in range(n)] for x in c.lengths])
    bad = np.zeros((B, n, H * R), bool)
    for b in range(B):
        c.meta[0, kind, b, 0, last[b], at] = float(value)
        bad[b, pos[b] // block == last[b], :R] = True
    assert bad.any() and not bad[:, :, :R].all()
    c.device()
    got = c.run()
    ls = compare(c, got, ref, bad)
    assert np.isnan(ls[bad]).all() == (kind == 0)
    plain = c.run(lse=False, mass=False)[0]
    compare(c, (plain, got[1] if kind else got[1].nan_to_num(0.0), None), ref, bad)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("value", [float("-inf"), float("inf")])
@pytest.mark.parametrize("T,n,R", [(20, 1, 2), (300, 5, 2), (9, 9, 8), (100, 100, 2), (70, 33, 3)])
def test_a_query_whose_scores_are_all_infinite(T, n, R, value, bf16):
    """No gauge, positive minima and codes: one infinite channel gives every visible key the
    same infinite score (all -inf: no weight is a number, and none is zero)."""
    c = Case(860 + T, T=T, n=n, R=R, g=0, bf16=bf16)
    c.meta[:, 0, ..., 0] = np.abs(c.meta[:, 0, ..., 0]) + np.float32(0.1)
    c.pay[:, 0, ..., 5] = np.maximum(c.pay[:, 0, ..., 5], 1)
    ref = c.reference()
    c.device()
    i = min(n - 1, 3)                       # in the prompts: a query that sees few tokens
    c.q[0, i, 1, 5] = value
    bad = np.zeros(c.q.shape[:3], bool)
    bad[0, i, 1] = True
    got = c.run()
    assert np.isnan(compare(c, got, ref, bad)[bad]).all()
    for lse in (False, True):
        out, ls, _ = c.run(lse=lse, mass=False)
        compare(c, (out, ls if lse else got[1], None), ref, bad)
        if lse:
            assert np.isnan(to_host(ls)[bad]).all()
