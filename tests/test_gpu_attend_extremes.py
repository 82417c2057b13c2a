"""Ranges and scores at their ends, in every form of cg_attend: constant blocks (step
0), value steps that differ by 2^40 between blocks, scores of hundreds, a rising
maximum.  Which form and how many splits a case takes is read off its workspace."""
import numpy as np
import pytest

from serve_util import D, FEW, Case, check_outputs, form

pytestmark = pytest.mark.gpu

# tokens, queries (4 heads a group), few rows or many, splits (None: more than two)
FORMS = [
    (200, 1, True, 1), (200, 16, True, 1),          # four waves, no merge
    (700, 1, True, 1), (700, 12, True, 1),          # eight waves
    (3000, 1, True, None), (3000, 12, True, None),  # four waves and a merge
    (9000, 5, True, None),
    (300, 20, False, 1), (700, 20, False, 2), (9000, 20, False, None), (300, 60, False, 1),
]


def extreme(c, kind, block):
    """Blocks whose tokens are worlds apart; reshaped views write through."""
    L, B, H, R, n, T, _, g = c.dims
    rng = np.random.default_rng(531)
    if kind == "constant":
        c.meta[:, :, :, :, ::2, 1] = 0.0
        c.pay.reshape(L, 2, B, H, -1, block, D)[:, :, :, :, ::2] = 0
    elif kind == "all constant":
        c.meta[..., 1] = 0.0
        c.pay[:] = 0
    elif kind == "steps":
        e = np.exp2(rng.uniform(-20, 20, c.meta[:, 1, ..., 1].shape)).astype(np.float32)
        c.meta[:, 1] *= e[..., None]
    elif kind == "heavy-tail":
        c.meta[:, 0] *= np.linspace(0.01, 4.0, c.meta.shape[4]).astype(np.float32)[:, None]
    elif kind == "far apart":       # the later half's scores are hundreds above: splits of unlike maxima
        c.meta[:, 0, :, :, : c.meta.shape[4] // 2] *= np.float32(2.0 ** -7)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("kind", ["constant", "all constant", "steps", "peaked", "heavy-tail", "far apart"])
@pytest.mark.parametrize("T,n,few,splits", FORMS)
def test_extreme_ranges(T, n, few, splits, kind, bf16):
    block = 32 if n == 60 else 16
    c = Case(530, T=T, block=block, B=1, bf16=bf16, n=n, qscale=30.0 if kind in ("peaked", "far apart") else 1.0)
    extreme(c, kind, block)
    c.device()
    for mass in (False, True):
        rows, is_few, got = form(c, mass)
        assert is_few == few == (rows <= FEW) and (got > 2 if splits is None else got == splits), (is_few, got)
    check_outputs(c)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("n", [1, 12, 20])
@pytest.mark.parametrize("rising", [True, False])
def test_a_maximum_that_moves_with_every_block(n, rising, bf16):
    """Scores along one channel, from -300 to 300 and back, a step of a few with every block."""
    T, block = 2900, 16
    c = Case(532, T=T, block=block, B=1, H=1, R=4, n=n, g=0, bf16=bf16, scale=1.0)
    nb = c.meta.shape[4]
    c.qh[...] = 0
    one = np.zeros(D, np.float32)
    one[7] = 1.0
    c.qh[:] = __import__("oracle").f32_to_bf16(one) if bf16 else one
    ramp = np.linspace(-300.0, 300.0, nb).astype(np.float32)
    c.meta[0, 0, 0, 0, :, 0] = ramp if rising else ramp[::-1]
    c.meta[0, 0, 0, 0, :, 1] = 2.0 ** -8
    c.device()
    check_outputs(c)
