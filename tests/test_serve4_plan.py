"""Into how many workgroups few rows over the 4-bit cache are split, read off the workspace (no GPU is touched here)."""
import ctypes

import pytest

from fixed_rate_compression_amd import binding as cg
from test_serve4_api import K4, attn, shape


def splits(rows, dtype, tokens=65536, heads=8):
    """Splits of one sequence's `rows` queries a KV head: parts of 512 + 8 bytes a row each, in whole 256 bytes."""
    n = ctypes.c_size_t()
    r = ctypes.byref
    sh = shape(layers=1, batch=1, heads=heads, tokens=tokens, token_capacity=tokens, dtype=dtype)
    assert cg.lib().cg_attend_workspace_bytes(r(sh), r(cg.make_gauge(0)), r(K4), r(attn(q_heads=heads, n_queries=rows)), 0,
                                              r(n)) == cg.CG_OK
    up = lambda x: -(-x // 256) * 256
    found = [s for s in range(2, 1025) if up(heads * rows * s * 512) + up(heads * rows * s * 8) == n.value]
    assert len(found) == 1, n.value
    return found[0]


@pytest.mark.parametrize("rows,dtype,resident", [
    (4, cg.CG_DTYPE_BF16, 3), (8, cg.CG_DTYPE_BF16, 3), (16, cg.CG_DTYPE_BF16, 3),
    (4, cg.CG_DTYPE_F32, 3), (8, cg.CG_DTYPE_F32, 3), (9, cg.CG_DTYPE_F32, 2), (16, cg.CG_DTYPE_F32, 2),
])
def test_one_round_of_what_a_compute_unit_holds(rows, dtype, resident):
    """Each part of a long sequence is in the first round of workgroups; 16 rows of fp32 storage take 57 KB of LDS, so
    that two of them fit the 160 KB of a compute unit, not three."""
    assert splits(rows, dtype) * 8 == 256 * resident
