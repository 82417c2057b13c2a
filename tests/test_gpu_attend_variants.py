"""The variants of cg_attend that the optional outputs choose, above 64 rows a KV head:
nothing but out (bf16: queries in one fp16 part), the log-sums, and those with the
blocks' weights, over head layouts, masks, padding, block sizes and gauge groups, each
against the fp64 definition within the bounds of the variant that runs."""
import numpy as np
import pytest

from gpu_util import empty_u8, to_host
from fixed_rate_compression_amd import binding as cg
from serve_util import D, FEW, Case, check, check_outputs, form

pytestmark = pytest.mark.gpu


def torch():
    return __import__("torch")


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B,H,R,n,T,block,g", [
    (2, 2, 4, 20, 90, 16, 16),
    (1, 2, 3, 33, 200, 32, 8),     # tiles that start inside a query's group of heads
    (2, 1, 1, 80, 80, 64, 32),     # a whole prompt, no groups of heads
    (1, 1, 20, 7, 150, 16, 0),     # more heads in a group than a wave's half has rows
    (1, 1, 130, 1, 100, 64, 16),   # one query of more heads than a tile has rows
    (1, 2, 2, 150, 333, 64, 128),
    (3, 1, 8, 9, 65, 64, 128),
    (1, 4, 5, 129, 140, 16, 0),
])
def test_many_rows(B, H, R, n, T, block, g, causal, bf16):
    assert n * R > FEW
    lengths = [T] + [max(1, T // 2 - 3)] * (B - 1)
    check_outputs(Case(600 + n, B=B, H=H, R=R, n=n, T=T, block=block, g=g, bf16=bf16, lengths=lengths, causal=causal).device())


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,starts,lengths", [
    (40, [0, 0, 20], [40, 7, 41]),         # right-padded prompts, the last with rows before them
    (40, [-1, -40, 30], [39, 12, 31]),     # left-padded ones, one without queries
    (33, [0, 0, 0], [33, 0, 1]),           # an empty sequence
    (70, [-22, 5, 47], [48, 48, 48]),      # queries past the last row
])
def test_padding(n, starts, lengths, causal, bf16):
    c = Case(640 + n, B=3, n=n, T=48, block=16, R=2, lengths=lengths, starts=starts, causal=causal, bf16=bf16).device()
    ref = check_outputs(c)
    none = np.isneginf(ref["lse"])
    assert n * 2 > FEW and none.any()
    for mass in (False, True):
        assert not to_host(c.run(lse=mass, mass=mass)[0])[none].any()      # zeros, not small values


@pytest.mark.parametrize("bf16", [True, False])
def test_strided_queries_and_second_layer(bf16):
    t = torch()
    c = Case(660, L=3, layer=2, B=3, n=30, T=80, bf16=bf16).device()
    one, two = c.reference(one_part=bf16), c.reference()
    wide = t.full((3, 32, 12, D), 9.0, dtype=c.q.dtype, device="cuda")
    wide[:, :30, 2:10].copy_(c.q)
    q = wide[:, :30, 2:10]
    for lse, mass, ref in ((False, False, one), (True, False, two), (True, True, two)):
        check(c, c.run(lse=lse, mass=mass, q=q, strides=(q.stride(0), q.stride(1))), ref)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,splits", [(300, 1), (700, 2), (3000, None), (9001, None)])
def test_split_tokens(T, splits, bf16):
    c = Case(670, B=1, H=1, R=4, n=40, T=T, block=64, bf16=bf16).device()
    for mass in (False, True):
        rows, few, got = form(c, mass)
        assert rows == 160 and not few and (got == splits if splits else got > 2)
    check_outputs(c)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("n", [30, 150])
def test_rows_behind_the_end_do_not_count(bf16, n):
    """Codes and ranges behind a sequence's end change no bit of any variant."""
    t = torch()
    for block, T, lengths in ((16, 96, [49, 30]), (32, 160, [65, 32]), (64, 192, [64, 70])):
        c = Case(680 + block, T=T, block=block, lengths=lengths, n=n, bf16=bf16).device()
        kinds = ((False, False), (True, False), (True, True))
        before = [c.run(lse=a, mass=b) for a, b in kinds]
        for b, x in enumerate(lengths):
            used = -(-x // block)
            c.payd[:, :, b, :, x:] = 255
            c.metad[:, :, b, :, used:, 0] = float("nan")
            c.metad[:, :, b, :, used:, 1] = float("inf")
        for (a, b), want in zip(kinds, before):
            for x, y in zip(c.run(lse=a, mass=b), want):
                assert x is None or t.equal(x, y), (block, a, b)


@pytest.mark.parametrize("lse,mass", [(False, False), (True, False), (True, True)])
def test_graph_replay_as_the_sequence_grows(lse, mass):
    """One recorded call of many rows, replayed with other lengths and queries, beside eager work."""
    t = torch()
    c = Case(690, T=1500, n=40, R=2).device()
    L, B, H, R, n, T, block, g = c.dims
    at = c.attn()
    out = t.empty_like(c.q)
    ls = t.empty((B, n, H * R), device="cuda") if lse else None
    ms = t.zeros((L, B, H, c.cap // block), device="cuda") if mass else None
    ws = empty_u8(max(16, cg.cg_attend_workspace_bytes(c.shape, c.gauge, c.codec, at, mass)))

    def call():
        cg.cg_attend(c.shape, c.payd, c.metad, c.gauge, c.codec, at, c.q, out, ls, ms, ws)

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        call()
    side.synchronize()
    gr = t.cuda.CUDAGraph()
    with t.cuda.graph(gr):
        call()
    for k, ln in enumerate(([1500, 77], [64, 1500], [1, 0], [1333, 334])):
        c.len_d.copy_(t.tensor(ln, dtype=t.int32))
        c.q.copy_(t.randn(c.q.shape, device="cuda", generator=t.Generator("cuda").manual_seed(k)))
        if mass:
            ms.zero_()
        gr.replay()
        t.cuda.synchronize()
        got = [x if x is None else x.clone() for x in (out, ls, ms)]
        for x, y in zip(got, c.run(lse=lse, mass=mass)):
            assert x is None or t.equal(x, y), ln
