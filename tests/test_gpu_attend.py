"""cg_attend on the GPU against the fp64 definition: outputs, log-sums and block
weights within bounds counted from the kernels' roundings (oracle.serving),
over types, groups, head layouts, block sizes, lengths, padding and splits."""
import numpy as np
import pytest

import oracle
from fixed_rate_compression_amd import binding as cg
from gpu_util import D, empty_u8, to_dev, to_host
from serve_util import Case, check

pytestmark = pytest.mark.gpu


def torch():
    return __import__("torch")


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,block,lengths", [
    (1, 16, [1, 1]), (16, 16, [16, 3]), (17, 16, [17, 1]), (47, 16, [47, 0]), (48, 16, [48, 33]), (31, 32, [31, 32]),
    (100, 32, [100, 65]), (64, 64, [64, 1]), (577, 64, [577, 128]), (1000, 32, [1000, 999]), (2500, 16, [2500, 40]),
])
def test_single_token(T, block, lengths, bf16):
    c = Case(10 + T, T=T, block=block, lengths=[min(x, T) for x in lengths], bf16=bf16).device()
    check(c, c.run())


@pytest.mark.parametrize("g", [0, 8, 16, 32, 128])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("H,R,n", [(1, 1, 1), (2, 5, 1), (3, 7, 2), (1, 16, 1)])
def test_groups_and_heads(g, bf16, H, R, n):
    c = Case(100 + g + R, B=2, H=H, R=R, n=n, T=300, block=32, g=g, bf16=bf16, lengths=[300, 131]).device()
    check(c, c.run())


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B,H,R,n,T,block,g", [
    (2, 2, 4, 5, 90, 16, 16),      # two row tiles, the second of four rows
    (1, 2, 3, 33, 200, 32, 8),     # tiles that start inside a query's group of heads
    (2, 1, 1, 64, 64, 64, 32),     # a whole prompt
    (1, 1, 20, 7, 150, 16, 0),     # more heads in a group than a tile has rows
    (1, 2, 2, 150, 333, 64, 128),
])
def test_many_rows(B, H, R, n, T, block, g, causal, bf16):
    lengths = [T] + [max(1, T // 2 - 3)] * (B - 1)
    c = Case(200 + n, B=B, H=H, R=R, n=n, T=T, block=block, g=g, bf16=bf16, lengths=lengths, causal=causal).device()
    check(c, c.run())


@pytest.mark.parametrize("n,starts,lengths", [
    (1, [0, 5, 2], [9, 6, 2]),              # a query that is not the last position
    (6, [0, 0, 0], [6, 2, 0]),         # right-padded prompts
    (6, [-3, 2, -6], [3, 8, 40]),      # left-padded prompts; a sequence without queries
    (40, [0, 0, 20], [40, 7, 41]),
    (40, [-1, -40, 30], [39, 12, 31]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_padding(n, starts, lengths, causal):
    c = Case(300 + n, B=3, n=n, T=48, block=16, R=2, lengths=lengths, starts=starts, causal=causal).device()
    ref = c.reference()
    got = c.run()
    check(c, got, ref)
    none = np.isneginf(ref["lse"])
    assert none.any() or n == 1
    assert not to_host(got[0])[none].any()             # zeros, not small values


def test_optional_outputs_and_no_queries():
    c = Case(400, T=70, n=2).device()
    ref = c.reference()
    for lse in (False, True):
        for mass in (False, True):
            check(c, c.run(lse=lse, mass=mass), ref, (lse, mass))
    out = torch().full_like(c.q, 7.0)
    cg.cg_attend(c.shape, c.payd, c.metad, c.gauge, c.codec, c.attn(n=0), c.q[:, :0], out)
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("n", [2, 30])
def test_rows_behind_the_end_do_not_count(bf16, n):
    """Codes, ranges (NaN, infinity) behind a sequence's end change no bit."""
    t = torch()
    for block, T, lengths in ((16, 96, [49, 30]), (32, 96, [65, 32]), (64, 192, [64, 70])):
        c = Case(500 + block, T=T, block=block, lengths=lengths, n=n, bf16=bf16).device()
        a = c.run()
        for b, x in enumerate(lengths):
            used = -(-x // block)
            c.payd[:, :, b, :, x:] = 255
            c.metad[:, :, b, :, used:, 0] = float("nan")
            c.metad[:, :, b, :, used:, 1] = float("inf")
        z = c.run()
        for x, y in zip(a, z):
            assert t.equal(x, y), block
        check(c, z)


def test_lengths_out_of_range_are_clamped():
    t = torch()
    c = Case(510, T=40, lengths=[40, 40]).device()
    want = c.run()
    c.len_d.copy_(t.tensor([1 << 30, 41], dtype=t.int32))
    c.st_d = t.tensor([39, 39], dtype=t.int32, device="cuda")
    for x, y in zip(c.run(), want):
        assert t.equal(x, y)
    c.len_d.copy_(t.tensor([-5, -(1 << 31)], dtype=t.int32))
    out, lse, mass = c.run()
    assert not out.any() and bool(t.isneginf(lse).all()) and not mass.any()
    c.len_d.fill_(40)
    c.st_d.copy_(t.tensor([(1 << 31) - 1, -(1 << 31)], dtype=t.int32))
    out, lse, mass = c.run()
    assert not out.any() and bool(t.isneginf(lse).all()) and not mass.any()


@pytest.mark.parametrize("bf16", [True, False])
def test_strided_queries_and_second_layer(bf16):
    """Queries as a part of a fused projection's rows; layer 2 of 3."""
    t = torch()
    for n in (1, 9):
        c = Case(520, L=3, layer=2, B=3, n=n, T=80, bf16=bf16).device()
        ref = c.reference()
        wide = t.full((3, n + 2, 12, D), 9.0, dtype=c.q.dtype, device="cuda")
        wide[:, :n, 2:10].copy_(c.q)
        q = wide[:, :n, 2:10]
        check(c, c.run(q=q, strides=(q.stride(0), q.stride(1))), ref)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("kind", ["constant", "steps", "peaked", "heavy-tail"])
@pytest.mark.parametrize("n", [1, 12])
def test_extreme_ranges(kind, bf16, n):
    """Constant blocks (step 0), steps that differ by 2^40 between blocks, scores
    of hundreds, a rising maximum."""
    c = Case(530, T=700, block=16, B=1, bf16=bf16, n=n, qscale=30.0 if kind == "peaked" else 1.0)
    rng = np.random.default_rng(531)
    if kind == "constant":
        c.meta[:, :, :, :, ::2, 1] = 0.0
        c.pay[:, :, :, :, :].reshape(1, 2, 1, 2, -1, 16, D)[:, :, :, :, ::2] = 0
    elif kind == "steps":
        e = np.exp2(rng.uniform(-20, 20, c.meta[:, 1, ..., 1].shape)).astype(np.float32)
        c.meta[:, 1, ..., 1] *= e
        c.meta[:, 1, ..., 0] *= e
    elif kind == "heavy-tail":
        k = np.linspace(0.01, 4.0, c.meta.shape[4]).astype(np.float32)
        c.meta[:, 0] *= k[:, None]
    c.device()
    check(c, c.run(), where=kind)


@pytest.mark.parametrize("n,R", [(1, 4), (9, 4), (64, 4)])
def test_long_and_split(n, R):
    """Enough tokens for many splits; heads and sequences of unlike lengths."""
    c = Case(540 + n, B=2, H=1, R=R, n=n, T=9001, block=64, lengths=[9001, 300]).device()
    check(c, c.run())


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("lengths", [
    [2600, 1], [0, 0, 0, 2500], [0] * 5, [2049] * 3, [5000, 37, 0, 1200, 256, 4999, 31], [100] * 15 + [6000] + [900],
    [(37 * i) % 300 for i in range(69)] + [4000], [4000] + [0] * 66, [33] * 130,
])
def test_unlike_lengths(lengths, bf16):
    """Splits are dealt by length: one long sequence among short and empty ones, more
    sequences than a wave has lanes, equal ones."""
    c = Case(546 + len(lengths), B=len(lengths), H=1, R=3, n=1, T=6016, block=32, lengths=lengths, bf16=bf16).device()
    ref = c.reference()
    check(c, c.run(), ref)
    check(c, c.run(lse=False, mass=False), ref)


@pytest.mark.parametrize("n", [2, 15])
def test_unlike_lengths_with_row_tiles_and_padding(n):
    c = Case(547 + n, B=6, H=3, R=4, n=n, T=3000, block=16, lengths=[3000, 2, 0, 700, 1500, 64],
             starts=[2999 - n, 0, 0, 695, 1000, -1]).device()
    check(c, c.run())


@pytest.mark.parametrize("n", [1, 6])
def test_replay_of_unlike_lengths(n):
    """The dealing follows the lengths on the device."""
    t = torch()
    c = Case(548, B=5, T=4000, n=n).device()
    L, B, H, R, _, T, block, g = c.dims
    at = c.attn()
    out, mass = t.empty_like(c.q), t.zeros((L, B, H, c.cap // block), device="cuda")
    ws = empty_u8(cg.cg_attend_workspace_bytes(c.shape, c.gauge, c.codec, at, True))
    cg.cg_attend(c.shape, c.payd, c.metad, c.gauge, c.codec, at, c.q, out, None, mass, ws)
    gr = t.cuda.CUDAGraph()
    with t.cuda.graph(gr):
        cg.cg_attend(c.shape, c.payd, c.metad, c.gauge, c.codec, at, c.q, out, None, mass, ws)
    for ln in ([4000] * 5, [1, 4000, 0, 77, 2000], [0, 0, 0, 0, 9], [3999, 3000, 2000, 1000, 500]):
        c.len_d.copy_(t.tensor(ln, dtype=t.int32))
        mass.zero_()
        gr.replay()
        t.cuda.synchronize()
        want = c.run()
        assert t.equal(out, want[0]) and t.equal(mass, want[2]), ln


def test_more_workgroups_than_are_resident():
    """522 row tiles of few rows, split all the same: 5742 rows are merged by sixteens
    and the blocks' weights finished apart."""
    rng = np.random.default_rng(545)
    lengths = rng.integers(1, 700, 58).tolist()
    lengths[7] = 2500
    c = Case(545, B=58, H=3, R=11, n=3, T=2500, lengths=lengths).device()
    check(c, c.run())


def test_offsets_past_32_bits():
    """The second of two layers of a cache of more than 2^32 bytes."""
    t = torch()
    L, B, H, cap, T, block = 2, 1, 8, 1 << 20, 500, 32
    c = Case(550, L=1, B=B, H=H, T=T, cap=512, block=block, n=2)
    ref = c.reference()
    c.device()
    big = t.zeros((L, 2, B, H, cap, D), dtype=t.uint8, device="cuda")
    meta = t.zeros((L, 2, B, H, cap // block, 2), device="cuda")
    big[1, :, :, :, :512] = c.payd[0]
    meta[1, :, :, :, :512 // block] = c.metad[0]
    G = t.cat([t.zeros_like(to_dev(c.G)), to_dev(c.G)])
    c.payd, c.metad, c.gauge, c.layer, c.cap = big, meta, cg.make_gauge(16, G), 1, cap
    c.dims = (L,) + c.dims[1:]
    c.shape = cg.make_shape(L, 2, B, H, T, cap, D, cg.CG_DTYPE_BF16)
    out, lse, mass = c.run()
    check(c, (out, lse, None), ref)
    m = to_host(mass).astype(np.float64)[1, :, :, :512 // block]
    assert np.all(np.abs(m - ref["mass"]) <= ref["mass_tol"]) and not mass[0].any() and not mass[1, :, :, 16:].any()


@pytest.mark.parametrize("T,n,block,causal,bf16", [(500, 150, 32, True, True), (500, 150, 64, False, True),
                                                   (3001, 131, 16, True, False)])
def test_block_weights_of_queries_taken_in_turn(T, n, block, causal, bf16):
    """A capacity at which the rows' sums would pass 1 GiB: the queries go in turn, some of
    them padding before the first position or behind the last."""
    t = torch()
    B, H, R, cap = 2, 4, 4, 1 << 20
    used = -(-T // block) * block
    c = Case(555 + n, B=B, H=H, R=R, n=n, T=T, cap=used, block=block, bf16=bf16, lengths=[T, 77], starts=[T - n + 3, -60],
             causal=causal)
    ref = c.reference()
    c.device()
    big = t.zeros((1, 2, B, H, cap, D), dtype=t.uint8, device="cuda")
    meta = t.zeros((1, 2, B, H, cap // block, 2), device="cuda")
    big[:, :, :, :, :used] = c.payd
    meta[:, :, :, :, :used // block] = c.metad
    c.payd, c.metad, c.cap = big, meta, cap
    c.shape = cg.make_shape(1, 2, B, H, T, cap, D, cg.CG_DTYPE_BF16 if bf16 else cg.CG_DTYPE_F32)
    need = cg.cg_attend_workspace_bytes(c.shape, c.gauge, c.codec, c.attn(), True)
    assert need < 2 ** 30 < B * H * R * n * (cap // min(block, 32)) * 8
    out, lse, mass = c.run()
    check(c, (out, lse, None), ref)
    m = to_host(mass).astype(np.float64)[0]
    assert np.all(np.abs(m[..., :used // block] - ref["mass"]) <= ref["mass_tol"]) and not m[..., used // block:].any()


@pytest.mark.parametrize("n", [1, 40])
def test_mass_accumulates_and_repeats_bit_for_bit(n):
    t = torch()
    c = Case(560, T=3000, B=1, H=2, n=n).device()
    a, z = c.run(), c.run()
    for x, y in zip(a, z):
        assert t.equal(x, y)
    at = c.attn()
    ws = empty_u8(cg.cg_attend_workspace_bytes(c.shape, c.gauge, c.codec, at, True))
    out = t.empty_like(c.q)
    mass = t.full_like(a[2], 0.5)
    cg.cg_attend(c.shape, c.payd, c.metad, c.gauge, c.codec, at, c.q, out, None, mass, ws)
    assert t.equal(mass, a[2] + 0.5)


@pytest.mark.parametrize("n", [1, 24])
def test_graph_replay_as_the_sequence_grows(n):
    """One recorded call, replayed with other lengths and queries, beside eager work."""
    t = torch()
    c = Case(570, T=600, n=n, R=2).device()
    L, B, H, R, _, T, block, g = c.dims
    at = c.attn()
    out, lse = t.empty_like(c.q), t.empty((B, n, H * R), device="cuda")
    mass = t.zeros((L, B, H, c.cap // block), device="cuda")
    ws = empty_u8(cg.cg_attend_workspace_bytes(c.shape, c.gauge, c.codec, at, True))

    def call():
        cg.cg_attend(c.shape, c.payd, c.metad, c.gauge, c.codec, at, c.q, out, lse, mass, ws)

    side = t.cuda.Stream()
    with t.cuda.stream(side):
        call()
    side.synchronize()
    gr = t.cuda.CUDAGraph()
    with t.cuda.graph(gr):
        call()
    for k, ln in enumerate(([600, 77], [64, 600], [1, 0], [333, 334])):
        c.len_d.copy_(t.tensor(ln, dtype=t.int32))
        c.q.copy_(t.randn(c.q.shape, device="cuda", generator=t.Generator("cuda").manual_seed(k)))
        mass.zero_()
        gr.replay()
        t.cuda.synchronize()
        got = [x.clone() for x in (out, lse, mass)]
        want = c.run()
        for x, y in zip(got, want):
            assert t.equal(x, y), ln


def test_other_stream_and_two_at_once():
    t = torch()
    cs = [Case(580 + k, T=2000, n=1 + 20 * k).device() for k in range(2)]
    want = [c.run() for c in cs]
    t.cuda.synchronize()
    streams = [t.cuda.Stream() for _ in cs]
    got = []
    for c, s in zip(cs, streams):
        with t.cuda.stream(s):
            got.append(c.run())
    t.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert t.equal(x, y)


def test_encoded_cache_end_to_end():
    """cg_encode, then attention on the payload against attention on cg_decode's
    rows (fp32 storage: both sides differ by fp32 roundings only)."""
    t = torch()
    for g in (0, 16, 128):
        c = Case(590 + g, L=2, layer=1, T=256, n=2, g=g, bf16=False).device()
        x = t.randn((2 * 2 * 2 * 2, 256, D), device="cuda", generator=t.Generator("cuda").manual_seed(g))
        cg.cg_encode(c.shape, x, c.gauge, c.codec, 0, 256, c.payd, c.metad)
        rows = t.empty_like(x)
        cg.cg_decode(c.shape, c.payd, c.metad, c.gauge, c.codec, 0, 256, rows)
        c.pay, c.meta = to_host(c.payd), to_host(c.metad)
        ref = c.reference()
        got = c.run()
        check(c, got, ref)
        kv = to_host(rows).astype(np.float64).reshape(2, 2, 2, 2, 256, D)[1]
        q = c.qh.astype(np.float64)
        for b in range(2):
            for i in range(2):
                for j in range(8):
                    vis = 256 - 2 + i + 1
                    s = kv[0, b, j // 4, :vis] @ q[b, i, j] / np.sqrt(D)
                    p = np.exp(s - s.max())
                    o = (p / p.sum()) @ kv[1, b, j // 4, :vis]
                    assert np.max(np.abs(o - ref["out"][b, i, j])) < 1e-4
