"""Ends of the 4-bit serving operators: sequences and queries that are taken in turn where a workspace would grow
too large, caches without tokens, workspaces that two recorded steps share, calls on other streams, operators that
follow one another on the same buffers."""
import numpy as np
import pytest

import oracle
from fixed_rate_compression_amd import binding as cg
from gpu_util import D, empty_u8, to_dev, to_host
from serve4_util import GROUP, Case4
from serve_util import check
from test_gpu_append4 import Filled4

pytestmark = pytest.mark.gpu


def torch():
    return __import__("torch")


def enlarge(c, cap):
    """The case's rows at the beginning of a cache of cap tokens, its bound of the lengths too."""
    t = torch()
    L, B, H, R, n, T, block, g = c.dims
    c.device()
    pay = t.zeros((L, 2, B, H, cap, D // 2), dtype=t.uint8, device="cuda")
    meta = t.zeros((L, 2, B, H, 4 * cap, 2), device="cuda")
    pay[..., :c.cap, :] = c.payd
    meta[..., :4 * c.cap, :] = c.metad
    c.payd, c.metad, c.cap = pay, meta, cap
    c.shape = cg.make_shape(L, 2, B, H, cap, cap, D, cg.CG_DTYPE_BF16 if c.bf16 else cg.CG_DTYPE_F32)
    return c


def blocks_first(got, small):
    """The mass of the blocks that the small cache has; none has gone to others."""
    out, lse, mass = got
    if mass is None:
        return got
    assert not bool(mass[..., small:].any())
    return out, lse, mass[..., :small].contiguous()


@pytest.mark.parametrize("bf16", [True, False])
def test_sequences_and_queries_in_turn(bf16):
    """Ranges for 3 sequences of 8 heads and 262144 tokens pass 256 MiB, and the sums of 1200 rows of the two
    that go first 1 GiB."""
    c = Case4(900, B=3, H=8, R=4, n=300, T=416, cap=416, lengths=[416, 317, 0], bf16=bf16)
    two = c.reference()
    one = c.reference(one_part=True) if bf16 else two
    small = c.cap // GROUP
    enlarge(c, 262144)
    need = cg.cg_attend_workspace_bytes(c.shape, c.gauge, c.codec, c.attn(), True)
    one_by_one = 8 * 8192 * (1536 if bf16 else 2048)
    assert one_by_one < need < 3 * one_by_one + (1 << 30) + (1 << 28)
    for lse, mass, ref in ((False, False, one), (True, False, two), (True, True, two)):
        check(c, blocks_first(c.run(lse=lse, mass=mass), small), ref, (lse, mass))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("n,R", [(13, 4), (16, 4), (49, 1), (12, 4)])
def test_four_row_tiles_of_many_tokens(n, R, bf16):
    """Past 262144 tokens of all heads 49 to 64 rows are taken by the many-row form."""
    c = Case4(905 + n, B=8, H=8, R=R, n=n, T=4096, lengths=[4096, 130, 64, 33, 97, 0, 1, 200], bf16=bf16).device()
    two = c.reference()
    one = c.reference(one_part=True) if bf16 and n * R > 48 else two
    for lse, mass, ref in ((False, False, one), (True, False, two), (True, True, two)):
        check(c, c.run(lse=lse, mass=mass), ref, (lse, mass))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("R,n", [(5, 1), (7, 1), (8, 1), (4, 2), (2, 3), (1, 9), (3, 4), (4, 4)])
@pytest.mark.parametrize("T,lengths", [(700, [700, 33, 300]), (5000, [5000, 31, 2300])])
def test_five_to_sixteen_rows(R, n, bf16, T, lengths):
    """The forms of 8 and of 16 rows, by eight waves and in splits that follow the lengths."""
    c = Case4(920 + R + n, B=3, H=2, R=R, n=n, T=T, lengths=lengths, bf16=bf16).device()
    ref = c.reference()
    for lse, mass in ((False, False), (True, False), (True, True)):
        check(c, c.run(lse=lse, mass=mass), ref, (lse, mass))


@pytest.mark.parametrize("n", [1, 4])
@pytest.mark.parametrize("B,H", [(48, 8), (64, 12), (33, 10)])
def test_many_sequences_of_unlike_lengths(B, H, n):
    """One split each, the workgroups that fill the compute units dealt by length."""
    rng = np.random.default_rng(B)
    lengths = np.where(rng.random(B) < 0.1, rng.integers(1500, 2301, B), rng.integers(0, 90, B)).tolist()
    lengths[1:4] = [2300, 0, 1]
    c = Case4(925 + B, B=B, H=H, R=2, n=n, T=2300, lengths=lengths).device()
    ref = c.reference()
    check(c, c.run(lse=False, mass=False), ref)
    check(c, c.run(lse=True, mass=True), ref)


@pytest.mark.parametrize("n", [1, 5, 40])
@pytest.mark.parametrize("cap", [0, 32, 4096])
def test_no_tokens(n, cap):
    """A cache that has no rows, or room for none: outputs of zeros, log-sums of minus infinity."""
    t = torch()
    B, H, R = 2, 2, 4
    shape = cg.make_shape(1, 2, B, H, 0, cap, D, cg.CG_DTYPE_BF16)
    codec, gauge = cg.make_codec(cg.CG_BACKEND_KIVI, 4, 32), cg.make_gauge(0)
    pay = t.zeros(max(16, 2 * B * H * cap * 64), dtype=t.uint8, device="cuda")
    meta = t.full((max(4, 2 * B * H * cap * 8),), float("nan"), device="cuda")
    mass = t.zeros((1, B, H, max(1, cap // 32)), device="cuda")
    q = t.randn(B, n, H * R, D, device="cuda").to(t.bfloat16)
    out, lse = t.full_like(q, 7.0), t.full((B, n, H * R), 7.0, device="cuda")
    at = cg.make_attn(0, H * R, n, 0.1, True)
    ws = empty_u8(max(16, cg.cg_attend_workspace_bytes(shape, gauge, codec, at, True)))
    cg.cg_attend(shape, pay, meta, gauge, codec, at, q, out, lse, mass, ws)
    assert not bool(out.any()) and bool(t.isneginf(lse).all()) and not bool(mass.any())
    k = t.full((B, 3, H, D), 7.0, dtype=t.bfloat16, device="cuda")
    cg.cg_read(shape, pay, meta, gauge, codec, 0, k, None)
    assert bool((k == 7.0).all())
    tail = t.full((2, B, H, 32, D), 7.0, dtype=t.bfloat16, device="cuda")
    cg.cg_append(shape, gauge, codec, 0, 3, k, k, tail, pay, meta)
    assert bool((tail == 7.0).all()) and not bool(pay.any()) and bool(meta.isnan().all())


@pytest.mark.parametrize("n", [1, 40])
def test_two_graphs_share_a_workspace(n):
    t = torch()
    cases = [Case4(910 + i, B=3, T=3000, n=n, lengths=[3000, 900 + i, 31], bf16=True).device() for i in range(2)]
    at = [c.attn() for c in cases]
    ws = empty_u8(max(cg.cg_attend_workspace_bytes(c.shape, c.gauge, c.codec, a, True) for c, a in zip(cases, at)))
    want = [c.run(mass=True) for c in cases]
    res, graphs = [], []
    for c, a in zip(cases, at):
        L, B, H, R, _, T, block, g = c.dims
        r = (t.empty_like(c.q), t.empty((B, n, H * R), device="cuda"), t.zeros((L, B, H, c.cap // block), device="cuda"))
        call = lambda c=c, a=a, r=r: cg.cg_attend(c.shape, c.payd, c.metad, c.gauge, c.codec, a, c.q, r[0], r[1], r[2], ws)
        call()
        gr = t.cuda.CUDAGraph()
        with t.cuda.graph(gr):
            call()
        res.append(r)
        graphs.append(gr)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for r in res:
            r[2].zero_()
        ws.fill_(255)
        for i in order:
            res[i][2].zero_()
            graphs[i].replay()
        t.cuda.synchronize()
        for i in set(order):
            for x, y in zip(res[i], want[i]):
                assert t.equal(x, y), (order, i)


def test_a_step_on_another_stream():
    """Rotation, append, attention and read of one step on a stream of its own."""
    t = torch()
    B, H, R, T, n = 2, 2, 4, 256, 40
    gen = t.Generator(device="cuda").manual_seed(5)
    shape = cg.make_shape(1, 2, B, H, T, T, D, cg.CG_DTYPE_BF16)
    codec, gauge = cg.make_codec(cg.CG_BACKEND_KIVI, 4, 32), cg.make_gauge(0)
    rot = cg.make_rotary((10000.0 ** (-t.arange(0, D, 2, device="cuda").double() / D)).float())
    q, k, v = (t.randn(B, n, h, D, generator=gen, device="cuda").to(t.bfloat16) for h in (H * R, H, H))
    lengths = t.tensor([200, 57], dtype=t.int32, device="cuda")
    at = cg.make_attn(0, H * R, n, 0.1, True, lengths)

    def step():
        pay, meta = t.zeros(2 * B * H * T * 64, dtype=t.uint8, device="cuda"), t.zeros(2 * B * H * T * 8, device="cuda")
        tail = t.zeros((2, B, H, 32, D), dtype=t.bfloat16, device="cuda")
        qr, kr, out, kb = t.empty_like(q), t.empty_like(k), t.empty_like(q), t.empty_like(k)
        ws = empty_u8(max(16, cg.cg_attend_workspace_bytes(shape, gauge, codec, at)))
        cg.cg_rotate(shape, rot, q, k, qr, kr, lengths)
        cg.cg_append(shape, gauge, codec, 0, n, kr, v, tail, pay, meta, lengths)
        cg.cg_attend(shape, pay, meta, gauge, codec, at, qr, out, workspace=ws)
        cg.cg_read(shape, pay, meta, gauge, codec, 0, kb, None, lengths)
        return qr, kr, out, kb, pay, meta, tail

    want = step()
    t.cuda.synchronize()
    s = t.cuda.Stream()
    with t.cuda.stream(s):
        got = step()
    s.synchronize()
    for x, y in zip(got, want):
        assert t.equal(x, y)
    assert float((want[3].float() - want[1].float()).abs().max()) < 0.5  # 4 bits of rows of a few units


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("g", [0, 8, 16, 32, 128])
def test_pieces_over_the_ends_of_blocks(g, bf16):
    """Rows that begin in one block and end in another: the raw rows kept are replaced after they have been read."""
    f = Filled4(940 + g, [310, 300, 287, 310], bf16=bf16, H=6, g=g)
    at = 0
    for n in (29, 31, 33, 40, 1, 62, 3, 95, 16):
        lo, at = at, at + n
        f.put(f.x[0][:, lo:at], f.x[1][:, lo:at], n, [min(at, T) for T in f.lengths], [lo] * 4)
    f.check()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("Hq,H,n", [(1, 1, 1), (1, 0, 1), (3, 5, 900), (130, 0, 300), (0, 7, 5000), (61, 1, 600)])
def test_rotation_of_any_number_of_heads(Hq, H, n, bf16):
    """One head to a lane group, or four of a row (past 32768 heads), the last group with fewer."""
    t = torch()
    rng = np.random.default_rng(930 + Hq)
    B = 2
    x = rng.standard_normal((B, n, Hq + H, D)).astype(np.float32)
    xh = oracle.f32_to_bf16(x) if bf16 else x
    x = oracle.to_f32(xh).astype(np.float64)
    w = (1 + 0.2 * rng.standard_normal((2, D))).astype(np.float32)
    freq = (1e4 ** (-np.arange(0, D, 2) / D)).astype(np.float32)
    dev, wd, fd = to_dev(xh), to_dev(w), to_dev(freq)
    shape = cg.make_shape(1, 2, B, max(H, 1), 1 << 20, 1 << 20, D, cg.CG_DTYPE_BF16 if bf16 else cg.CG_DTYPE_F32)
    rot = cg.make_rotary(fd, q_weight=wd[0], k_weight=wd[1], eps=1e-6)
    starts = np.array([5, 70000], np.int32)
    q, k = (dev[:, :, :Hq] if Hq else None), (dev[:, :, Hq:] if H else None)
    qo, ko = (None if y is None else t.full((B, n, y.shape[2], D), 7.0, dtype=y.dtype, device="cuda") for y in (q, k))
    cg.cg_rotate(shape, rot, q, k, qo, ko, None, to_dev(starts))
    pos = (starts[:, None] + np.arange(n))[None]
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    for got, part, wt in ((qo, x[:, :, :Hq], w[0]), (ko, x[:, :, Hq:], w[1])):
        if got is None:
            continue
        y, tol = oracle.serving4.rotate(part, wt, np.float64(np.float32(1e-6)), freq, pos, False)
        err = np.abs(oracle.to_f32(to_host(got)).astype(np.float64) - y)
        assert np.all(err <= tol + half * (np.abs(y) + tol))
