"""cg_rotate on the GPU against the fp64 formula: norms, both pairings, partial rotation, several axes, far
positions, padding, strides and in place."""
import numpy as np
import pytest

import oracle
from fixed_rate_compression_amd import binding as cg
from gpu_util import D, to_dev, to_host

pytestmark = pytest.mark.gpu


def torch():
    return __import__("torch")


class Rot:
    def __init__(self, seed, B=2, n=3, Hq=4, H=2, dim=128, norm=True, bf16=True, sections=None, interleaved=False,
                 dealt=False, far=5000, base=1e6, magnitude=1.0, scale=1.0):
        rng = np.random.default_rng(seed)
        self.B, self.n, self.Hq, self.H, self.bf16 = B, n, Hq, H, bf16
        conv = oracle.f32_to_bf16 if bf16 else (lambda x: x)
        sc = np.exp(0.5 * rng.standard_normal((Hq + H, D))).astype(np.float32) * np.float32(scale)
        x = rng.standard_normal((B, n, Hq + H, D)).astype(np.float32) * sc
        self.qh, self.kh = conv(np.ascontiguousarray(x[:, :, :Hq])), conv(np.ascontiguousarray(x[:, :, Hq:]))
        self.q, self.k = to_dev(self.qh), to_dev(self.kh)
        self.freq = (base ** (-np.arange(0, dim, 2) / max(dim, 1))).astype(np.float32)
        self.w = (1 + 0.3 * rng.standard_normal((2, D))).astype(np.float32) if norm else (None, None)
        self.sections, self.interleaved, self.dealt, self.magnitude, self.eps = sections, interleaved, dealt, magnitude, 1e-6
        self.starts = rng.integers(0, far, B).astype(np.int32)
        axes = len(sections) if sections else 1
        self.pos = rng.integers(-far, far, (axes, B, n)).astype(np.int32) if axes > 1 else None
        self.shape = cg.make_shape(1, 2, B, H, 1 << 40, 1 << 40, D, cg.CG_DTYPE_BF16 if bf16 else cg.CG_DTYPE_F32)

    def rotary(self):
        dev = lambda x: None if x is None else to_dev(np.ascontiguousarray(x))
        return cg.make_rotary(dev(self.freq), self.sections, self.interleaved, self.dealt, dev(self.w[0]), dev(self.w[1]),
                              self.eps, self.magnitude)

    def run(self, q=None, k=None, qo=None, ko=None, lengths=None, positions="own"):
        t = torch()
        q, k = self.q if q is None else q, self.k if k is None else k
        qo = t.full_like(self.q, 7.0) if qo is None else qo
        ko = t.full_like(self.k, 7.0) if ko is None else ko
        pos = self.pos if isinstance(positions, str) else positions
        cg.cg_rotate(self.shape, self.rotary(), q, k, qo, ko, None if lengths is None else t.tensor(lengths, dtype=t.int32, device="cuda"),
                     to_dev(self.starts), None if pos is None else to_dev(pos))
        return qo, ko

    def places(self):
        return (self.starts[:, None].astype(np.int64) + np.arange(self.n))[None] if self.pos is None else self.pos

    def check(self, got, there=None):
        for x, h, w in ((got[0], self.qh, self.w[0]), (got[1], self.kh, self.w[1])):
            ref, tol = oracle.serving4.rotate(oracle.to_f32(h), w, self.eps, self.freq, self.places(), self.interleaved,
                                              self.sections, self.dealt, self.magnitude)
            y = oracle.to_f32(to_host(x)).astype(np.float64)
            half = 2.0 ** -8 if self.bf16 else 2.0 ** -24
            bad = np.abs(y - ref) > tol + half * (np.abs(ref) + tol)
            keep = np.ones(ref.shape[:2], bool) if there is None else there
            assert not bad[keep].any(), float((np.abs(y - ref) - tol)[keep].max())
            assert np.all(y[~keep] == 7.0)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dim", [0, 16, 32, 64, 96, 112, 128])
def test_pairs_and_partial_rotation(bf16, norm, interleaved, dim):
    r = Rot(10 + dim, dim=dim, norm=norm, bf16=bf16, interleaved=interleaved)
    r.check(r.run())


@pytest.mark.parametrize("B,n,Hq,H", [(1, 1, 1, 1), (1, 1, 32, 8), (3, 1, 5, 1), (2, 37, 7, 7), (1, 300, 16, 2), (64, 1, 12, 4)])
@pytest.mark.parametrize("bf16", [True, False])
def test_head_layouts_and_lengths(B, n, Hq, H, bf16):
    r = Rot(30 + n, B=B, n=n, Hq=Hq, H=H, bf16=bf16)
    r.check(r.run())


@pytest.mark.parametrize("sections,dealt,dim", [([32, 32], False, 128), ([16, 24, 24], False, 128), ([24, 20, 20], True, 128),
                                                ([16, 16, 16, 16], True, 128), ([16, 16, 16, 16], False, 128), ([0, 16], False, 32),
                                                ([8, 4, 4], True, 32), ([48, 0, 0], True, 96), ([1, 62, 1], False, 128),
                                                ([22, 21, 21], True, 128)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_axes(sections, dealt, dim, interleaved):
    for bf16 in (True, False):
        r = Rot(50, n=21, sections=sections, dealt=dealt, dim=dim, interleaved=interleaved, bf16=bf16)
        r.check(r.run())


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 1000])
def test_far_positions(far):
    """An angle of 2^31 radians is as good as a small one."""
    r = Rot(60, n=5, far=far, bf16=False, sections=[30, 34])
    r.check(r.run())
    r = Rot(61, n=5, far=min(far, (1 << 30) - 10), bf16=False, norm=False)
    r.check(r.run())


def test_magnitude_and_frequencies_of_any_size():
    r = Rot(70, bf16=False, magnitude=1.37)
    r.check(r.run())
    r = Rot(71, bf16=False, norm=False)
    r.freq = np.array([0.0, -1.0, 3.0, 1e-30, 100.0] + [0.5] * 59, np.float32)
    r.check(r.run())


def test_zero_rows_and_small_ones():
    """eps carries a row of zeros; rows far below and above 1 (the squares stay in fp32)."""
    for scale in (0.0, 1e-15, 1e15):
        r = Rot(75, bf16=False, scale=scale)
        r.eps = 0.0 if scale > 1 else 1e-6
        r.check(r.run())


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("n", [1, 6])
def test_in_place_in_a_fused_projection(bf16, n):
    """Queries and keys turned where they lie; values and the rest of the rows stay."""
    t = torch()
    r = Rot(80, B=3, n=n, Hq=6, H=2, bf16=bf16)
    wide = t.full((3, n, 6 + 2 + 2 + 1, D), 5.0, dtype=r.q.dtype, device="cuda")
    wide[:, :, :6], wide[:, :, 6:8] = r.q, r.k
    q, k = wide[:, :, :6], wide[:, :, 6:8]
    r.run(q, k, q, k)
    r.check((q, k))
    assert bool((wide[:, :, 8:] == 5.0).all())
    # out of rows of one width into rows of another
    wide[:, :, :6], wide[:, :, 6:8] = r.q, r.k
    other = t.full((3, n, 9, D), 7.0, dtype=r.q.dtype, device="cuda")
    r.check(r.run(q, k, other[:, :, 3:9], other[:, :, 1:3]))
    assert bool((other[:, :, :1] == 7.0).all()) and t.equal(q, r.q)


def test_padding_rows_stay():
    r = Rot(85, B=4, n=9)
    r.starts = np.array([0, -4, 100, 20], np.int32)
    lengths = [5, 3, 100, 400]
    p = r.starts[:, None] + np.arange(9)
    there = (p >= 0) & (p < np.array(lengths)[:, None])
    r.check(r.run(lengths=lengths), there)
    t = torch()
    r.q[t.from_numpy(~there).cuda()] = float("nan")
    r.check(r.run(lengths=lengths), there)


def test_default_place_is_the_last_rows():
    t = torch()
    r = Rot(86, B=3, n=4)
    ln = t.tensor([10, 4, 300], dtype=t.int32, device="cuda")
    qo, ko = t.full_like(r.q, 7.0), t.full_like(r.k, 7.0)
    cg.cg_rotate(r.shape, r.rotary(), r.q, r.k, qo, ko, ln)
    r.starts = np.array([6, 0, 296], np.int32)
    r.check((qo, ko))


def test_queries_or_keys_alone():
    t = torch()
    r = Rot(87)
    both = r.run()
    qo, ko = t.empty_like(r.q), t.empty_like(r.k)
    cg.cg_rotate(r.shape, r.rotary(), r.q, None, qo, None, starts=to_dev(r.starts))
    cg.cg_rotate(r.shape, r.rotary(), None, r.k, None, ko, starts=to_dev(r.starts))
    assert t.equal(qo, both[0]) and t.equal(ko, both[1])


def test_captured_rotation():
    t = torch()
    r = Rot(88, B=2, n=2)
    st, rot = to_dev(r.starts), r.rotary()
    qo, ko = t.empty_like(r.q), t.empty_like(r.k)
    call = lambda: cg.cg_rotate(r.shape, rot, r.q, r.k, qo, ko, starts=st)
    call()
    gr = t.cuda.CUDAGraph()
    with t.cuda.graph(gr):
        call()
    for s in ([0, 5], [100000, 7], [1, 2]):
        r.starts = np.array(s, np.int32)
        st.copy_(t.tensor(s, dtype=t.int32))
        qo.zero_()
        gr.replay()
        r.check((qo, ko))
