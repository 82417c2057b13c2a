"""Inputs of the serving tests: random encoded caches, gauges and queries."""
import numpy as np

import oracle
from fixed_rate_compression_amd import binding as cg
from gpu_util import D, gauges_for, to_dev, to_host


def random_cache(rng, L, B, H, cap, block, spread=1.0):
    """payload uint8 [L,2,B,H,cap,128], meta fp32 [L,2,B,H,cap/block,2]: blocks of
    unlike centres and steps."""
    pay = rng.integers(0, 256, (L, 2, B, H, cap, D), dtype=np.uint8)
    st = np.exp(spread * rng.standard_normal((L, 2, B, H, cap // block))) * 2.0 / 255
    mn = -st * (127 + 30 * rng.standard_normal(st.shape))
    return pay, np.stack([mn, st], -1).astype(np.float32)


class Case:
    """A cache with queries on both sides (host arrays and device tensors)."""

    def __init__(self, seed, L=1, B=2, H=2, R=4, n=1, T=100, cap=None, block=32, g=16, bf16=True,
                 lengths=None, starts=None, causal=True, scale=None, layer=0, qscale=1.0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.cap = cap or -(-T // block) * block
        self.dims = (L, B, H, R, n, T, block, g)
        self.bf16, self.causal, self.layer = bf16, causal, layer
        self.scale = 1 / np.sqrt(D) if scale is None else scale
        self.pay, self.meta = random_cache(rng, L, B, H, self.cap, block, spread)
        self.G = gauges_for(seed + 1, L, 2, H, g)
        q = (qscale * rng.standard_normal((B, n, H * R, D))).astype(np.float32)
        self.qh = oracle.f32_to_bf16(q) if bf16 else q
        self.lengths = [T] * B if lengths is None else list(lengths)
        self.starts = starts

    def reference(self, one_part=False):
        L, B, H, R, n, T, block, g = self.dims
        q = oracle.to_f32(self.qh).astype(np.float64)
        return oracle.serving.attend(q, self.pay, self.meta, self.G, self.layer, block, np.float64(np.float32(self.scale)),
                                     self.causal, self.lengths, self.starts, fp32=not self.bf16, one_part=one_part)

    def device(self):
        t = __import__("torch")
        L, B, H, R, n, T, block, g = self.dims
        self.shape = cg.make_shape(L, 2, B, H, T, self.cap, D, cg.CG_DTYPE_BF16 if self.bf16 else cg.CG_DTYPE_F32)
        self.codec = cg.make_codec(cg.CG_BACKEND_BLOCK_UNIFORM, 8, block)
        self.gauge = cg.make_gauge(g, to_dev(np.ascontiguousarray(self.G)) if g else None)
        self.payd, self.metad, self.q = to_dev(self.pay), to_dev(self.meta), to_dev(self.qh)
        self.len_d = t.tensor(self.lengths, dtype=t.int32, device="cuda")
        self.st_d = None if self.starts is None else t.tensor(self.starts, dtype=t.int32, device="cuda")
        return self

    def attn(self, strides=(0, 0), n=None):
        L, B, H, R, nq, T, block, g = self.dims
        return cg.make_attn(self.layer, H * R, nq if n is None else n, float(self.scale), self.causal, self.len_d,
                            self.st_d, strides)

    def run(self, lse=True, mass=True, q=None, strides=(0, 0), stream=None):
        """-> (out, lse, mass) device tensors; guard rows behind the outputs are checked by check()."""
        t = __import__("torch")
        L, B, H, R, n, T, block, g = self.dims
        at = self.attn(strides)
        out = t.full_like(self.q, 7.0).contiguous()
        ls = t.full((B, n, H * R), 7.0, device="cuda") if lse else None
        ms = t.zeros((L, B, H, self.cap // block), device="cuda") if mass else None
        need = cg.cg_attend_workspace_bytes(self.shape, self.gauge, self.codec, at, mass)
        # stale contents: nothing in a workspace is taken for granted
        ws = t.full((max(need, 16) // 4,), float("nan"), device="cuda")
        cg.cg_attend(self.shape, self.payd, self.metad, self.gauge, self.codec, at, self.q if q is None else q, out,
                     ls, ms, ws, stream)
        return out, ls, ms


FEW = 64         # rows (queries times heads of a group) of the few-row form at most


def form(case, mass):
    """(rows of a KV head, whether the few-row form takes them, splits) of a case with one
    sequence, read off the workspace it asks for."""
    L, B, H, R, n, T, block, g = case.dims
    assert B == 1
    at = case.attn()
    need = cg.cg_attend_workspace_bytes(case.shape, case.gauge, case.codec, at, mass)
    rows = n * R
    up = lambda x: -(-x // 256) * 256
    if mass:
        need -= up(H * rows * 8 * (case.cap // min(block, 32)))
    found = set()
    for few in (True, False):
        for splits in range(1, 1025):
            parts = H * rows * splits
            size = up(parts * 512) + up(parts * 8) if splits > 1 else up(parts * 8) if few and mass else 0
            if not few and mass:
                size += up(H * rows * 4)
            if size == need and few == (rows <= FEW):
                found.add((rows, few, splits))
    assert len(found) == 1, (need, found)
    return found.pop()


def check_outputs(case):
    """The case with no optional output, the log-sums, and those with the blocks' weights,
    each within the bounds of the variant that then runs."""
    L, B, H, R, n, T, block, g = case.dims
    two = case.reference()
    one = case.reference(one_part=True) if case.bf16 and n * R > FEW else two
    check(case, case.run(lse=False, mass=False), one, "out")
    check(case, case.run(lse=True, mass=False), two, "out, lse")
    check(case, case.run(lse=True, mass=True), two, "out, lse, mass")
    return two


def check(case, got, ref=None, where=None):
    out, lse, mass = got
    ref = ref or case.reference()
    o = oracle.to_f32(to_host(out)).astype(np.float64)
    half = 2.0 ** -8 if case.bf16 else 2.0 ** -24
    err, bound = np.abs(o - ref["out"]), ref["out_tol"] + half * (np.abs(ref["out"]) + ref["out_tol"])
    assert np.all(np.isfinite(o)), where
    assert np.all(err <= bound), (where, float((err - bound).max()), np.argwhere(err > bound)[:4].tolist())
    if lse is not None:
        x = to_host(lse).astype(np.float64)
        none = np.isneginf(ref["lse"])
        assert np.array_equal(np.isneginf(x), none), where
        d = np.abs(x[~none] - ref["lse"][~none]) - ref["lse_tol"][~none]
        assert np.all(d <= 0), (where, float(d.max()))
    if mass is not None:
        x = to_host(mass).astype(np.float64)
        for l in range(x.shape[0]):
            if l != case.layer:
                assert not x[l].any(), (where, l)
        d = np.abs(x[case.layer] - ref["mass"])
        assert np.all(d <= ref["mass_tol"]), (where, float((d - ref["mass_tol"]).max()))
