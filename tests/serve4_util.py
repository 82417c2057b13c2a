"""Inputs of the tests of the 4-bit serving cache: random encoded caches, and the
cases of serve_util on them."""
import numpy as np

import oracle
from fixed_rate_compression_amd import binding as cg
from gpu_util import D, to_dev
from serve_util import Case

GROUP = 32


def random_cache4(rng, L, B, H, cap, spread=1.0):
    """payload uint8 [L,2,B,H,cap,64], meta fp32 [L,2,B,H,4 cap,2]: channels and tokens of unlike
    centres and steps."""
    pay = rng.integers(0, 256, (L, 2, B, H, cap, D // 2), dtype=np.uint8)
    st = np.exp(spread * 0.5 * rng.standard_normal((L, 2, B, H, 4 * cap))) * 3.0 / 15
    mn = -st * (7.5 + 4 * rng.standard_normal(st.shape))
    return pay, np.stack([mn, st], -1).astype(np.float32)


class Case4(Case):
    """A 4-bit cache with queries on both sides."""

    def __init__(self, seed, **kw):
        kw.pop("block", None)
        super().__init__(seed, block=GROUP, **kw)
        L, B, H = self.dims[:3]
        self.pay, self.meta = random_cache4(np.random.default_rng(seed + 5), L, B, H, self.cap, kw.get("spread", 1.0))

    def reference(self, one_part=False):
        q = oracle.to_f32(self.qh).astype(np.float64)
        return oracle.serving4.attend(q, self.pay, self.meta, self.G, self.layer, np.float64(np.float32(self.scale)),
                                      self.causal, self.lengths, self.starts, fp32=not self.bf16, one_part=one_part)

    def device(self):
        super().device()
        self.codec = cg.make_codec(cg.CG_BACKEND_KIVI, 4, GROUP)
        self.payd, self.metad = to_dev(self.pay), to_dev(self.meta)
        return self
