"""An 8-bit block-uniform cache that is served from where it lies: new K/V rows
go in token by token (cg_append), attention reads the codes (cg_attend), and the
blocks that received the least attention leave (cg_evict).

One step of a decoder, the same for prompts, chunks of them and single tokens:

    cache.begin(n)                      # every sequence grows by n rows
    for layer in range(layers):
        cache.append(layer, k, v)       # k, v [batch, n, heads, 128] after RoPE, of the same strides
        o = cache.attend(layer, q)      # q, o [batch, n, q_heads, 128]

begin(n, valid) takes right-padded rows: sequence b gets the first valid[b] of
them (the host's bound of the lengths counts all n).  Sequences have their own
lengths, on the device; nothing here waits for them, so a step may be recorded
into a graph and replayed (the host's bound, which refuses a step that cannot
fit, does not see replays: rows past the capacity are dropped).

Attention is planned for sequences as long as the capacity (a recorded step has to
serve them at any length), so a capacity far above what is there costs splits and
a merge: with 8 KV heads x 4 query heads a token over 1000 takes 13 us at a capacity
of 131072 and 11 at 1024, a prompt of 300 tokens 32 us from 1024 on and 18.5 at 320, four
prompts of 1000 with weights 93 us up to 32768 (1000 MiB of workspace there, 32 at 1024)
and 213 at 131072.

Sequences grow by steps and shrink by evict() alone: only the raw rows of a sequence's
last block are kept, so rows that were appended (drafts that were not accepted) cannot
be taken back by setting `lengths`.

All arithmetic runs in the HIP library; this class only owns buffers.  A cache
belongs to one stream at a time.
"""
from __future__ import annotations

from . import binding as cg


class ServingCache:
    def __init__(self, layers, batch, heads, q_heads, capacity, gauge, block_tokens=32,
                 dtype=cg.CG_DTYPE_BF16, head_dim=128, with_mass=False):
        import torch

        if capacity < 0 or block_tokens <= 0 or capacity % block_tokens:
            raise ValueError("capacity must be a multiple of block_tokens")
        self.codec = cg.make_codec(cg.CG_BACKEND_BLOCK_UNIFORM, 8, block_tokens)
        self.shape = cg.make_shape(layers, 2, batch, heads, capacity, capacity, head_dim, dtype)
        self.gauge, self.q_heads = gauge, q_heads
        self.dtype = torch.bfloat16 if dtype == cg.CG_DTYPE_BF16 else torch.float32
        pay, meta, _ = cg.cg_encoded_bytes(self.shape, self.codec)
        dev = {"device": "cuda"}
        self.payload = torch.zeros(pay, dtype=torch.uint8, **dev)
        self.meta = torch.zeros(meta // 4, **dev)
        self.tail = torch.zeros((layers, 2, batch, heads, block_tokens, head_dim), dtype=self.dtype, **dev)
        self.mass = torch.zeros((layers, batch, heads, capacity // block_tokens), **dev) if with_mass else None
        self.lengths = torch.zeros(batch, dtype=torch.int32, **dev)
        self.starts = torch.zeros(batch, dtype=torch.int32, **dev)   # of the present step
        self._counts = (torch.int32, torch.int64)                    # types of a step's valid rows
        self.n = 0                                                   # rows of the present step
        self._put = set()                                            # layers that have them
        self.most = 0                                                # no sequence is longer
        self._need = {}                                              # workspace bytes by queries a step
        self._work = []                                              # workspaces, growing; none is freed: a
                                                                     # recorded step may use it

    def begin(self, n, valid=None):
        """A step of n rows a sequence; valid: device int32 [batch], rows that are there (or None: all)."""
        if n < 0:
            raise ValueError("n < 0")
        if self.most + n > self.shape.token_capacity:
            raise ValueError(f"{n} rows do not fit: up to {self.most} of {self.shape.token_capacity} are taken")
        if valid is not None:     # before anything changes: a refused step has not begun
            at = self.lengths
            if getattr(valid, "dtype", None) not in self._counts or valid.shape != at.shape or \
                    valid.device != at.device:
                raise ValueError("valid must be int32 [batch] beside the cache")
            valid = valid.clamp(0, n)
        self.n = n
        self._put.clear()
        self.most += n
        self.starts.copy_(self.lengths)
        if valid is None:
            self.lengths.add_(n)
        else:
            self.lengths.add_(valid)

    def append(self, layer, k, v):
        """The step's rows of one layer, before that layer's attend; every layer once a step (only
        the raw rows of a sequence's last block are kept, which may be another by then)."""
        if layer in self._put:
            raise ValueError(f"layer {layer} has the step's rows")
        cg.cg_append(self.shape, self.gauge, self.codec, layer, self.n, k, v, self.tail, self.payload, self.meta,
                     self.lengths, self.starts)
        self._put.add(layer)

    def attend(self, layer, q, scale=None, causal=True, out=None, lse=None):
        """Attention of the step's queries; gathers the blocks' weights where the cache has them."""
        import torch

        if out is None:
            out = torch.empty(q.shape, dtype=self.dtype, device=q.device)
        at = cg.make_attn(layer, self.q_heads, self.n, self.shape.head_dim ** -0.5 if scale is None else scale, causal,
                          self.lengths, self.starts,
                          tuple(q.stride(d) if q.shape[d] > 1 else 0 for d in (0, 1)))   # of one row: any
        need = self._need.get(self.n)
        if need is None:
            need = self._need[self.n] = cg.cg_attend_workspace_bytes(self.shape, self.gauge, self.codec, at,
                                                                     self.mass is not None)
        if not self._work or self._work[-1].numel() < need:
            size = max(need, 16, self._work[-1].numel() * 3 // 2 if self._work else 0)
            self._work.append(torch.empty(size, dtype=torch.uint8, device=self.payload.device))
        cg.cg_attend(self.shape, self.payload, self.meta, self.gauge, self.codec, at, q, out, lse, self.mass,
                     self._work[-1])
        return out

    def evict(self, budget, sink=1, recent=1):
        """Keep `budget` blocks of every (layer, sequence, head), in place; -> the kept blocks' former numbers.

        Between steps: the rows' positions change, so the present step ends here."""
        import torch

        if self.mass is None:
            raise ValueError("the cache was made without with_mass")
        s = self.shape
        kept = torch.empty((s.layers, s.batch, s.heads, max(budget, 0)), dtype=torch.int32, device=self.payload.device)
        cg.cg_evict(s, self.codec, budget, sink, recent, self.mass, self.payload, self.meta, s, self.payload, self.meta,
                    self.mass, kept, self.lengths, self.lengths)
        self.most = min(self.most, budget * self.codec.block_tokens)
        self.n = 0
        return kept
