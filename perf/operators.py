"""Cases and plain forms of the serving operators of the 8-bit block-uniform cache.

The cache is the library's block-uniform payload at 8 bits: one byte a value in
gauged coordinates, one (minimum, step) pair for each block of `block` tokens of
a field (layer, K/V, sequence, head), so value = minimum + step * code.

  append   new K/V rows of every sequence are gauged, quantized and put into the
           blocks they fall in; the raw rows of the current block stay beside it
  attend   softmax(scale (G_K q) . k') v' over a sequence's rows, then G_V^T, for
           one to many queries a sequence and grouped heads; optionally the log
           of each row's sum, and the weight each block of tokens received
  evict    each head keeps its first and last blocks and those that received the
           most weight, up to a budget; the cache is compacted

run() computes them with elementary torch operations, or with the library's
entry points where `own` is set.
"""
import math
import random

import torch

own = False

D = 128
NEG = float("-inf")


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _attend(name, batch, heads, ratio, tokens, n=1, dtype="bf16", block=32, group=16, layers=1, ragged=False,
            prompt=False, causal=True, lse=False, mass=False):
    return {"name": name, "op": "attend", "batch": batch, "heads": heads, "ratio": ratio, "tokens": tokens, "n": n,
            "dtype": dtype, "block": block, "group": group, "layers": layers, "ragged": ragged, "prompt": prompt,
            "causal": causal, "lse": lse, "mass": mass}


def _append(name, batch, heads, tokens, n=1, dtype="bf16", block=32, group=16, ragged=True, prompt=False):
    return {"name": name, "op": "append", "batch": batch, "heads": heads, "tokens": tokens, "n": n, "dtype": dtype,
            "block": block, "group": group, "ragged": ragged, "prompt": prompt}


def _evict(name, layers, batch, heads, tokens, budget, sink, recent, block=32, ragged=False):
    return {"name": name, "op": "evict", "layers": layers, "batch": batch, "heads": heads, "tokens": tokens,
            "budget": budget, "sink": sink, "recent": recent, "block": block, "ragged": ragged}


def listed():
    return [
        # one sequence, a short history, one new token: the latency of a chat's first answers
        _attend("token-1x1k", 1, 8, 4, 1024),
        # a serving batch at unlike lengths, one new token each
        _attend("token-16x8k-ragged", 16, 8, 4, 8192, ragged=True, lse=True),
        # one long document
        _attend("token-1x256k", 1, 8, 4, 262144 - 77, block=64),
        # fp32 storage, five query heads a KV head, the smaller blocks, the second of two layers
        _attend("token-f32-8x4k", 8, 4, 5, 4001, dtype="f32", block=16, group=32, layers=2, lse=True),
        # a chunk of a prompt against the history before it
        _attend("chunk-2048-of-8k", 1, 8, 4, 8192, n=2048),
        # several drafted tokens a sequence to be checked, full-head gauge, a head layout without groups
        _attend("draft-9-5x3000", 5, 16, 1, 3000, n=9, group=128, ragged=True),
        # one new token each, with the weight every block received
        _attend("token-weights-8x16k", 8, 8, 4, 16384, ragged=True, lse=True, mass=True),
        # right-padded prompts from their first token on, with the weights
        _attend("prompt-weights-2x1000", 2, 8, 4, 1000, n=1000, ragged=True, prompt=True, lse=True, mass=True),
        # a token for each of 64 sequences at unlike lengths
        _append("append-64x1", 64, 8, 2048),
        # right-padded prompts into an empty cache
        _append("append-4x2000", 4, 8, 2000, n=2000, block=64, prompt=True),
        # half of every head's blocks leave a 32-layer cache
        _evict("evict-32x8k-half", 32, 1, 8, 8192, 128, 1, 2),
        # few blocks out of many, the smaller blocks, unlike lengths
        _evict("evict-4x4x40k", 4, 4, 8, 40000, 256, 4, 16, block=16, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["token", "token", "many", "append", "evict"])
    block = rng.choice([16, 32, 64])
    if op == "token":
        tokens = _log_int(rng, 40, 131072)
        batch = _log_int(rng, 1, max(1, min(48, 262144 // tokens)))
        c = _attend("", batch, rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8]), tokens, rng.choice([1, 1, 1, 2, 4]),
                    rng.choice(["bf16", "bf16", "f32"]), block, rng.choice([0, 8, 16, 32, 128]), rng.choice([1, 1, 2]),
                    rng.random() < 0.6, False, True, rng.random() < 0.5, rng.random() < 0.4)
    elif op == "many":
        n = _log_int(rng, 5, 2048)
        prompt = rng.random() < 0.4
        tokens = n if prompt else _log_int(rng, n, max(n + 1, 8192))
        heads, ratio = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
        most = max(1, (2048 * 8192 * 16) // (n * tokens * heads * ratio))
        batch = _log_int(rng, 1, min(8, most))
        c = _attend("", batch, heads, ratio, tokens, n, rng.choice(["bf16", "bf16", "f32"]), block,
                    rng.choice([0, 8, 16, 32, 128]), 1, rng.random() < 0.6, prompt, rng.random() < 0.8,
                    rng.random() < 0.5, rng.random() < 0.4)
    elif op == "append":
        prompt = rng.random() < 0.4
        if prompt:
            n = _log_int(rng, 20, 2048)
            c = _append("", rng.randint(1, 4), rng.choice([1, 2, 4, 8]), n, n, "bf16", block, rng.choice([0, 8, 16, 32]),
                        True, True)
        else:
            c = _append("", _log_int(rng, 1, 64), rng.choice([1, 2, 4, 8]), _log_int(rng, 70, 2048), rng.choice([1, 1, 2, 5]),
                        "bf16", block, rng.choice([0, 8, 16, 32]), rng.random() < 0.7)
    else:
        tokens = _log_int(rng, 500, 32768)
        layers, batch, heads = rng.randint(1, 8), rng.randint(1, 4), rng.choice([1, 2, 4, 8])
        blocks = -(-tokens // block)
        budget = rng.randint(6, max(7, blocks))
        c = _evict("", layers, batch, heads, tokens, budget, rng.randint(0, 2), rng.randint(1, 3), block, rng.random() < 0.6)
    del c["name"]
    return c


# --------------------------------------------------------------------------
# what a program has in hand before the call
# --------------------------------------------------------------------------

def _cap(c):
    return -(-c["tokens"] // c["block"]) * c["block"]


def _lengths(c):
    """Valid rows of each sequence: all of them, or spread with the longest and a single row among them."""
    if not c["ragged"]:
        return [c["tokens"]] * c["batch"]
    r = random.Random(1000003 * c["batch"] + c["tokens"])
    lo = 1 if c.get("prompt") else min(c["tokens"], c.get("n", 1))
    out = [r.randint(lo, c["tokens"]) for _ in range(c["batch"])]
    out[0] = c["tokens"]
    if c["batch"] > 2:
        out[-1] = lo
    return out


def _starts(c):
    """Position of each sequence's first query or new row."""
    return [0] * c["batch"] if c["prompt"] else [n - c["n"] for n in _lengths(c)]


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _gauges(gen, kinds, heads, g):
    """Orthogonal g x g matrices: exponentials of small skew-symmetric ones."""
    a = 0.1 * torch.randn(kinds * heads * (D // g), g, g, generator=gen, device="cuda", dtype=torch.float64)
    return torch.linalg.matrix_exp(a - a.transpose(1, 2)).float().reshape(kinds, heads, D // g, g, g).contiguous()


def _field(gen, tokens, cap, block):
    """Codes and ranges of one field: channels of unlike scales, four of them large."""
    sc = torch.exp(0.4 * torch.randn(D, generator=gen, device="cuda"))
    sc[torch.randint(0, D, (4,), generator=gen, device="cuda")] *= 4.0
    x = torch.randn(cap, D, generator=gen, device="cuda") * sc
    x = x.reshape(cap // block, block * D)
    mn, mx = x.amin(1, keepdim=True), x.amax(1, keepdim=True)
    code = torch.round((x - mn) * (255.0 / (mx - mn))).clamp_(0, 255).to(torch.uint8)
    return code.reshape(cap, D), torch.cat([mn, (mx - mn) / 255.0], 1)


def _cache(gen, c, fields):
    cap, block = _cap(c), c["block"]
    payload = torch.empty(fields, cap, D, dtype=torch.uint8, device="cuda")
    meta = torch.empty(fields, cap // block, 2, device="cuda")
    for f in range(fields):
        if f < 256:
            payload[f], meta[f] = _field(gen, c["tokens"], cap, block)
        else:  # more than enough fields of their own: the others are these again, shifted by some rows
            payload[f], meta[f] = payload[f - 256].roll(block * (f // 256), 0), meta[f - 256].roll(f // 256, 0)
    return payload, meta


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    block, cap, B, H = c["block"], _cap(c), c["batch"], c["heads"]
    ln = _lengths(c)
    s = {"case": c, "lengths": torch.tensor(ln, dtype=torch.int32, device="cuda")}
    if c["op"] == "attend":
        L, n, q_heads = c["layers"], c["n"], H * c["ratio"]
        s["payload"], s["meta"] = _cache(gen, c, L * 2 * B * H)
        s["gauge"] = torch.cat([_gauges(gen, 2, H, c["group"]) for _ in range(L)]).reshape(
            L, 2, H, D // c["group"], c["group"], c["group"]) if c["group"] else None
        # the queries are a part of a fused projection's rows
        qkv = torch.randn(B, n, (q_heads + 2 * H) * D, generator=gen, device="cuda").to(_dtype(c))
        s["q"] = qkv[:, :, : q_heads * D].unflatten(2, (q_heads, D))
        s["out"] = torch.zeros(B, n, q_heads, D, dtype=_dtype(c), device="cuda")
        s["lse"] = torch.zeros(B, n, q_heads, device="cuda") if c["lse"] else None
        s["mass"] = torch.zeros(L, B, H, cap // block, device="cuda") if c["mass"] else None
        s["starts"] = torch.tensor(_starts(c), dtype=torch.int32, device="cuda")
    elif c["op"] == "append":
        n = c["n"]
        s["payload"] = torch.zeros(2 * B * H, cap, D, dtype=torch.uint8, device="cuda")
        s["meta"] = torch.zeros(2 * B * H, cap // block, 2, device="cuda")
        s["gauge"] = _gauges(gen, 2, H, c["group"]).reshape(1, 2, H, D // c["group"], c["group"], c["group"]) if c["group"] else None
        sc = torch.exp(0.4 * torch.randn(2, 1, H, 1, D, generator=gen, device="cuda"))
        s["tail"] = (torch.randn(2, B, H, block, D, generator=gen, device="cuda") * sc).to(_dtype(c))
        new = (torch.randn(2, B, H, n, D, generator=gen, device="cuda") * sc).to(_dtype(c))
        s["k"], s["v"] = new.transpose(2, 3).contiguous().unbind(0)  # [batch][row][head][128]
        s["starts"] = torch.tensor(_starts(c), dtype=torch.int32, device="cuda")
    else:
        L, budget = c["layers"], c["budget"]
        s["payload"], s["meta"] = _cache(gen, c, L * 2 * B * H)
        # a few blocks take most of the weight
        s["mass"] = torch.exp(1.5 * torch.randn(L, B, H, cap // block, generator=gen, device="cuda"))
        s["payload_out"] = torch.zeros(L * 2 * B * H, budget * block, D, dtype=torch.uint8, device="cuda")
        s["meta_out"] = torch.zeros(L * 2 * B * H, budget, 2, device="cuda")
        s["mass_out"] = torch.zeros(L, B, H, budget, device="cuda")
        s["kept"] = torch.zeros(L, B, H, budget, dtype=torch.int32, device="cuda")
        s["lengths_out"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    if own:
        s["plan"] = _plan(s)
    return s


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------

def _plan(s):
    """The descriptors and the workspace that a serving program builds once."""
    from fixed_rate_compression_amd import binding as cg
    c = s["case"]
    dt = cg.CG_DTYPE_BF16 if c.get("dtype", "bf16") == "bf16" else cg.CG_DTYPE_F32
    p = {"cg": cg, "codec": cg.make_codec(cg.CG_BACKEND_BLOCK_UNIFORM, 8, c["block"]),
         "shape": cg.make_shape(c.get("layers", 1), 2, c["batch"], c["heads"], c["tokens"], _cap(c), D, dt)}
    if c["op"] != "evict":
        p["gauge"] = cg.make_gauge(c["group"], s["gauge"])
    if c["op"] == "attend":
        p["attn"] = cg.make_attn(c["layers"] - 1, c["heads"] * c["ratio"], c["n"], 1.0 / math.sqrt(D), c["causal"],
                                 lengths=s["lengths"], starts=s["starts"],
                                 q_strides=(s["q"].stride(0), s["q"].stride(1)))
        need = cg.cg_attend_workspace_bytes(p["shape"], p["gauge"], p["codec"], p["attn"], c["mass"])
        p["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    if c["op"] == "evict":
        p["out_shape"] = cg.make_shape(c["layers"], 2, c["batch"], c["heads"], c["budget"] * c["block"],
                                       c["budget"] * c["block"], D, dt)
    return p


def _own(s):
    c, p = s["case"], s["plan"]
    cg = p["cg"]
    if c["op"] == "attend":
        cg.cg_attend(p["shape"], s["payload"], s["meta"], p["gauge"], p["codec"], p["attn"], s["q"], s["out"],
                     s["lse"], s["mass"], p["ws"])
        return _attend_out(s, s["out"], s["lse"], s["mass"])
    if c["op"] == "append":
        cg.cg_append(p["shape"], p["gauge"], p["codec"], 0, c["n"], s["k"], s["v"], s["tail"], s["payload"],
                     s["meta"], s["lengths"], s["starts"])
        return {"tail": s["tail"], "values": _touched(s, s["payload"], s["meta"])}
    cg.cg_evict(p["shape"], p["codec"], c["budget"], c["sink"], c["recent"], s["mass"], s["payload"], s["meta"],
                p["out_shape"], s["payload_out"], s["meta_out"], s["mass_out"], s["kept"], s["lengths_out"],
                s["lengths"])
    return {"payload": s["payload_out"], "meta": s["meta_out"], "mass": s["mass_out"], "kept": s["kept"],
            "lengths": s["lengths_out"]}


def _attend_out(s, out, lse, mass):
    r = {"out": out}
    if lse is not None:
        r["lse"] = lse
    if mass is not None:
        r["mass"] = mass
    return r


def _touched(s, payload, meta):
    """The values that the appended blocks stand for, in the storage format: the whole cache of a prompt, the last
    block of each field otherwise."""
    c = s["case"]
    block, cap, B, H = c["block"], _cap(c), c["batch"], c["heads"]
    code, m = payload.view(2, B, H, cap // block, block * D), meta.view(2, B, H, cap // block, 2)
    if not c["prompt"]:
        at = ((s["lengths"].long() - 1) // block).view(1, B, 1, 1, 1)
        code = code.take_along_dim(at.expand(2, B, H, 1, block * D), 3)
        m = m.take_along_dim(at.expand(2, B, H, 1, 2), 3)
    return torch.addcmul(m[..., :1], m[..., 1:], code.float()).to(_dtype(c))


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def _dense(g):
    """[heads][D/g][g][g] -> block-diagonal [heads][D][D]."""
    H, r, w, _ = g.shape
    m = g.new_zeros(H, r, w, r, w)
    m.diagonal(dim1=1, dim2=3).copy_(g.permute(0, 2, 3, 1))
    return m.reshape(H, D, D)


def _positions(s, n):
    """Position of each query or new row, and whether the sequence has it: [batch][n]."""
    pos = s["starts"].view(-1, 1) + torch.arange(n, device="cuda", dtype=torch.int32)
    return pos, (pos >= 0) & (pos < s["lengths"].view(-1, 1))


def _plain_attend(s):
    c = s["case"]
    block, cap, B, H, R, n = c["block"], _cap(c), c["batch"], c["heads"], c["ratio"], c["n"]
    layer = c["layers"] - 1
    code = s["payload"].view(c["layers"], 2, B, H, cap // block, block, D)[layer].float()
    m = s["meta"].view(c["layers"], 2, B, H, cap // block, 1, 2)[layer]
    k, v = torch.addcmul(m[..., :1], m[..., 1:], code).reshape(2, B, H, cap, D).unbind(0)
    del code
    q = s["q"].float().reshape(B, n, H, R, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * R, D)
    if c["group"]:
        gk, gv = _dense(s["gauge"][layer, 0]), _dense(s["gauge"][layer, 1])
        q = torch.matmul(q, gk.transpose(1, 2).contiguous())
    sc = torch.matmul(q, k.transpose(2, 3).contiguous()) * (1.0 / math.sqrt(D))
    pos, has = _positions(s, n)
    t = torch.arange(cap, device="cuda", dtype=torch.int32)
    see = (t < s["lengths"].view(B, 1, 1)) & has.view(B, n, 1)
    if c["causal"]:
        see = see & (t <= pos.view(B, n, 1))
    sc = sc.view(B, H, n, R, cap).masked_fill_(~see.view(B, 1, n, 1, cap), NEG).view(B, H, n * R, cap)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc.sub_(torch.where(top == NEG, torch.zeros_like(top), top)))
    l = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(l == 0, torch.ones_like(l), l))
    o = torch.matmul(p, v)
    if c["group"]:
        o = torch.matmul(o, gv)
    o = o.view(B, H, n, R, D).permute(0, 2, 1, 3, 4).reshape(B, n, H * R, D).to(_dtype(c))
    lse = (top + torch.log(l)).view(B, H, n, R).permute(0, 2, 1, 3).reshape(B, n, H * R) if c["lse"] else None
    mass = None
    if c["mass"]:
        s["mass"][layer] += p.view(B, H, n * R, cap // block, block).sum((2, 4))
        mass = s["mass"]
    return _attend_out(s, o, lse, mass)


def _plain_append(s):
    c = s["case"]
    block, cap, B, H, n = c["block"], _cap(c), c["batch"], c["heads"], c["n"]
    nb = cap // block
    new = torch.stack([s["k"], s["v"]]).transpose(2, 3)  # [2][B][H][n][D]
    pos, has = _positions(s, n)
    first = s["starts"].clamp(min=0)
    # raw rows of every block from the first new row's on, as a strip that starts with the tail's block
    head = (first // block) * block
    strip = (n + 2 * block - 1) // block * block
    at = torch.arange(strip, device="cuda", dtype=torch.int32) + head.view(B, 1)      # positions of the strip's rows
    j = (at - s["starts"].view(B, 1)).long()
    is_new = (j >= 0) & (j < n) & (at < s["lengths"].view(B, 1)) & (at >= 0)
    rows = new.take_along_dim(j.clamp(0, n - 1).view(1, B, 1, strip, 1).expand(2, B, H, strip, D), 3)
    old = (at < first.view(B, 1)) & (torch.arange(strip, device="cuda") < block)
    raw = torch.zeros_like(rows)
    raw[..., :block, :] = s["tail"]
    raw = torch.where(is_new.view(1, B, 1, strip, 1), rows, raw)
    valid = (is_new | old).view(1, B, 1, strip, 1)
    x = raw.float()
    if c["group"]:
        g = torch.stack([_dense(s["gauge"][0, 0]), _dense(s["gauge"][0, 1])])
        x = torch.matmul(x, g.transpose(2, 3).contiguous().view(2, 1, H, D, D))
    x = x.unflatten(3, (strip // block, block))
    vb = valid.unflatten(3, (strip // block, block))
    mn = torch.where(vb, x, math.inf).amin((-1, -2), keepdim=True)
    mx = torch.where(vb, x, -math.inf).amax((-1, -2), keepdim=True)
    diff = mx - mn
    inv = torch.where(diff > 0, 255.0 / diff, torch.zeros_like(diff))
    step = torch.where(diff > 0, diff / 255.0, torch.zeros_like(diff))
    code = torch.round((x - mn) * inv).clamp(0, 255)
    # blocks of the strip that hold a new row, back into the cache
    touched = is_new.view(B, strip // block, block).any(-1)
    blk = (head // block).view(B, 1).long() + torch.arange(strip // block, device="cuda")
    b, i = torch.nonzero(touched, as_tuple=True)
    pay, met = s["payload"].view(2, B, H, nb, block, D), s["meta"].view(2, B, H, nb, 2)
    keep = vb.expand_as(code)[:, b, :, i]
    pay[:, b, :, blk[b, i]] = torch.where(keep, code[:, b, :, i].to(torch.uint8), pay[:, b, :, blk[b, i]])
    met[:, b, :, blk[b, i]] = torch.cat([mn, step], -1)[:, b, :, i].squeeze(-2)
    # the raw rows of the last block
    end = torch.minimum(s["lengths"], s["starts"] + n)
    last = ((end - 1).clamp(min=0) // block) * block
    off = (last - head).view(B, 1) + torch.arange(block, device="cuda", dtype=torch.int32)
    idx = off.clamp(0, strip - 1).long().view(1, B, 1, block, 1).expand(2, B, H, block, D)
    fresh = valid.expand(2, B, H, strip, 1).take_along_dim(idx[..., :1], 3) & (end > first).view(1, B, 1, 1, 1)
    s["tail"].copy_(torch.where(fresh, raw.take_along_dim(idx, 3), s["tail"]))
    return {"tail": s["tail"], "values": _touched(s, s["payload"], s["meta"])}


def _plain_evict(s):
    c = s["case"]
    L, B, H, block, budget = c["layers"], c["batch"], c["heads"], c["block"], c["budget"]
    nb = _cap(c) // block
    blocks = ((s["lengths"] + block - 1) // block).view(1, B, 1, 1)
    i = torch.arange(nb, device="cuda", dtype=torch.int32)
    w = torch.where((i < c["sink"]) | (i >= blocks - c["recent"]), torch.full_like(s["mass"], math.inf), s["mass"])
    w = w.masked_fill(i >= blocks, NEG)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
    if nb < budget:
        order = torch.cat([order, order.new_full((L, B, H, budget - nb), nb)], -1)
    order = torch.where(order < blocks, order, nb).sort(-1).values
    has = order < nb
    at = order.clamp(max=nb - 1)
    src = at.unsqueeze(1).expand(L, 2, B, H, budget).unsqueeze(-1)
    both = has.view(L, 1, B, H, budget, 1)
    code = s["payload"].view(L, 2, B, H, nb, block * D).take_along_dim(src.expand(L, 2, B, H, budget, block * D), 4)
    code = torch.where(both, code, torch.zeros_like(code))
    meta = torch.where(both, s["meta"].view(L, 2, B, H, nb, 2).take_along_dim(src.expand(L, 2, B, H, budget, 2), 4), 0.0)
    ln, bl = s["lengths"], blocks.view(B)
    return {"payload": code.view(-1, budget * block, D), "meta": meta.reshape(-1, budget, 2),
            "mass": torch.where(has, s["mass"].take_along_dim(at, 3), 0.0),
            "kept": torch.where(has, order, -1).int(),
            "lengths": torch.where(bl > budget, ln - (bl - budget) * block, ln).int()}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_attend(state) if op == "attend" else _plain_append(state) if op == "append" else _plain_evict(state)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _matrix64(g, h):
    """Head h's groups [D/g][g][g] as one D x D matrix."""
    return torch.block_diag(*g[h].double().unbind(0))


def _exact_attend(c, s):
    block, cap, B, H, R, n = c["block"], _cap(c), c["batch"], c["heads"], c["ratio"], c["n"]
    layer = c["layers"] - 1
    pay = s["payload"].view(c["layers"], 2, B, H, cap, D)[layer]
    met = s["meta"].view(c["layers"], 2, B, H, cap // block, 2)[layer].double()
    out = torch.zeros(B, n, H * R, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, n, H * R), NEG, dtype=torch.float64, device="cuda")
    mass = torch.zeros(c["layers"], B, H, cap // block, dtype=torch.float64, device="cuda")
    lengths, starts = _lengths(c), _starts(c)
    for b in range(B):
        i0, i1 = max(0, -starts[b]), min(n, lengths[b] - starts[b])
        T = lengths[b]
        if i1 <= i0 or T <= 0:
            continue
        for h in range(H):
            kv = []
            for kind in (0, 1):
                mm = met[kind, b, h].repeat_interleave(block, 0)[:T]
                kv.append(mm[:, :1] + mm[:, 1:] * pay[kind, b, h, :T].double())
            x = s["q"][b, i0:i1, h * R:(h + 1) * R].double().reshape(-1, D)
            if c["group"]:
                x = x @ _matrix64(s["gauge"][layer, 0], h).T
            z = (x @ kv[0].T) / math.sqrt(D)
            if c["causal"]:
                p = torch.arange(starts[b] + i0, starts[b] + i1, device="cuda").repeat_interleave(R)
                z[torch.arange(T, device="cuda")[None, :] > p[:, None]] = NEG
            w = torch.softmax(z, -1)
            y = w @ kv[1]
            if c["group"]:
                y = y @ _matrix64(s["gauge"][layer, 1], h)
            out[b, i0:i1, h * R:(h + 1) * R] = y.view(-1, R, D)
            lse[b, i0:i1, h * R:(h + 1) * R] = torch.logsumexp(z, -1).view(-1, R)
            if c["mass"]:
                t = w.sum(0)
                t = torch.cat([t, t.new_zeros(cap - T)]).view(-1, block).sum(1)
                mass[layer, b, h] += t
    return _attend_out(s, out, lse if c["lse"] else None, mass if c["mass"] else None)


def _exact_append(c, s):
    """Each sequence's blocks from its raw rows, one by one; rows that nothing was put into stand for the block's minimum."""
    block, cap, B, H, n = c["block"], _cap(c), c["batch"], c["heads"], c["n"]
    vals = torch.zeros(2, B, H, cap // block, block, D, dtype=torch.float64, device="cuda")
    tail = s["tail"].clone()
    lengths, starts = _lengths(c), _starts(c)
    for b in range(B):
        p0, p1 = max(0, starts[b]), min(starts[b] + n, lengths[b])
        if p1 <= p0:
            continue
        for blk in range(p0 // block, (p1 - 1) // block + 1):
            lo, hi = blk * block, min(p1, (blk + 1) * block)
            parts = [tail[:, b, :, : p0 - lo]] if lo < p0 else []
            parts += [torch.stack([s["k"][b, max(lo, p0) - starts[b]:hi - starts[b]],
                                   s["v"][b, max(lo, p0) - starts[b]:hi - starts[b]]]).transpose(1, 2)]
            raw = torch.cat(parts, 2)
            x = raw.double()
            if c["group"]:
                x = torch.stack([torch.stack([x[kd, h] @ _matrix64(s["gauge"][0, kd], h).T for h in range(H)])
                                 for kd in (0, 1)])
            mn, mx = x.amin((2, 3), keepdim=True), x.amax((2, 3), keepdim=True)
            step = (mx - mn) / 255.0
            y = mn.expand(2, H, block, D).clone()
            y[:, :, : hi - lo] += step * torch.round((x - mn) / step)
            vals[:, b, :, blk] = y
            if blk == (p1 - 1) // block:
                tail[:, b, :, : hi - lo] = raw
    if not c["prompt"]:
        at = torch.tensor([max(0, (x - 1) // block) for x in lengths], device="cuda")
        vals = vals.take_along_dim(at.view(1, B, 1, 1, 1, 1).expand(2, B, H, 1, block, D), 3)
    return {"tail": None, "values": vals.flatten(-2)}


def exact(case, seed):
    c = case
    if c["op"] == "evict" or (c["op"] == "append" and c["dtype"] != "bf16"):
        return None  # moved bytes and whole numbers; codes of fp32 rows turn on the last bit of a value
    s = prepare(case, seed)
    return _exact_attend(c, s) if c["op"] == "attend" else _exact_append(c, s)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    block, B, H, ln = c["block"], c["batch"], c["heads"], _lengths(case)
    row = D + 8.0 / block  # a row of codes and its share of the range
    if c["op"] == "evict":
        kept = sum(min(c["budget"], -(-n // block)) for n in ln)
        nb = sum(-(-n // block) for n in ln)
        L = c["layers"]
        return {"bytes": L * H * (kept * (2.0 * 2 * block * row + 8) + nb * 4), "flops": 0}
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "append":
        rows = sum(max(0, min(s + c["n"], n) - max(0, s)) for s, n in zip(_starts(c), ln))
        # the block that the first row falls into is read from the raw rows and written again
        again = sum((max(0, s) % block) for s in _starts(c))
        return {"bytes": 2.0 * H * ((rows + again) * D * e + (rows + again) * row + rows * D * e),
                "flops": 2.0 * H * (rows + again) * D * (2 * c["group"] + 4)}
    R, n = c["ratio"], c["n"]
    seen = keys = rows = 0
    for s, T in zip(_starts(c), ln):
        i0, i1 = max(0, -s), min(n, T - s)
        if i1 <= i0:
            continue
        rows += i1 - i0
        keys += T if not c["causal"] else min(T, s + i1)
        seen += (i1 - i0) * T if not c["causal"] else sum(range(s + i0 + 1, s + i1 + 1))
    return {"bytes": 2.0 * H * keys * row + 2.0 * rows * H * R * D * e + (rows * H * R * 4.0 if c["lse"] else 0)
            + (2.0 * H * keys / block * 4.0 if c["mass"] else 0),
            "flops": H * R * (4.0 * D * seen + 4.0 * D * c["group"] * rows)}
