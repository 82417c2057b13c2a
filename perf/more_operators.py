"""Cases and plain forms of the operators of a cache held in 4 bits, and of those beside it.

The 4-bit cache is the library's KIVI-style payload: two codes a byte in gauged coordinates, keys
with one (minimum, step) pair for 32 tokens of a channel, values with one for 32 channels of a
token, so value = minimum + step * code.

  attend   softmax(scale (G_K q) . k') v' over a sequence's rows, then G_V^T, for one to many
           queries a sequence and grouped heads; optionally the log of each row's sum, and the
           weight each 32-token block received
  append   new K/V rows of every sequence are gauged, quantized and put into the blocks they fall
           in (the raw rows of the current block stay beside the cache), and the rows of those
           blocks are read back
  read     rows of every sequence of a layer, decoded and turned back, 4-bit and 8-bit caches
  evict    each head keeps its first and last blocks and those of the most weight, up to a budget
  rotate   queries and keys of a fused projection: a norm of each head, then the rotation by the
           row's position, or by its positions on several axes (time, height, width)

run() computes them with elementary torch operations, or with the library's entry points where
`own` is set.
"""
import math
import random

import torch

own = False

D = 128
GROUP = 32  # tokens of a key range, channels of a value range
NEG = float("-inf")


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _attend(name, batch, heads, ratio, tokens, n=1, dtype="bf16", group=16, layers=1, ragged=False, prompt=False,
            causal=True, lse=False, mass=False):
    return {"name": name, "op": "attend", "batch": batch, "heads": heads, "ratio": ratio, "tokens": tokens, "n": n,
            "dtype": dtype, "group": group, "layers": layers, "ragged": ragged, "prompt": prompt, "causal": causal,
            "lse": lse, "mass": mass}


def _append(name, batch, heads, tokens, n=1, dtype="bf16", group=16, ragged=True, prompt=False):
    return {"name": name, "op": "append", "batch": batch, "heads": heads, "tokens": tokens, "n": n, "dtype": dtype,
            "group": group, "ragged": ragged, "prompt": prompt}


def _read(name, batch, heads, tokens, n, bits=4, dtype="bf16", group=16, layers=1, ragged=False):
    return {"name": name, "op": "read", "batch": batch, "heads": heads, "tokens": tokens, "n": n, "bits": bits,
            "dtype": dtype, "group": group, "layers": layers, "ragged": ragged, "prompt": False}


def _evict(name, layers, batch, heads, tokens, budget, sink, recent, ragged=False):
    return {"name": name, "op": "evict", "layers": layers, "batch": batch, "heads": heads, "tokens": tokens,
            "budget": budget, "sink": sink, "recent": recent, "ragged": ragged}


def _rotate(name, batch, heads, ratio, n, far, dtype="bf16", norm=True, dim=D, axes=1, interleaved=False, dealt=False):
    return {"name": name, "op": "rotate", "batch": batch, "heads": heads, "ratio": ratio, "n": n, "far": far,
            "dtype": dtype, "norm": norm, "dim": dim, "axes": axes, "interleaved": interleaved, "dealt": dealt}


def listed():
    return [
        # one sequence, a short history, one new token: the latency of a chat's first answers
        _attend("token4-1x1k", 1, 8, 4, 1024),
        # a serving batch at unlike lengths, one new token each, with log-sums
        _attend("token4-16x8k-ragged", 16, 8, 4, 8192, ragged=True, lse=True),
        # one long document, the second of two layers
        _attend("token4-1x256k", 1, 8, 4, 262144 - 77, layers=2),
        # a chunk of a prompt against the history before it
        _attend("chunk4-2048-of-8k", 1, 8, 4, 8192, n=2048),
        # a token for each of 64 sequences at unlike lengths
        _append("append4-64x1", 64, 8, 2048),
        # right-padded prompts into an empty cache
        _append("append4-4x2000", 4, 8, 2000, n=2000, prompt=True),
        # the last 1000 rows of a few sequences for a consumer of plain rows
        _read("read4-3x1000", 3, 8, 5000, 1000, ragged=True),
        # a whole layer of the 8-bit cache, to be moved to another format
        _read("read8-1x128k", 1, 8, 131072, 131072, bits=8, group=32),
        # half of every head's blocks leave a 32-layer cache
        _evict("evict4-32x8k-half", 32, 1, 8, 8192, 128, 1, 2),
        # few blocks out of many, unlike lengths
        _evict("evict4-4x4x40k", 4, 4, 8, 40000, 128, 2, 8, ragged=True),
        # a decoding step of 64 sequences, far into long documents
        _rotate("rotate-64x1", 64, 8, 4, 1, 1 << 20),
        # prompts with images in them: positions on three axes
        _rotate("rotate-2x4000-3axes", 2, 8, 4, 4000, 8000, axes=3),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["token", "token", "many", "append", "read", "evict", "rotate"])
    if op == "token":
        tokens = _log_int(rng, 40, 131072)
        batch = _log_int(rng, 1, max(1, min(48, 262144 // tokens)))
        c = _attend("", batch, rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8]), tokens, rng.choice([1, 1, 1, 2, 4]),
                    rng.choice(["bf16", "bf16", "f32"]), rng.choice([0, 8, 16, 32, 128]), rng.choice([1, 1, 2]),
                    rng.random() < 0.6, False, True, rng.random() < 0.5, rng.random() < 0.4)
    elif op == "many":
        n = _log_int(rng, 5, 2048)
        prompt = rng.random() < 0.4
        tokens = n if prompt else _log_int(rng, n, max(n + 1, 8192))
        heads, ratio = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
        most = max(1, (2048 * 8192 * 16) // (n * tokens * heads * ratio))
        batch = _log_int(rng, 1, min(8, most))
        c = _attend("", batch, heads, ratio, tokens, n, rng.choice(["bf16", "bf16", "f32"]),
                    rng.choice([0, 8, 16, 32, 128]), 1, rng.random() < 0.6, prompt, rng.random() < 0.8,
                    rng.random() < 0.5, rng.random() < 0.4)
    elif op == "append":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if rng.random() < 0.4:
            n = _log_int(rng, 20, 2000)
            c = _append("", rng.randint(1, 4), rng.choice([1, 2, 4, 8]), n, n, dtype, rng.choice([0, 16]), True, True)
        else:
            c = _append("", _log_int(rng, 1, 64), rng.choice([1, 2, 4, 8]), _log_int(rng, 70, 2048), rng.choice([1, 1, 2, 5]),
                        dtype, rng.choice([0, 16]), rng.random() < 0.7)
    elif op == "read":
        tokens = _log_int(rng, 40, 32768)
        batch = _log_int(rng, 1, max(1, min(16, 131072 // tokens)))
        c = _read("", batch, rng.choice([1, 2, 4, 8]), tokens, _log_int(rng, 1, tokens), rng.choice([4, 4, 8]),
                  rng.choice(["bf16", "bf16", "f32"]), rng.choice([0, 8, 16, 32, 128]), rng.choice([1, 2]), rng.random() < 0.6)
    elif op == "evict":
        tokens = _log_int(rng, 500, 32768)
        layers, batch, heads = rng.randint(1, 8), rng.randint(1, 4), rng.choice([1, 2, 4, 8])
        budget = rng.randint(6, max(7, -(-tokens // GROUP)))
        c = _evict("", layers, batch, heads, tokens, budget, rng.randint(0, 2), rng.randint(1, 3), rng.random() < 0.6)
    else:
        n = _log_int(rng, 1, 4000)
        c = _rotate("", _log_int(rng, 1, max(1, min(64, 8000 // n))), rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 5]), n,
                    _log_int(rng, 5000, 1 << 21), rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.7,
                    rng.choice([32, 64, 96, 128, 128]), rng.choice([1, 1, 2, 3]), rng.random() < 0.3, rng.random() < 0.4)
    del c["name"]
    return c


# --------------------------------------------------------------------------
# what a program has in hand before the call
# --------------------------------------------------------------------------

def _cap(c):
    return -(-c["tokens"] // GROUP) * GROUP


def _lengths(c):
    """Valid rows of each sequence: all of them, or spread with the longest and a single row among them."""
    if not c["ragged"]:
        return [c["tokens"]] * c["batch"]
    r = random.Random(1000003 * c["batch"] + c["tokens"])
    lo = 1 if c.get("prompt") or c["op"] in ("read", "evict") else min(c["tokens"], c["n"])
    out = [r.randint(lo, c["tokens"]) for _ in range(c["batch"])]
    out[0] = c["tokens"]
    if c["batch"] > 2:
        out[-1] = lo
    return out


def _starts(c):
    """Position of each sequence's first query, new row or row that is read: the last n of them, or all from the first."""
    return [0] * c["batch"] if c["prompt"] else [n - c["n"] for n in _lengths(c)]


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _gauges(gen, kinds, heads, g):
    """Orthogonal g x g matrices: exponentials of small skew-symmetric ones."""
    a = 0.1 * torch.randn(kinds * heads * (D // g), g, g, generator=gen, device="cuda", dtype=torch.float64)
    return torch.linalg.matrix_exp(a - a.transpose(1, 2)).float().reshape(kinds, heads, D // g, g, g).contiguous()


def _hadamard16(kinds, heads):
    """The control gauge of 16 channels: entries +-1/4."""
    h = torch.ones(1, 1, device="cuda")
    for _ in range(4):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return (h / 4).expand(kinds, heads, D // 16, 16, 16).contiguous()


def _scales(gen, shape):
    """Channels of unlike scales, four of them large."""
    sc = torch.exp(0.4 * torch.randn(*shape, D, generator=gen, device="cuda"))
    at = torch.randint(0, D, (*shape, 4), generator=gen, device="cuda")
    return sc.scatter(-1, at, sc.gather(-1, at) * 4.0)


def _ranges(x, axes, top):
    """Codes and (minimum, step) of the ranges over `axes` of x."""
    mn, mx = x.amin(axes, keepdim=True), x.amax(axes, keepdim=True)
    code = torch.round((x - mn) * (top / (mx - mn))).clamp_(0, top).to(torch.uint8)
    return code, torch.stack([mn, (mx - mn) / top], -1)


def _cache4(gen, c, L, B, H):
    """payload [L][2][B][H][cap][64] of two codes a byte, meta [L][2][B][H][4 cap][2]."""
    cap = _cap(c)
    payload = torch.empty(L * 2 * B * H, cap, D // 2, dtype=torch.uint8, device="cuda")
    meta = torch.empty(L * 2 * B * H, 4 * cap, 2, device="cuda")
    for f in range(L * 2 * B * H):
        if f < 256:
            x = torch.randn(cap, D, generator=gen, device="cuda") * _scales(gen, ())
            if (f // (B * H)) % 2 == 0:
                code, m = _ranges(x.view(cap // GROUP, GROUP, D), (1,), 15)
            else:
                code, m = _ranges(x.view(cap, D // GROUP, GROUP), (2,), 15)
            code = code.view(cap, D // 2, 2)
            payload[f], meta[f] = code[..., 0] | code[..., 1] << 4, m.view(4 * cap, 2)
        else:  # more than enough fields of their own: the others are these again, shifted by some blocks
            k = f // 256
            g = f - 256 * k if (f // (B * H)) % 2 == ((f - 256 * k) // (B * H)) % 2 else (f - 256 * k + B * H) % 256
            payload[f], meta[f] = payload[g].roll(GROUP * k, 0), meta[g].roll(4 * GROUP * k, 0)
    return payload, meta


def _cache8(gen, c, L, B, H):
    """payload [L][2][B][H][cap][128], meta [L][2][B][H][cap / 32][2]."""
    cap = _cap(c)
    payload = torch.empty(L * 2 * B * H, cap, D, dtype=torch.uint8, device="cuda")
    meta = torch.empty(L * 2 * B * H, cap // GROUP, 2, device="cuda")
    for f in range(L * 2 * B * H):
        code, m = _ranges((torch.randn(cap, D, generator=gen, device="cuda") * _scales(gen, ())).view(cap // GROUP, -1), (1,), 255)
        payload[f], meta[f] = code.view(cap, D), m.view(-1, 2)
    return payload, meta


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "rotate":
        _prepare_rotate(s, gen)
    else:
        cap, B, H = _cap(c), c["batch"], c["heads"]
        s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
        if c["op"] != "evict":
            s["starts"] = torch.tensor(_starts(c), dtype=torch.int32, device="cuda")
        if c["op"] in ("attend", "read"):
            L = c["layers"]
            s["payload"], s["meta"] = (_cache8 if c.get("bits") == 8 else _cache4)(gen, c, L, B, H)
            s["gauge"] = torch.cat([_gauges(gen, 2, H, c["group"]) for _ in range(L)]).reshape(
                L, 2, H, D // c["group"], c["group"], c["group"]) if c["group"] else None
        if c["op"] == "attend":
            n, q_heads = c["n"], H * c["ratio"]
            # the queries are a part of a fused projection's rows
            qkv = torch.randn(B, n, (q_heads + 2 * H) * D, generator=gen, device="cuda").to(_dtype(c))
            s["q"] = qkv[:, :, : q_heads * D].unflatten(2, (q_heads, D))
            s["out"] = torch.zeros(B, n, q_heads, D, dtype=_dtype(c), device="cuda")
            s["lse"] = torch.zeros(B, n, q_heads, device="cuda") if c["lse"] else None
            s["mass"] = torch.zeros(L, B, H, cap // GROUP, device="cuda") if c["mass"] else None
        elif c["op"] == "read":
            s["k"], s["v"] = torch.zeros(2, B, c["n"], H, D, dtype=_dtype(c), device="cuda").unbind(0)
        elif c["op"] == "append":
            _prepare_append(s, gen)
        else:
            L, budget = c["layers"], c["budget"]
            s["payload"], s["meta"] = _cache4(gen, c, L, B, H)
            # a few blocks take most of the weight
            s["mass"] = torch.exp(1.5 * torch.randn(L, B, H, cap // GROUP, generator=gen, device="cuda"))
            s["payload_out"] = torch.zeros(L * 2 * B * H, budget * GROUP, D // 2, dtype=torch.uint8, device="cuda")
            s["meta_out"] = torch.zeros(L * 2 * B * H, 4 * budget * GROUP, 2, device="cuda")
            s["mass_out"] = torch.zeros(L, B, H, budget, device="cuda")
            s["kept"] = torch.zeros(L, B, H, budget, dtype=torch.int32, device="cuda")
            s["lengths_out"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    if own:
        s["plan"] = _plan(s)
    return s


def _strip(c):
    """Rows that are read back: from the first new row's block on."""
    return (c["n"] + 2 * GROUP - 1) // GROUP * GROUP


def _prepare_append(s, gen):
    """Rows of the storage format on a grid of 2^-6, and the Hadamard gauge: every gauged value is exact in fp32 in
    whatever order it is summed, so a code does not turn on its last bit."""
    c = s["case"]
    cap, B, H, n = _cap(c), c["batch"], c["heads"], c["n"]
    s["payload"] = torch.zeros(2 * B * H, cap, D // 2, dtype=torch.uint8, device="cuda")
    s["meta"] = torch.zeros(2 * B * H, 4 * cap, 2, device="cuda")
    s["gauge"] = _hadamard16(2, H).unsqueeze(0).contiguous() if c["group"] else None
    sc = _scales(gen, (2, 1, H, 1))
    def rows(m):
        return (torch.round(torch.randn(2, B, H, m, D, generator=gen, device="cuda") * sc * 64) / 64).to(_dtype(c))
    s["tail"] = rows(GROUP)
    s["k"], s["v"] = rows(n).transpose(2, 3).contiguous().unbind(0)  # [batch][row][head][128]
    first = s["starts"].clamp(min=0) // GROUP * GROUP
    s["first"] = first
    s["k_back"], s["v_back"] = torch.zeros(2, B, _strip(c), H, D, dtype=_dtype(c), device="cuda").unbind(0)


def _prepare_rotate(s, gen):
    c = s["case"]
    B, n, H, Hq, dt = c["batch"], c["n"], c["heads"], c["heads"] * c["ratio"], _dtype(c)
    qkv = torch.randn(B, n, (Hq + 2 * H) * D, generator=gen, device="cuda") * torch.exp(
        0.5 * torch.randn((Hq + 2 * H) * D, generator=gen, device="cuda"))
    qkv = qkv.to(dt)
    s["q"], s["k"] = qkv[:, :, : Hq * D].unflatten(2, (Hq, D)), qkv[:, :, Hq * D: (Hq + H) * D].unflatten(2, (H, D))
    s["q_out"] = torch.zeros(B, n, Hq, D, dtype=dt, device="cuda")
    s["k_out"] = torch.zeros(B, n, H, D, dtype=dt, device="cuda")
    s["freq"] = (1e6 ** (-torch.arange(0, c["dim"], 2, device="cuda", dtype=torch.float64) / c["dim"])).float()
    s["weights"] = (1 + 0.2 * torch.randn(2, D, generator=gen, device="cuda")).unbind(0) if c["norm"] else (None, None)
    s["starts"] = torch.randint(0, max(1, c["far"] - n), (B,), generator=gen, device="cuda", dtype=torch.int32)
    s["positions"] = None
    if c["axes"] > 1:  # stretches of text, on all axes alike, and of images, whose rows and columns run on two of them
        at = s["starts"].view(1, B, 1) + torch.arange(n, device="cuda", dtype=torch.int32)
        side = 24
        cell = torch.arange(n, device="cuda", dtype=torch.int32) % (side * side)
        image = (torch.arange(n, device="cuda") // (side * side)) % 2 == 1
        p = at.expand(c["axes"], B, n).clone()
        p[0] = torch.where(image, p[0] - cell, p[0])
        p[1] = torch.where(image, p[1] - cell + cell // side, p[1])
        if c["axes"] > 2:
            p[2] = torch.where(image, p[2] - cell + cell % side, p[2])
        s["positions"] = p.contiguous()


def _sections(c):
    """Pairs of channels that each axis turns: the first axis a little less than the others."""
    pairs, axes = c["dim"] // 2, c["axes"]
    each = pairs * 3 // (3 * axes - 1) if axes > 1 and not c["dealt"] else pairs // axes
    return [pairs - each * (axes - 1)] + [each] * (axes - 1)


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------

def _plan(s):
    """The descriptors and the workspace that a serving program builds once."""
    from fixed_rate_compression_amd import binding as cg
    c = s["case"]
    dt = cg.CG_DTYPE_BF16 if c.get("dtype", "bf16") == "bf16" else cg.CG_DTYPE_F32
    if c["op"] == "rotate":
        return {"cg": cg, "shape": cg.make_shape(1, 2, c["batch"], c["heads"], c["far"], c["far"], D, dt),
                "rotary": cg.make_rotary(s["freq"], sections=_sections(c), interleaved=c["interleaved"], dealt=c["dealt"],
                                         q_weight=s["weights"][0], k_weight=s["weights"][1], eps=1e-6)}
    p = {"cg": cg, "shape": cg.make_shape(c.get("layers", 1), 2, c["batch"], c["heads"], c["tokens"], _cap(c), D, dt),
         "codec": cg.make_codec(cg.CG_BACKEND_BLOCK_UNIFORM, 8, GROUP) if c.get("bits") == 8 else
         cg.make_codec(cg.CG_BACKEND_KIVI, 4, GROUP)}
    if c["op"] != "evict":
        p["gauge"] = cg.make_gauge(c["group"], s["gauge"])
    if c["op"] == "attend":
        p["attn"] = cg.make_attn(c["layers"] - 1, c["heads"] * c["ratio"], c["n"], 1.0 / math.sqrt(D), c["causal"],
                                 lengths=s["lengths"], starts=s["starts"],
                                 q_strides=(s["q"].stride(0), s["q"].stride(1)))
        need = cg.cg_attend_workspace_bytes(p["shape"], p["gauge"], p["codec"], p["attn"], c["mass"])
        p["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    if c["op"] == "evict":
        p["out_shape"] = cg.make_shape(c["layers"], 2, c["batch"], c["heads"], c["budget"] * GROUP, c["budget"] * GROUP, D, dt)
    return p


def _own(s):
    c, p = s["case"], s["plan"]
    cg = p["cg"]
    if c["op"] == "rotate":
        cg.cg_rotate(p["shape"], p["rotary"], s["q"], s["k"], s["q_out"], s["k_out"], starts=s["starts"],
                     positions=s["positions"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "attend":
        cg.cg_attend(p["shape"], s["payload"], s["meta"], p["gauge"], p["codec"], p["attn"], s["q"], s["out"],
                     s["lse"], s["mass"], p["ws"])
        return _attend_out(s["out"], s["lse"], s["mass"])
    if c["op"] == "append":
        cg.cg_append(p["shape"], p["gauge"], p["codec"], 0, c["n"], s["k"], s["v"], s["tail"], s["payload"],
                     s["meta"], s["lengths"], s["starts"])
        cg.cg_read(p["shape"], s["payload"], s["meta"], p["gauge"], p["codec"], 0, s["k_back"], s["v_back"],
                   s["lengths"], s["first"])
        return {"tail": s["tail"], "k": s["k_back"], "v": s["v_back"]}
    if c["op"] == "read":
        cg.cg_read(p["shape"], s["payload"], s["meta"], p["gauge"], p["codec"], c["layers"] - 1, s["k"], s["v"],
                   s["lengths"], s["starts"])
        return {"k": s["k"], "v": s["v"]}
    cg.cg_evict(p["shape"], p["codec"], c["budget"], c["sink"], c["recent"], s["mass"], s["payload"], s["meta"],
                p["out_shape"], s["payload_out"], s["meta_out"], s["mass_out"], s["kept"], s["lengths_out"],
                s["lengths"])
    return {"payload": s["payload_out"], "meta": s["meta_out"], "mass": s["mass_out"], "kept": s["kept"],
            "lengths": s["lengths_out"]}


def _attend_out(out, lse, mass):
    r = {"out": out}
    if lse is not None:
        r["lse"] = lse
    if mass is not None:
        r["mass"] = mass
    return r


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
    """Position of each query or row, and whether the sequence has it: [batch][n]."""
    pos = s["starts"].view(-1, 1) + torch.arange(n, device="cuda", dtype=torch.int32)
    return pos, (pos >= 0) & (pos < s["lengths"].view(-1, 1))


def _decoded(s, layer):
    """The layer's values in gauged coordinates: keys and values [B][H][cap][D] in fp32."""
    c = s["case"]
    cap, B, H, L = _cap(c), c["batch"], c["heads"], c.get("layers", 1)
    if c.get("bits") == 8:
        code = s["payload"].view(L, 2, B, H, cap // GROUP, GROUP, D)[layer].float()
        m = s["meta"].view(L, 2, B, H, cap // GROUP, 1, 2)[layer]
        return (m[..., :1] + m[..., 1:] * code).reshape(2, B, H, cap, D).unbind(0)
    byte = s["payload"].view(L, 2, B, H, cap, D // 2)[layer]
    code = torch.stack([byte & 15, byte >> 4], -1).float()
    mk = s["meta"].view(L, 2, B, H, cap // GROUP, 1, D, 2)[layer, 0]
    mv = s["meta"].view(L, 2, B, H, cap, D // GROUP, 1, 2)[layer, 1]
    k = mk[..., 0] + mk[..., 1] * code[0].view(B, H, cap // GROUP, GROUP, D)
    v = mv[..., 0] + mv[..., 1] * code[1].view(B, H, cap, D // GROUP, GROUP)
    return k.reshape(B, H, cap, D), v.reshape(B, H, cap, D)


def _plain_attend(s):
    c = s["case"]
    cap, B, H, R, n = _cap(c), c["batch"], c["heads"], c["ratio"], c["n"]
    layer = c["layers"] - 1
    k, v = _decoded(s, layer)
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
        s["mass"][layer] += p.view(B, H, n * R, cap // GROUP, GROUP).sum((2, 4))
        mass = s["mass"]
    return _attend_out(o, lse, mass)


def _rows_back(s, layer, first, n, into):
    """Rows first .. first + n of every sequence, turned back, where it has them (the others as they are in `into`)."""
    c = s["case"]
    B, H, cap = c["batch"], c["heads"], _cap(c)
    pos = first.view(B, 1) + torch.arange(n, device="cuda", dtype=torch.int32)
    has = ((pos >= 0) & (pos < s["lengths"].view(B, 1))).view(B, n, 1, 1)
    idx = pos.clamp(0, cap - 1).long().view(B, 1, n, 1).expand(B, H, n, D)
    out = []
    for kind, x in enumerate(_decoded(s, layer)):
        x = x.take_along_dim(idx, 2)
        if c["group"]:
            x = torch.matmul(x, _dense(s["gauge"][layer, kind]))
        out.append(torch.where(has, x.transpose(1, 2).to(_dtype(c)), into[kind]))
    return out


def _plain_read(s):
    k, v = _rows_back(s, s["case"]["layers"] - 1, s["starts"], s["case"]["n"], (s["k"], s["v"]))
    return {"k": k, "v": v}


def _fresh(x, keep, axes):
    """Codes and ranges over `axes` of the rows that are there, in the encoder's fp32 operations."""
    mn = torch.where(keep, x, math.inf).amin(axes, keepdim=True)
    mx = torch.where(keep, x, -math.inf).amax(axes, keepdim=True)
    diff, top = mx - mn, torch.full_like(mx, 15.0)  # quotients of tensors: by a number torch multiplies with its inverse
    inv = torch.where(diff > 0, top / diff, torch.zeros_like(diff))
    step = torch.where(diff > 0, diff / top, torch.zeros_like(diff))
    return torch.round((x - mn) * inv).clamp(0, 15).to(torch.uint8), mn, step


def _plain_append(s):
    c = s["case"]
    cap, B, H, n = _cap(c), c["batch"], c["heads"], c["n"]
    nb = cap // GROUP
    new = torch.stack([s["k"], s["v"]]).transpose(2, 3)  # [2][B][H][n][D]
    # raw rows of every block from the first new row's on, as a strip that starts with the tail's block
    first, strip, head = s["starts"].clamp(min=0), _strip(c), s["first"]
    ns = strip // GROUP
    at = torch.arange(strip, device="cuda", dtype=torch.int32) + head.view(B, 1)      # positions of the strip's rows
    j = (at - s["starts"].view(B, 1)).long()
    is_new = (j >= 0) & (j < n) & (at < s["lengths"].view(B, 1)) & (at >= 0)
    rows = new.take_along_dim(j.clamp(0, n - 1).view(1, B, 1, strip, 1).expand(2, B, H, strip, D), 3)
    old = (at < first.view(B, 1)) & (torch.arange(strip, device="cuda") < GROUP)
    raw = torch.zeros_like(rows)
    raw[..., :GROUP, :] = s["tail"]
    raw = torch.where(is_new.view(1, B, 1, strip, 1), rows, raw)
    valid = (is_new | old).view(B, 1, strip, 1)
    x = raw.float()
    if c["group"]:
        g = torch.stack([_dense(s["gauge"][0, 0]), _dense(s["gauge"][0, 1])])
        x = torch.matmul(x, g.transpose(2, 3).contiguous().view(2, 1, H, D, D))
    vb = valid.view(B, 1, ns, GROUP, 1)
    kc, kmn, kst = _fresh(x[0].unflatten(2, (ns, GROUP)), vb, (3,))
    vc, vmn, vst = _fresh(x[1].unflatten(3, (D // GROUP, GROUP)), torch.ones_like(valid).unsqueeze(-1), (4,))
    # blocks of the strip that hold a new row, back into the cache; their rows that are there
    touched = is_new.view(B, ns, GROUP).any(-1)
    blk = (head // GROUP).view(B, 1).long() + torch.arange(ns, device="cuda")
    b, i = torch.nonzero(touched, as_tuple=True)
    to = blk[b, i]
    pay = s["payload"].view(2, B, H, nb, GROUP, D // 2)
    for kind, code in enumerate((kc, vc.reshape(B, H, ns, GROUP, D))):
        byte = code[..., 0::2] | code[..., 1::2] << 4
        keep = vb.expand_as(byte)[b, :, i]
        pay[kind, b, :, to] = torch.where(keep, byte[b, :, i], pay[kind, b, :, to])
    mk = s["meta"].view(2, B, H, nb, D, 2)[0]
    mk[b, :, to] = torch.stack([kmn, kst], -1)[b, :, i].squeeze(2)
    mv = s["meta"].view(2, B, H, nb, GROUP, D // GROUP, 2)[1]
    fresh = torch.stack([vmn, vst], -1).squeeze(4).unflatten(2, (ns, GROUP))
    mv[b, :, to] = torch.where(vb.unsqueeze(-1)[b, :, i], fresh[b, :, i], mv[b, :, to])
    # the raw rows of the last block
    end = torch.minimum(s["lengths"], s["starts"] + n)
    last = ((end - 1).clamp(min=0) // GROUP) * GROUP
    off = (last - head).view(B, 1) + torch.arange(GROUP, device="cuda", dtype=torch.int32)
    idx = off.clamp(0, strip - 1).long().view(1, B, 1, GROUP, 1).expand(2, B, H, GROUP, D)
    there = valid.unsqueeze(0).expand(2, B, H, strip, 1).take_along_dim(idx[..., :1], 3) & (end > first).view(1, B, 1, 1, 1)
    s["tail"].copy_(torch.where(there, raw.take_along_dim(idx, 3), s["tail"]))
    k, v = _rows_back(s, 0, head, strip, (s["k_back"], s["v_back"]))
    return {"tail": s["tail"], "k": k, "v": v}


def _plain_evict(s):
    c = s["case"]
    L, B, H, budget = c["layers"], c["batch"], c["heads"], c["budget"]
    nb = _cap(c) // GROUP
    blocks = ((s["lengths"] + GROUP - 1) // GROUP).view(1, B, 1, 1)
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

    def moved(x):
        x = x.view(L, 2, B, H, nb, -1)
        x = x.take_along_dim(src.expand(*src.shape[:-1], x.shape[-1]), 4)
        return torch.where(both, x, torch.zeros_like(x))
    ln, bl = s["lengths"], blocks.view(B)
    return {"payload": moved(s["payload"]).view(-1, budget * GROUP, D // 2),
            "meta": moved(s["meta"]).view(-1, 4 * budget * GROUP, 2),
            "mass": torch.where(has, s["mass"].take_along_dim(at, 3), 0.0),
            "kept": torch.where(has, order, -1).int(),
            "lengths": torch.where(bl > budget, ln - (bl - budget) * GROUP, ln).int()}


def _axis_of_pairs(c):
    """The axis whose position turns each pair of channels."""
    pairs, sec = c["dim"] // 2, _sections(c)
    if not c["dealt"]:
        return [a for a, m in enumerate(sec) for _ in range(m)]
    return [i % c["axes"] if i < c["axes"] * sec[i % c["axes"]] else 0 for i in range(pairs)]


def _plain_rotate(s):
    c = s["case"]
    B, n, dim = c["batch"], c["n"], c["dim"]
    if s["positions"] is None:
        pos = (s["starts"].view(B, 1) + torch.arange(n, device="cuda", dtype=torch.int32)).view(B, n, 1)
    else:
        pos = s["positions"][torch.tensor(_axis_of_pairs(c), device="cuda")].permute(1, 2, 0)
    angle = pos.double() * s["freq"].double()
    cos, sin = torch.cos(angle).float().unsqueeze(2), torch.sin(angle).float().unsqueeze(2)
    out = {}
    for name, w in (("q", s["weights"][0]), ("k", s["weights"][1])):
        x = s[name].float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        if c["interleaved"]:
            a, b = x[..., 0:dim:2], x[..., 1:dim:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., : dim // 2], x[..., dim // 2: dim]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        out[name] = torch.cat([y, x[..., dim:]], -1).to(_dtype(c))
    return out


def run(state):
    if own:
        return _own(state)
    return {"attend": _plain_attend, "append": _plain_append, "read": _plain_read, "evict": _plain_evict,
            "rotate": _plain_rotate}[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _matrix64(g, h):
    """Head h's groups [D/g][g][g] as one D x D matrix."""
    return torch.block_diag(*g[h].double().unbind(0))


def _field64(c, s, layer, kind, b, h, t0, t1):
    """Gauged values of rows [t0, t1) of a field."""
    cap, B, H, L = _cap(c), c["batch"], c["heads"], c.get("layers", 1)
    f = ((layer * 2 + kind) * B + b) * H + h
    t = torch.arange(t0, t1, device="cuda")
    ch = torch.arange(D, device="cuda")
    if c.get("bits") == 8:
        code, m = s["payload"].view(-1, cap, D)[f, t0:t1].double(), s["meta"].view(-1, cap // GROUP, 2)[f].double()[t // GROUP]
        return m[:, :1] + m[:, 1:] * code
    byte = s["payload"].view(-1, cap, D // 2)[f, t0:t1][:, ch // 2].int()
    code = torch.where(ch % 2 == 0, byte % 16, byte // 16).double()
    pair = s["meta"].view(-1, 4 * cap, 2)[f].double()
    m = pair[(t // GROUP).view(-1, 1) * D + ch] if kind == 0 else pair[t.view(-1, 1) * 4 + ch // GROUP]
    return m[..., 0] + m[..., 1] * code


def _exact_attend(c, s):
    cap, B, H, R, n = _cap(c), c["batch"], c["heads"], c["ratio"], c["n"]
    layer = c["layers"] - 1
    out = torch.zeros(B, n, H * R, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, n, H * R), NEG, dtype=torch.float64, device="cuda")
    mass = torch.zeros(c["layers"], B, H, cap // GROUP, dtype=torch.float64, device="cuda")
    lengths, starts = _lengths(c), _starts(c)
    for b in range(B):
        i0, i1 = max(0, -starts[b]), min(n, lengths[b] - starts[b])
        T = lengths[b]
        if i1 <= i0 or T <= 0:
            continue
        for h in range(H):
            k, v = (_field64(c, s, layer, kind, b, h, 0, T) for kind in (0, 1))
            x = s["q"][b, i0:i1, h * R:(h + 1) * R].double().reshape(-1, D)
            if c["group"]:
                x = x @ _matrix64(s["gauge"][layer, 0], h).T
            z = (x @ k.T) / math.sqrt(D)
            if c["causal"]:
                p = torch.arange(starts[b] + i0, starts[b] + i1, device="cuda").repeat_interleave(R)
                z[torch.arange(T, device="cuda")[None, :] > p[:, None]] = NEG
            w = torch.softmax(z, -1)
            y = w @ v
            if c["group"]:
                y = y @ _matrix64(s["gauge"][layer, 1], h)
            out[b, i0:i1, h * R:(h + 1) * R] = y.view(-1, R, D)
            lse[b, i0:i1, h * R:(h + 1) * R] = torch.logsumexp(z, -1).view(-1, R)
            if c["mass"]:
                t = w.sum(0)
                mass[layer, b, h] += torch.cat([t, t.new_zeros(cap - T)]).view(-1, GROUP).sum(1)
    return _attend_out(out, lse if c["lse"] else None, mass if c["mass"] else None)


def _exact_read(c, s):
    B, H, n, layer = c["batch"], c["heads"], c["n"], c["layers"] - 1
    out = torch.zeros(2, B, n, H, D, dtype=torch.float64, device="cuda")
    lengths, starts = _lengths(c), _starts(c)
    for b in range(B):
        p0, p1 = max(0, starts[b]), min(starts[b] + n, lengths[b])
        if p1 <= p0:
            continue
        for kind in (0, 1):
            for h in range(H):
                x = _field64(c, s, layer, kind, b, h, p0, p1)
                if c["group"]:
                    x = x @ _matrix64(s["gauge"][layer, kind], h)
                out[kind, b, p0 - starts[b]:p1 - starts[b], h] = x
    return {"k": out[0], "v": out[1]}


def _exact_append(c, s):
    """Each sequence's blocks from its raw rows, one by one, turned back where the sequence has the row.  A code is
    defined by its operations in fp32 (many values lie half way between two codes), what it stands for is not."""
    B, H, n, strip = c["batch"], c["heads"], c["n"], _strip(c)
    out = torch.zeros(2, B, strip, H, D, dtype=torch.float64, device="cuda")
    lengths, starts = _lengths(c), _starts(c)
    for b in range(B):
        p0, p1 = max(0, starts[b]), min(starts[b] + n, lengths[b])
        if p1 <= p0:
            continue
        head = p0 // GROUP * GROUP
        for blk in range(p0 // GROUP, (p1 - 1) // GROUP + 1):
            lo, hi = blk * GROUP, min(p1, (blk + 1) * GROUP)
            for kind, new in ((0, s["k"]), (1, s["v"])):
                raw = [s["tail"][kind, b, :, : p0 - lo]] if lo < p0 else []
                raw += [new[b, max(lo, p0) - starts[b]:hi - starts[b]].transpose(0, 1)]
                x = torch.cat(raw, 1).double()
                if c["group"]:
                    x = torch.stack([x[h] @ _matrix64(s["gauge"][0, kind], h).T for h in range(H)])
                z = x if kind == 0 else x.unflatten(2, (D // GROUP, GROUP))
                ax = 1 if kind == 0 else 3
                mn, mx = z.amin(ax, keepdim=True), z.amax(ax, keepdim=True)
                z, mn, diff = z.float(), mn.float(), mx.float() - mn.float()
                top = torch.full_like(diff, 15.0)
                code = torch.where(diff > 0, torch.round((z - mn) * (top / diff)), 0.0)
                y = (mn.double() + (diff / top).double() * code.double()).reshape(H, hi - lo, D)
                if c["group"]:
                    y = torch.stack([y[h] @ _matrix64(s["gauge"][0, kind], h) for h in range(H)])
                out[kind, b, lo - head:hi - head] = y.transpose(0, 1)
    return {"tail": None, "k": out[0], "v": out[1]}


def _exact_rotate(c, s):
    """Each pair of channels as a complex number, times the point of the circle that its angle names."""
    B, n, dim = c["batch"], c["n"], c["dim"]
    axis = _axis_of_pairs(c)
    turn = torch.empty(B, n, 1, dim // 2, dtype=torch.complex128, device="cuda")
    for i in range(dim // 2):
        p = s["starts"].view(B, 1).double() + torch.arange(n, device="cuda") if s["positions"] is None else s["positions"][axis[i]]
        turn[:, :, 0, i] = torch.polar(torch.ones(B, n, dtype=torch.float64, device="cuda"), p.double() * float(s["freq"][i]))
    first = torch.arange(0, dim, 2) if c["interleaved"] else torch.arange(dim // 2)
    second = first + (1 if c["interleaved"] else dim // 2)
    out = {}
    for name, w in (("q", s["weights"][0]), ("k", s["weights"][1])):
        y = s[name].double()
        if w is not None:
            y = y / torch.sqrt((y.square().sum(-1, keepdim=True)) / D + 1e-6) * w.double()
        z = torch.complex(y[..., first.cuda()], y[..., second.cuda()]) * turn
        y = y.clone()
        y[..., first.cuda()], y[..., second.cuda()] = z.real, z.imag
        out[name] = y
    return out


def exact(case, seed):
    if case["op"] == "evict":
        return None  # moved bytes and whole numbers
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "read": _exact_read, "rotate": _exact_rotate}[case["op"]](case, s)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def _bytes(rows, bits=4):
    """Bytes of that many rows of a field from a block's start on, codes and ranges."""
    blocks = -(-rows // GROUP)
    return (rows * D // 2 + blocks * D * 8, rows * D // 2 + rows * 32) if bits == 4 else (rows * D + blocks * 8,) * 2


def work(case):
    c = case
    B, H = c["batch"], c["heads"]
    e = 4 if c.get("dtype") == "f32" else 2
    if c["op"] == "rotate":
        rows = B * c["n"]
        heads = rows * H * (c["ratio"] + 1)
        return {"bytes": 2.0 * heads * D * e + 4.0 * (rows * c["axes"] if c["axes"] > 1 else B), "flops": heads * (3.0 * c["dim"] + 4 * D)}
    ln = _lengths(c)
    if c["op"] == "evict":
        kept = sum(min(c["budget"], -(-n // GROUP)) for n in ln)
        nb = sum(-(-n // GROUP) for n in ln)
        return {"bytes": c["layers"] * H * (kept * (2.0 * sum(_bytes(GROUP)) + 8) + nb * 4), "flops": 0}
    if c["op"] == "read":
        got = [(max(0, p), min(p + c["n"], n)) for p, n in zip(_starts(c), ln)]
        got = [(a, b) for a, b in got if b > a]
        rows = sum(b - a for a, b in got)
        moved = sum(sum(_bytes(b - a, c["bits"])) for a, b in got)
        return {"bytes": H * (moved + 2.0 * rows * D * e), "flops": 2.0 * H * rows * D * (2 * c["group"] + 2)}
    if c["op"] == "append":
        got = [(max(0, p), min(p + c["n"], n)) for p, n in zip(_starts(c), ln)]
        got = [(a, b, a // GROUP * GROUP) for a, b in got if b > a]
        rows, again = sum(b - a for a, b, _ in got), sum(a - h for a, b, h in got)
        tail = sum(min(b - a, (b - 1) % GROUP + 1) for a, b, _ in got)
        moved = sum(_bytes(b - h)[0] + _bytes(b - a)[1] for a, b, h in got)
        back = 2.0 * (rows + again) * D * e  # the rows of the touched blocks; what they hold is on the chip
        return {"bytes": H * (2.0 * rows * D * e + again * D * e + 2.0 * tail * D * e + moved + back),
                "flops": 2.0 * H * (rows + again) * D * (4 * c["group"] + 6)}
    R, n = c["ratio"], c["n"]
    seen = rows = 0
    moved = blocks = 0
    for p, T in zip(_starts(c), ln):
        i0, i1 = max(0, -p), min(n, T - p)
        if i1 <= i0:
            continue
        rows += i1 - i0
        keys = T if not c["causal"] else min(T, p + i1)
        moved += sum(_bytes(keys))
        blocks += -(-keys // GROUP)
        seen += (i1 - i0) * T if not c["causal"] else sum(range(p + i0 + 1, p + i1 + 1))
    return {"bytes": H * moved + 2.0 * rows * H * R * D * e + (rows * H * R * 4.0 if c["lse"] else 0)
            + (2.0 * H * blocks * 4.0 if c["mass"] else 0),
            "flops": H * R * (4.0 * D * seen + 4.0 * D * c["group"] * rows)}
