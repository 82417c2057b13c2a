"""Plain fp64 definitions of the serving operators on the 4-bit KIVI-style cache
(attend, append, read) and of the rotation of queries and keys, with error bounds
for what the kernels round.

Arrays: payload uint8 [L, 2, B, H, cap, 64] (two codes a byte, the lower channel in the
low half), meta fp32 [L, 2, B, H, 4 cap, 2] (minimum, step): of keys (row / 32) 128 +
channel, of values row 4 + channel / 32.  gauges fp32 [L, 2, H, 128 / g, g, g] or None.
Query or row i of sequence b stands at starts[b] + i and is there if
0 <= position < lengths[b].
"""
from __future__ import annotations

import numpy as np

from .serving import D, dense

GROUP = 32
U = 2.0 ** -24


def codes(payload):
    """[..., 64] bytes -> [..., 128] codes."""
    return np.stack([payload & 15, payload >> 4], -1).reshape(*payload.shape[:-1], D)


def packed(code):
    """[..., 128] codes -> [..., 64] bytes."""
    return (code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8)


def ranges(meta, kind, T):
    """A field's meta [4 cap, 2] -> minimum and step of rows [0, T) and every channel, fp64 [T, 128]."""
    t = np.arange(T)[:, None]
    c = np.arange(D)[None, :]
    m = meta.astype(np.float64)[t // GROUP * D + c if kind == 0 else t * 4 + c // GROUP]
    return m[..., 0], m[..., 1]


def decoded(payload, meta, kind, T):
    """A field's rows [0, T) in gauged coordinates, fp64."""
    mn, st = ranges(meta, kind, T)
    with np.errstate(invalid="ignore"):
        return mn + st * codes(payload[:T]).astype(np.float64)


def quantize(x, kind):
    """Gauged fp32 rows of a field from its first on -> (bytes [T, 64], meta of the ranges that hold a row: keys
    [ceil(T / 32) * 128, 2], values [T * 4, 2]), the encoder's fp32 operations."""
    x = np.asarray(x, np.float32)
    T = x.shape[0]
    code = np.zeros((T, D), np.uint8)
    meta = []
    f = np.float32

    def one(y):
        """Ranges along the first axis of y."""
        mn, mx = y.min(0), y.max(0)
        with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
            diff = (mx - mn).astype(f)
            inv = np.where(diff > 0, f(15.0) / diff, f(0)).astype(f)
            zero = (mx == mn) | ~(inv <= np.finfo(f).max)
            p = ((y - mn).astype(f) * inv).astype(f)
        q = np.where(zero, 0, np.clip(np.rint(p), 0, 15)).astype(np.uint8)
        return q, np.stack([mn, np.where(zero, f(0), (diff / f(15.0)).astype(f))], -1)

    if kind == 0:
        for lo in range(0, T, GROUP):
            code[lo:lo + GROUP], m = one(x[lo:lo + GROUP])
            meta.append(m)
    else:
        q, m = one(np.moveaxis(x.reshape(T, D // GROUP, GROUP), 2, 0))
        code[:] = np.moveaxis(q, 0, 2).reshape(T, D)
        meta.append(m.reshape(T * 4, 2))
    return packed(code), np.concatenate(meta).astype(np.float32) if T else np.zeros((0, 2), np.float32)


def attend(q, payload, meta, G, layer, scale, causal, lengths, starts=None, fp32=False, one_part=False):
    """q [B, n, Hq, 128] fp64 -> dict of out, lse, mass (this layer's gain) and bounds out_tol, lse_tol, mass_tol
    of the kernels' unrounded results.

    With u = 2^-24, k' a key, K_b the largest of |minimum| and |minimum + 15 step| of token t's block b,
    V_b that of the values of its block, Q the row's largest |q'|, a_c = |minimum| + 15 step of
    channel c in the block:
      score   q' is an fp32 chain (g u sum |G| |q| a channel).  The products q'_c step_c stand in two fp16
              parts, scaled so that Q is at least 2^13 and the steps by 2^(2 - E), 2^E <= 2 K_b.  The first
              is a multiple of 2^3, the second at most 2^2 and so rounded by 2^-9: 2^-9 2^-13 2^(E - 2) Q <=
              2^-23 Q K_b a channel, times a code, 15; its sum loses 2^-18 Q K_b in all to the matrix
              cores' alignment; the parts' sums, their sum and the sum with the minima round by 16 u of
              sum |q'_c| a_c.  So
                ds_t = scale (128 15 2^-23 Q K_b + 2^-18 Q K_b + 16 u sum |q'_c| a_c + g u sum_c (|G| |q|)_c a_c)
                       + 8 u max |s|
              one_part: keys and queries are each one fp16 number, their product
              off by (2^-11 + 2^-11 + 2^-22) of the channel's terms |q'_c| (|k'_tc| + 2^-10 a_c), plus 2^-12 of
              (|minimum| + 15 step) for the key's own pieces, plus 2^-34 K_b where it is small.
      weight  dw = 2 ds + 2^-21, and the rounding wr to fp16 (2^-11, in two parts 2^-21) beside the values,
              2^-33 of the largest p_t V_b for small ones.
      value   rounded pieces: dv = r (8 step + |centre| + |v|) + 2^-31 V_b, r = 2^-11, or 2^-20 in two parts.
      sums    fp32, cut instead of rounded: 2^-18 + 2^-23 a unit of 32 tokens of sum p |v|.
    """
    B, n, Hq, _ = q.shape
    H = payload.shape[3]
    R = Hq // H
    nblk = payload.shape[4] // GROUP
    out, tol = np.zeros((B, n, Hq, D)), np.zeros((B, n, Hq, D))
    lse, lse_tol = np.full((B, n, Hq), -np.inf), np.zeros((B, n, Hq))
    mass, mass_tol = np.zeros((B, H, nblk)), np.zeros((B, H, nblk))
    wr, vr = (2.0 ** -21, 2.0 ** -20) if fp32 else (2.0 ** -11, 2.0 ** -11)
    for b in range(B):
        T = int(lengths[b])
        p0 = T - n if starts is None else int(starts[b])
        if T <= 0:
            continue
        for h in range(H):
            GK = dense(None if G is None else G[layer, 0, h])
            GV = dense(None if G is None else G[layer, 1, h])
            g = 0 if G is None else G.shape[-1]
            at0, at1 = (layer, 0, b, h), (layer, 1, b, h)
            km, ks = ranges(meta[at0], 0, T)
            K = km + ks * codes(payload[at0][:T])
            vm, vs = ranges(meta[at1], 1, T)
            V = vm + vs * codes(payload[at1][:T])
            ka = np.abs(km) + 15 * ks
            kb = np.maximum(np.abs(km), np.abs(km + 15 * ks)).max(1)           # the same for a block's tokens
            vtop = np.maximum(np.abs(vm), np.abs(vm + 15 * vs)).max(1)
            pad = np.zeros(-(-T // GROUP) * GROUP)
            pad[:T] = vtop
            vb = np.repeat(pad.reshape(-1, GROUP).max(1), GROUP)[:T]
            dv = vr * (8 * vs + np.abs(vm + 8 * vs) + np.abs(V)) + 2.0 ** -31 * vb[:, None]
            for i in range(n):
                pos = p0 + i
                if not 0 <= pos < T:
                    continue
                vis = pos + 1 if causal else T
                for j in range(R):
                    x = q[b, i, h * R + j]
                    qg = GK @ x
                    aq, Q = np.abs(qg), np.abs(qg).max()
                    s = (K[:vis] @ qg) * scale
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    p = p / l
                    o = p @ V[:vis]
                    out[b, i, h * R + j] = o @ GV
                    lse[b, i, h * R + j] = m + np.log(l)
                    ds = (128 * 15 * 2.0 ** -23 + 2.0 ** -18) * Q * kb[:vis] + 16 * U * (ka[:vis] @ aq)
                    if one_part:
                        ds = ds + (np.abs(K[:vis]) * 2.0 ** -9.9) @ aq + (ka[:vis] * 2.0 ** -11) @ aq + 128 * 2.0 ** -34 * Q * kb[:vis]
                    ds = scale * (ds + g * U * (ka[:vis] @ (np.abs(GK) @ np.abs(x)))) + 8 * U * np.abs(s).max()
                    moved = 0.0
                    if one_part:
                        moved = (p * np.expm1(ds)) @ np.abs(V[:vis] - o) * np.exp(ds.max())
                    ds = ds.max()
                    dw = 2 * ds + 2.0 ** -21
                    lse_tol[b, i, h * R + j] = ds + 2.0 ** -20 + 4 * U * abs(m)
                    av = p @ np.abs(V[:vis])
                    units = -(-vis // GROUP)
                    et = p @ dv[:vis] + wr * av + ((2.0 ** -21 if one_part else dw) + 2.0 ** -18 + units * 2.0 ** -23) * av
                    et += vis * 2.0 ** -33 * (p * vb[:vis]).max() + moved
                    tol[b, i, h * R + j] = np.abs(GV).T @ et + g * U * (np.abs(GV).T @ np.abs(o))
                    full = np.zeros(nblk * GROUP)
                    full[:vis] = p
                    w = full.reshape(nblk, GROUP).sum(1)
                    mass[b, h] += w
                    mass_tol[b, h] += (dw + 2.0 ** -19) * w + 2.0 ** -40
    return dict(out=out, out_tol=tol, lse=lse, lse_tol=lse_tol, mass=mass, mass_tol=mass_tol)


def rotate(x, weight, eps, freq, positions, interleaved, sections=None, dealt=False, magnitude=1.0):
    """x [B, n, heads, 128] fp64, positions [axes, B, n], freq fp32 [dim / 2] -> (y, bound of the unrounded fp32
    result).  A normed value is off by 12 u (half of the 13 of the sum of squares, root and quotient 2 each,
    products), a cosine or sine by 2^-22 (the turn rounded to fp32, 2^-26 of a turn, and the functions), the
    products and the sum by 2 u."""
    y = np.array(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    pairs = len(freq)
    if pairs == 0:
        return y, 12 * U * np.abs(y)
    axes = positions.shape[0]
    sec = [pairs] if axes == 1 else list(sections)
    if dealt:
        axis = [i % axes if i < axes * sec[i % axes] else 0 for i in range(pairs)]
    else:
        axis = [a for a, m in enumerate(sec) for _ in range(m)]
    ang = np.stack([positions[axis[i]].astype(np.float64) * np.float64(freq[i]) for i in range(pairs)], -1)[:, :, None]
    c, s = np.cos(ang) * magnitude, np.sin(ang) * magnitude
    a = np.arange(pairs) * 2 if interleaved else np.arange(pairs)
    b = a + 1 if interleaved else a + pairs
    out, tol = y.copy(), 12 * U * np.abs(y)
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    both = (np.abs(y[..., a]) + np.abs(y[..., b])) * abs(magnitude)
    tol[..., a] = tol[..., b] = (14 * U + 2.0 ** -22) * both
    return out, tol
