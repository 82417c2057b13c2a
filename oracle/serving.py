"""Plain fp64 definitions of the serving operators on the 8-bit block-uniform
cache (append, attend, evict), with error bounds for what the kernels round.

Arrays: payload uint8 [L, 2, B, H, cap, 128], meta fp32 [L, 2, B, H, cap / T_b, 2]
(minimum, step), gauges fp32 [L, 2, H, 128 / g, g, g] or None.  Query or row i
of sequence b stands at starts[b] + i and is there if 0 <= position < lengths[b].
"""
from __future__ import annotations

import numpy as np

D = 128


def dense(G):
    """[128/g, g, g] -> block-diagonal 128 x 128 (fp64); None -> identity."""
    if G is None:
        return np.eye(D)
    R, g, _ = G.shape
    M = np.zeros((D, D))
    for r in range(R):
        M[r * g:(r + 1) * g, r * g:(r + 1) * g] = G[r]
    return M


def _rows(payload, meta, T, block):
    mm = np.repeat(meta.astype(np.float64), block, axis=0)[:T]
    with np.errstate(invalid="ignore"):
        return mm[:, :1], mm[:, 1:], payload[:T].astype(np.float64)


def attend(q, payload, meta, G, layer, block, scale, causal, lengths, starts=None, fp32=False, one_part=False):
    """q [B, n, Hq, 128] fp64 -> dict of out, lse, mass (this layer's gain) and
    bounds out_tol, lse_tol, mass_tol of the kernels' unrounded results.

    Bounds, with u = 2^-24 and per row S = max_t sum_c |q'_c| (|mn_t| + 255 st_t):
    q' is an fp32 chain over g channels (g u sum |G| |q| a channel), split into
    two fp16 parts (2^-23 of the row's largest |q'| at most), its product
    with the codes a sum of 256 terms in fp32 and two more operations, so a
    score in units of log2 is off by at most
      ds = scale log2(e) (2^-16 S + g u S_g),
    S_g the same sum with the chain's magnitudes; a row's log-sum by ds and its
    rounding.  A weight is off by 2 ds + 2^-21 (exp2 and its argument's
    rounding, |s| u at most), plus the rounding of the weight to fp16 (2^-11, in
    two parts 2^-21) in the sum over the codes, plus 2^-33 of the largest for
    weights below 2^-23 of it.

    one_part: the bounds of queries in one fp16 part, where only out is asked for.  A
    channel of q' is rounded by 2^-11 of itself (below 2^-14 of the operands, 2^-27 of
    the row's largest, by 2^-25 of them, which is below the other terms), in the products
    with the codes and in the sum beside the minima alike, so a score moves by that of
    the channels' products with the key.  Codes are fp16 subnormals there: the matrix
    cores align products by exponent fields, and a subnormal's field is up to 2^10 above
    a code's own (2^-24 a code, field 2^-14), so each of the 128 products loses up to
    2^-23 2^10 of the largest channel in units of a code, 2^-6 of it in all; the sums in
    fp32, cut instead of rounded, 2^-15 S.  In units of log2 the score of token t is off by
      ds_t = scale log2(e) (2^-11 sum_c |q'_c k_tc| + 2^-6 max_c |q'_c| step_t + 2^-15 S + g u S_g)
    and by the roundings of large scores as above.  With weights w_t = p_t 2^e_t,
    |e_t| <= ds_t, the mean moves by sum_t p_t (2^e_t - 1) (v_t - out) over sum_t p_t 2^e_t.
    """
    B, n, Hq, _ = q.shape
    H = payload.shape[3]
    R = Hq // H
    nblk = meta.shape[4]
    out, tol = np.zeros((B, n, Hq, D)), np.zeros((B, n, Hq, D))
    lse, lse_tol = np.full((B, n, Hq), -np.inf), np.zeros((B, n, Hq))
    mass, mass_tol = np.zeros((B, H, nblk)), np.zeros((B, H, nblk))
    u = 2.0 ** -24
    wr = 2.0 ** -21 if fp32 else 2.0 ** -11
    for b in range(B):
        T = int(lengths[b])
        p0 = T - n if starts is None else int(starts[b])
        for h in range(H):
            GK = dense(None if G is None else G[layer, 0, h])
            GV = dense(None if G is None else G[layer, 1, h])
            g = 0 if G is None else G.shape[-1]
            if T <= 0:
                continue
            kmn, kst, kc = _rows(payload[layer, 0, b, h], meta[layer, 0, b, h], T, block)
            vmn, vst, vc = _rows(payload[layer, 1, b, h], meta[layer, 1, b, h], T, block)
            K, V = kmn + kst * kc, vmn + vst * vc
            kmag = (np.abs(kmn) + 255 * kst)[:, 0].max()
            for i in range(n):
                pos = p0 + i
                if not 0 <= pos < T:
                    continue
                vis = pos + 1 if causal else T
                for j in range(R):
                    x = q[b, i, h * R + j]
                    qg = GK @ x
                    s = (K[:vis] @ qg) * scale
                    m = s.max()
                    e = np.exp(s - m)
                    l = e.sum()
                    p = e / l
                    o = p @ V[:vis]
                    out[b, i, h * R + j] = o @ GV
                    lse[b, i, h * R + j] = m + np.log(l)
                    qs, qsg = np.abs(qg).sum(), (np.abs(GK) @ np.abs(x)).sum()
                    ds = scale * kmag * (2.0 ** -16 * qs + g * u * qsg)
                    ds += np.abs(s).max() * 8 * u
                    moved = 0.0
                    if one_part:
                        d1 = 2.0 ** -11 * (np.abs(K[:vis]) @ np.abs(qg)) + 2.0 ** -6 * np.abs(qg).max() * kst[:vis, 0]
                        d1 += kmag * (2.0 ** -15 * qs + g * u * qsg)
                        d1 = scale * d1 + np.abs(s).max() * 8 * u          # of exp, so without log2(e)
                        moved = (p * np.expm1(d1)) @ np.abs(V[:vis] - o) * np.exp(d1.max())
                        ds = d1.max()
                    dw = 2 * ds + 2.0 ** -21
                    lse_tol[b, i, h * R + j] = ds + 2.0 ** -20 + 4 * u * abs(m)
                    cw = p @ (vst[:vis] * vc[:vis])      # sum of p step code
                    ab = (np.abs(p[:, None] * vmn[:vis])).sum() + (p[:, None] * 255 * vst[:vis]).sum()
                    big = (p[:, None] * vst[:vis]).max()
                    et = wr * cw + ((2.0 ** -21 if one_part else dw) + 2.0 ** -18) * ab + 255 * vis * 2.0 ** -33 * big + moved
                    tol[b, i, h * R + j] = np.abs(GV).T @ et + g * u * (np.abs(GV).T @ np.abs(o))
                    full = np.zeros(nblk * block)
                    full[:vis] = p
                    w = full.reshape(nblk, block).sum(1)
                    mass[b, h] += w
                    mass_tol[b, h] += (dw + 2.0 ** -19) * w + 2.0 ** -40
    return dict(out=out, out_tol=tol, lse=lse, lse_tol=lse_tol, mass=mass, mass_tol=mass_tol)


def quantize(x, block):
    """Gauged fp32 rows from a block's start on -> (codes, [(min, step)]), the
    encoder's fp32 operations."""
    x = np.asarray(x, np.float32)
    codes, meta = np.zeros(x.shape, np.uint8), []
    for lo in range(0, x.shape[0], block):
        y = x[lo:lo + block]
        mn, mx = y.min(), y.max()
        diff = np.float32(mx - mn)
        inv = np.float32(255.0) / diff if diff > 0 else np.float32(0)
        if mx == mn or not inv <= np.finfo(np.float32).max:
            meta.append((mn, np.float32(0)))
            continue
        p = (y - mn) * inv
        codes[lo:lo + block] = np.clip(np.rint(p), 0, 255).astype(np.uint8)
        meta.append((mn, np.float32(diff / np.float32(255.0))))
    return codes, np.array(meta, np.float32).reshape(-1, 2)


def keep_blocks(mass, length, block, budget, sink, recent):
    """Numbers of the blocks of one head that stay."""
    n = -(-int(length) // block)
    if n <= budget:
        return list(range(n))
    mid = list(range(sink, n - recent))
    w = [(-np.inf if np.isnan(mass[i]) else float(mass[i]), np.isnan(mass[i])) for i in range(n)]
    mid.sort(key=lambda i: (w[i][1], -w[i][0], i))
    return sorted(list(range(sink)) + mid[:budget - sink - recent] + list(range(n - recent, n)))
