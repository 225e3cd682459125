"""Event-history operators in 64 bits, one row and one query at a time, and
the tolerances that their rounding allows."""
import math

import numpy as np

# half a unit in the last place, relative, of each storage type (24, 11 and 8
# significand bits)
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
# smallest step of a subnormal value, halved
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}


def pairs(rot, interleaved):
    """(first, second, angle) of every turned pair."""
    half = rot // 2
    return [(2 * i, 2 * i + 1, i) if interleaved else (i, i + half, i) for i in range(half)]


def turn(z, row, rot, interleaved, back=False):
    """z[..., d] turned by a rope row (cosines, then sines); also by magnitudes."""
    y, mag = z.copy(), np.abs(z)
    for a, b, i in pairs(rot, interleaved):
        c, s = row[..., i], row[..., i + rot // 2] * (-1 if back else 1)
        y[..., a], y[..., b] = z[..., a] * c - z[..., b] * s, z[..., b] * c + z[..., a] * s
        mag[..., a] = np.abs(z[..., a] * c) + np.abs(z[..., b] * s)
        mag[..., b] = np.abs(z[..., b] * c) + np.abs(z[..., a] * s)
    return y, mag


def norm_rope(x, w, eps, rope, positions, interleaved=False):
    """(y, magnitude) of x[n][heads][d]."""
    z = x.astype(np.float64)
    if w is not None:
        z = z / np.sqrt((z * z).mean(-1, keepdims=True) + eps) * w
    if rope is None:
        return z, np.abs(z)
    return turn(z, rope.astype(np.float64)[positions][:, None], rope.shape[1], interleaved)


def norm_rope_bwd(dy, x, w, eps, rope, positions, interleaved=False):
    """(dx, its magnitude, dw, its magnitude)."""
    dz, dzm = dy.astype(np.float64), np.abs(dy.astype(np.float64))
    if rope is not None:
        dz, dzm = turn(dz, rope.astype(np.float64)[positions][:, None], rope.shape[1], interleaved, back=True)
    if w is None:
        return dz, dzm, None, None
    x = x.astype(np.float64)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g, gm = dz * w, dzm * np.abs(w)
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdims=True))
    mag = r * (gm + np.abs(x) * r * r * (gm * np.abs(x)).mean(-1, keepdims=True))
    return dx, mag, (dz * x * r).sum((0, 1)), (dzm * np.abs(x) * r).sum((0, 1))


# Rows in fp32: the sum of squares is 8 products in a lane, then 5 additions
# across lanes; with the division, root, products and the rotation's two
# products no element passes more than 16 roundings of 2^-24 of its magnitude
# (the gradient: twice that).  Then one rounding to the type.
def rows_tolerance(value, mag, dtype, roundings=16):
    return roundings * 2.0 ** -24 * mag + U[dtype] * np.abs(value) * 1.01 + TINY[dtype]


# A weight's gradient: at most `chain` additions one after another.
def weight_tolerance(mag, chain):
    return (chain + 32) * 2.0 ** -24 * mag


def slots(table_row, positions, page):
    return [(int(table_row[p // page]), p % page) for p in positions]


def attention(q, counts, lengths, table, kc, vc, scale, causal, window):
    """q[n][hq][d] over kc, vc [pages][page][hk][d].  Returns out, lse and, per
    output element, the sum of p |v|, per row the largest sum of |q k| * scale,
    and per element sum |v| / l for weights p <= 1 (l: their sum)."""
    n, hq, d = q.shape
    page, hk = kc.shape[1], kc.shape[2]
    out, absout, flat = np.zeros((n, hq, d)), np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse, smax = np.full((n, hq), -np.inf), np.zeros((n, hq))
    first = 0
    for s, (c, length) in enumerate(zip(counts, lengths)):
        for i in range(c):
            hi = max(0, length - c + i + 1) if causal else length
            lo = max(0, hi - window) if window else 0
            if hi <= lo:
                continue
            at = np.arange(lo, hi)
            pg = table[s, at // page]
            ok = ((pg >= 0) & (pg < kc.shape[0]))[:, None, None]
            k = np.where(ok, kc[np.where(ok[:, 0, 0], pg, 0), at % page], 0).astype(np.float64)
            v = np.where(ok, vc[np.where(ok[:, 0, 0], pg, 0), at % page], 0).astype(np.float64)
            for h in range(hq):
                kh, vh, row = k[:, h * hk // hq], v[:, h * hk // hq], q[first + i, h].astype(np.float64)
                score = scale * (kh @ row)
                top = score.max()
                p = np.exp(score - top)
                total = p.sum()
                out[first + i, h] = p @ vh / total
                absout[first + i, h] = p @ np.abs(vh) / total
                flat[first + i, h] = np.abs(vh).sum(0) / total
                lse[first + i, h] = top + math.log(total)
                smax[first + i, h] = scale * (np.abs(kh) @ np.abs(row)).max()
        first += c
    return out, lse, absout, smax, flat


# A score is d products and d - 1 additions in fp32, then one product by
# scale * log2(e) (itself rounded): (d + 4) roundings of 2^-24 -- of 2^-23 where the tensor
# core truncates -- of its magnitude; its weight is off by that, by the
# exponential's 2^-22, and by the type's rounding of p; so is the sum, without the last.
# Rescaling and joining splits add a few roundings each.
def attention_tolerance(out, absout, smax, flat, d, dtype):
    score = (d + 4) * 2.0 ** -23 * smax[..., None]
    weight = 0.0 if dtype == "f32" else U[dtype]
    return (2 * score + 2.0 ** -18 + weight) * absout + U[dtype] * np.abs(out) * 1.01 + TINY[dtype] * (1 + flat)


def lse_tolerance(lse, smax, d):
    finite = np.where(np.isfinite(lse), np.abs(lse), 0)
    return (d + 4) * 2.0 ** -23 * smax + 2.0 ** -20 * (1 + finite)
