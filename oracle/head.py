"""Float64 oracle of the way out of a model: rows in 8 bits (e4m3 codes with a
power-of-two scale for each block of 128), their product with 8-bit weights,
and the sampling of a token. Plain loops from the definitions; sums of the
sampler are Python's whole numbers. Shares no code with the GPU path."""
from __future__ import annotations

import math

import numpy as np

BLOCK = 128
TOP = 448.0
ONE = 1 << 40


# ------------------------------------------------------------------ 8-bit rows
def e4m3_values():
    """What the 256 codes stand for."""
    out = []
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        v = math.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out.append(-v if s else v)
    return np.array(out)


VALUES = e4m3_values()


def to_e4m3(x):
    """The code nearest to each x (|x| <= 448, float64), ties to the even code."""
    x = np.asarray(x, np.float64)
    mag = VALUES[:127]
    i = np.clip(np.searchsorted(mag, np.abs(x)), 1, 126)
    lo, hi = mag[i - 1], mag[i]
    a = np.abs(x)
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))
    return (np.where(up, i, i - 1) | (np.signbit(x) * 128)).astype(np.uint8)


def scale_exponent(top):
    """The smallest whole e >= -127 with top <= 448 2^e; 0 for a block of zeros."""
    if top == 0:
        return 0
    e = -127
    while top > TOP * 2.0 ** e:
        e += 1
    return e


def rows8(x):
    """Codes [rows, 128 n] and scale bytes [rows, n] of x [rows, K]."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    n = -(-K // BLOCK)
    pad = np.zeros((rows, n * BLOCK))
    pad[:, :K] = x
    codes, scales = np.zeros(pad.shape, np.uint8), np.zeros((rows, n), np.uint8)
    for r in range(rows):
        for b in range(n):
            v = pad[r, b * BLOCK:(b + 1) * BLOCK]
            if not np.isfinite(v).all():
                codes[r, b * BLOCK:(b + 1) * BLOCK], scales[r, b] = 127, 255
                continue
            e = scale_exponent(np.abs(v).max())
            codes[r, b * BLOCK:(b + 1) * BLOCK] = to_e4m3(v * 2.0 ** -e)
            scales[r, b] = e + 127
    return codes, scales


def held(codes, scales):
    """What 8-bit rows stand for."""
    e = scales.astype(np.float64) - 127
    return VALUES[codes] * np.repeat(np.where(scales == 255, math.nan, 2.0 ** np.where(scales == 255, 0, e)), BLOCK, 1)


def linear8(x, w):
    """Product of two sets of 8-bit rows' values, and what its error is measured by: for each output the sum over groups
    of 8 columns of the largest product's magnitude, and the sum of all magnitudes."""
    y = x @ w.T
    a, b = np.abs(x), np.abs(w)
    top = np.zeros_like(y)
    for c in range(0, x.shape[1], 8):
        top += np.max(a[:, None, c:c + 8] * b[None, :, c:c + 8], -1)
    return y, top, a @ b.T


# -------------------------------------------------------------------- sampling
def share(f, total, most=1 << 31):
    return min(int(math.floor(min(max(float(f), 0.0), 1.0) * 2 ** 31)), most) * total >> 31


def sample(logits, u, t=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log-probability, kept weights by index) of one row; token -1 where the row has none."""
    l = [float(v) for v in logits]
    u, t, top_p, min_p = float(u), float(t), float(top_p), float(min_p)      # 64 bits whatever they come in
    none = (-1, math.nan, {})
    if any(math.isnan(v) or v == math.inf for v in l) or max(l) == -math.inf or not 0 <= t < math.inf:
        return none
    top = max(l)
    if t == 0:
        return l.index(top), 0.0, {l.index(top): ONE}
    if any(math.isnan(v) for v in (u, top_p, min_p)):
        return none
    w = [int(round(math.exp((v - top) / t) * ONE)) if v > -math.inf else 0 for v in l]
    order = sorted(range(len(l)), key=lambda i: (-l[i], i))
    first = order[:top_k] if top_k > 0 else order
    need = max(1, share(top_p, sum(w[i] for i in first)))
    kept, before = {}, 0
    for i in first:
        if before < need and w[i] >= min(min_p, 1.0) * ONE:
            kept[i] = w[i]
        before += w[i]
    total = sum(kept.values())
    target, run = share(u, total, (1 << 31) - 1), 0
    for i in sorted(kept):
        run += kept[i]
        if run > target:
            return i, math.log(kept[i] / total), kept
    raise AssertionError("no token")
