"""Float64 oracle of the operators between a block's linears: rotary positions,
the 8-bit key/value cache, the attention over it, and the norms with gate and
residual. Plain loops over sequences and heads from the definitions; shares
no code with the GPU path."""
from __future__ import annotations

import math

import numpy as np

BLOCK = 64
CODE_MAX = {"int8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------- rotary
def frequencies(rot, theta=10000.0, scaling="none", factor=1.0, original=8192.0, fast=32.0, slow=1.0):
    """Angle of each pair per position, and the factor on cosine and sine."""
    base, mag = theta, 1.0
    if scaling == "base":
        base = theta * factor ** (rot / max(1, rot - 2))
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        def pair(turns):
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(0.0, math.floor(pair(fast))), min(rot - 1.0, math.ceil(pair(slow)))
        for i in range(rot // 2):
            r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            f[i] = f[i] * (1 - r) + f[i] / factor * r
        mag = 0.1 * math.log(factor) + 1.0
    return f, mag


def rope(x, pos, f, mag=1.0, layout="half", inverse=False):
    """x [tokens, heads, dim] float64 with its first 2 len(f) elements turned."""
    n = len(f)
    y = np.array(x, dtype=np.float64)
    for i in range(n):
        a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        ang = np.asarray(pos, np.float64) * f[i]
        c, s = (mag * np.cos(ang))[:, None], (mag * np.sin(ang))[:, None]
        if inverse:
            s = -s
        xa, xb = np.asarray(x[..., a], np.float64), np.asarray(x[..., b], np.float64)
        y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    return y


# -------------------------------------------------------------------- cache
def e4m3_values():
    """The 127 values of the non-negative finite e4m3 codes 0 .. 126."""
    v = []
    for u in range(127):
        e, m = u >> 3, u & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


E4M3 = e4m3_values()


def to_e4m3(x):
    """Nearest e4m3 byte of finite x, ties to the even code, |x| above 448 to 448."""
    a = np.minimum(np.abs(np.asarray(x, np.float64)), 448.0)
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    u = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (u | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def from_codes(codes, fmt):
    """Values of code bytes."""
    u = np.asarray(codes).view(np.uint8)
    if fmt == "int8":
        return u.view(np.int8).astype(np.float64)
    if ((u & 127) == 127).any():
        raise ValueError("NaN code")
    return np.where(u & 128, -1.0, 1.0) * E4M3[u & 127]


def quantise(x, fmt):
    """One block of one head, x float16 (any shape): code bytes and the scale,
    by the definition's fp32 steps: 1 / amax, times M, x times it, round half
    to even; amax / M."""
    x = np.asarray(x).astype(np.float32)
    amax = np.float32(np.abs(x).max()) if x.size else np.float32(0)
    M = np.float32(CODE_MAX[fmt])
    if amax == 0:
        return np.zeros(x.shape, np.uint8), np.float32(0)
    with np.errstate(over="ignore"):
        t = x * (M * (np.float32(1) / amax))
    if fmt == "int8":
        c = np.clip(np.rint(t), -127, 127).astype(np.int8).view(np.uint8)
    else:
        c = to_e4m3(t)
    return c, amax / M


class Cache:
    """The cache as numpy arrays (codes as bytes)."""

    def __init__(self, blocks, slots, kv_heads, dim, fmt):
        self.fmt, self.dim, self.kv_heads = fmt, dim, kv_heads
        self.k_codes = np.zeros((blocks, kv_heads, BLOCK, dim), np.uint8)
        self.v_codes = np.zeros((blocks, kv_heads, dim, BLOCK), np.uint8)
        self.k_scale = np.zeros((blocks, kv_heads), np.float32)
        self.v_scale = np.zeros((blocks, kv_heads), np.float32)
        self.k_tail = np.zeros((slots, kv_heads, BLOCK, dim), np.float16)
        self.v_tail = np.zeros((slots, kv_heads, dim, BLOCK), np.float16)

    def put(self, seq_len, table, slot, k, v):
        """Append k, v [n, kv_heads, dim] float16 as the last of seq_len tokens,
        token by token."""
        n = k.shape[0]
        for i in range(n):
            p = seq_len - n + i
            if p < 0:
                continue
            for h in range(self.kv_heads):
                kr, vr = k[i, h].copy(), v[i, h].copy()
                if not (np.isfinite(kr).all() and np.isfinite(vr).all()):
                    kr[:] = np.nan
                    vr[~np.isfinite(vr)] = 0
                self.k_tail[slot, h, p % BLOCK] = kr
                self.v_tail[slot, h, :, p % BLOCK] = vr
            if p % BLOCK == BLOCK - 1:
                b = table[p // BLOCK]
                for h in range(self.kv_heads):
                    kb, vb = self.k_tail[slot, h], self.v_tail[slot, h]
                    bad = not np.isfinite(kb).all()
                    c, s = quantise(np.where(np.isfinite(kb), kb, np.float16(0)), self.fmt)
                    self.k_codes[b, h], self.k_scale[b, h] = c, np.float32(np.nan) if bad else s
                    self.v_codes[b, h], self.v_scale[b, h] = quantise(vb, self.fmt)

    def read(self, seq_len, table, slot, h):
        """Keys and values [seq_len, dim] of one kv head in float64."""
        full = seq_len // BLOCK
        k = [from_codes(self.k_codes[b, h], self.fmt) * np.float64(self.k_scale[b, h]) for b in table[:full]]
        v = [from_codes(self.v_codes[b, h], self.fmt).T * np.float64(self.v_scale[b, h]) for b in table[:full]]
        k.append(self.k_tail[slot, h, :seq_len % BLOCK].astype(np.float64))
        v.append(self.v_tail[slot, h, :, :seq_len % BLOCK].T.astype(np.float64))
        return np.concatenate(k), np.concatenate(v)


# ---------------------------------------------------------------- attention
def attend(q, k, v, visible, scale):
    """One query row: (output, sum of p |v|, largest scale sum |q| |k|) over the
    first `visible` tokens; zeros where there is none."""
    if visible <= 0:
        return np.zeros(v.shape[1]), np.zeros(v.shape[1]), 0.0
    k, v = k[:visible], v[:visible]
    s = scale * (k @ q)
    p = np.exp(s - s.max()) if np.isfinite(s).all() else np.full(s.shape, np.nan)
    p = p / p.sum()
    return p @ v, p @ np.abs(v), abs(scale) * float(np.max(np.abs(k) @ np.abs(q)))


# -------------------------------------------------------------------- norms
def norm_residual(y, r, w_pre, w_post, gate, alpha, beta, eps, offset):
    """(r', sum of its terms' magnitudes) in float64 before r' is stored, and
    the function that gives h from a stored r'."""
    r = np.asarray(r, np.float64)
    if y is None:
        out, mag = r, np.abs(r)
    else:
        b = np.asarray(y, np.float64)
        if w_post is not None:
            b = b / np.sqrt((b * b).mean(1, keepdims=True) + eps) * (np.asarray(w_post, np.float64) + offset)
        if gate is not None:
            b = b * np.asarray(gate, np.float64)
        out, mag = alpha * r + beta * b, np.abs(alpha * r) + np.abs(beta * b)

    def h(stored):
        s = np.asarray(stored, np.float64)
        return s / np.sqrt((s * s).mean(1, keepdims=True) + eps) * (np.asarray(w_pre, np.float64) + offset)
    return out, mag, h
