"""64-bit definitions of the rotation of queries and keys, of caches in 8 bits and of attention over
them, with the error bounds that the tests hold the kernels to.  numpy; test infrastructure only.

As in ``oracle/serving.py`` every bound counts roundings: half a step of the type for each (bf16 2^-8,
fp16 2^-11, fp32 2^-24), and n 2^-24 times the sum of the magnitudes for a sum of n fp32 terms.
"""
from __future__ import annotations

import math

import numpy as np

from oracle.serving import U32, UBF

U16 = 2.0 ** -11
SMALLEST = 2.0 ** -110


# ---------------------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------------------
def frequencies(rot, theta, scaling="none", factor=1.0, context=0.0, low=1.0, high=32.0):
    """Radians per position of every pair, written pair by pair."""
    out = []
    for i in range(rot // 2):
        f = theta ** (-2.0 * i / rot)
        if scaling == "linear":
            f = f / factor
        elif scaling != "none":
            if scaling == "turns":
                w = (context * f / (2 * math.pi) - low) / (high - low)
            else:
                at = [rot / 2 * math.log(context / (2 * math.pi * r)) / math.log(theta) for r in (high, low)]
                w = 1 - (i - at[0]) / (at[1] - at[0])
            w = min(1.0, max(0.0, w))
            f = f * w + f / factor * (1 - w)
        out.append(f)
    return np.array(out)


def rope(x, pos, freq, layout="half", amplitude=1.0, gain=None, eps=0.0):
    """x [T][heads][d] at positions pos [T]: the rotated rows and their error bounds (bf16 results)."""
    T, _, d = x.shape
    half = len(freq)
    rel = 0.0
    if gain is not None:
        x = x / np.sqrt((x ** 2).mean(2, keepdims=True) + eps) * gain
        # the sum of d squares and eps (halved by the root), the root's 2 ulp, two products, the mean
        rel = (d / 2 + 8) * U32
    angle = np.asarray(pos, dtype=np.float64)[:, None, None] * freq
    c, s = np.cos(angle) * amplitude, np.sin(angle) * amplitude
    i = np.arange(half)
    a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
    y, err = x.copy(), rel * np.abs(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    # the fraction of a turn to fp32 (2^-25 turns, times 2 pi), sine and cosine (2 ulp), the amplitude,
    # two products and a sum; the frequency's and the angle's 64 bits, here and there
    turn = 2 * math.pi * 2.0 ** -25 + 8 * U32 + 2.0 ** -50 * np.abs(angle)
    pair = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(amplitude)
    err[..., a] = err[..., b] = pair * (rel + turn)
    err = err * (1 + UBF) + UBF * np.abs(y)
    if gain is None:
        err[..., 2 * half:] = 0.0               # neither normed nor rotated: as it was
    return y, err


# ---------------------------------------------------------------------------------------
# codes
# ---------------------------------------------------------------------------------------
def e4m3_table():
    """The number of every code: sign, four bits of exponent (bias 7), three of mantissa."""
    t = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = math.nan if (c & 127) == 127 else (-v if c & 128 else v)
    return t


E4M3 = e4m3_table()


def quantise(x, block, fmt):
    """Codes (bytes) and scales of x [positions][d], positions a multiple of block."""
    codes, scales = np.zeros(x.shape, dtype=np.uint8), []
    for b in range(0, len(x), block):
        y = x[b:b + block]
        if not np.isfinite(y).all():
            scales.append(math.nan)
            continue
        amax = max(float(np.abs(y).max()), SMALLEST)
        if fmt == "int8":
            s = np.float32(amax) / np.float32(127)
            z = (y.astype(np.float32) / s).astype(np.float64)
            codes[b:b + block] = np.rint(z).astype(np.int8).view(np.uint8)      # halves to even
        else:
            s = 2.0 ** -130
            while amax > 448 * s:
                s *= 2
            z = y / s
            mag = E4M3[:127]
            i = np.clip(np.searchsorted(mag, np.abs(z)), 1, 126)                # mag[i - 1] < |z| <= mag[i]
            lo, hi = np.abs(z) - mag[i - 1], mag[i] - np.abs(z)
            take = np.where((lo < hi) | ((lo == hi) & (i % 2 == 1)), i - 1, i)  # halves to the even code
            codes[b:b + block] = take.astype(np.uint8) | np.where(np.signbit(z), 128, 0).astype(np.uint8)
        scales.append(float(s))
    return codes, np.array(scales)


def values(codes, scales, block, fmt):
    """What codes [positions][d] stand for, block by block."""
    v = codes.view(np.int8).astype(np.float64) if fmt == "int8" else E4M3[codes]
    return v * np.repeat(scales, block)[:len(v), None]


# ---------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------
def attention(q, keys, vals, v_scale, low: int, coded: int):
    """One query group on one KV head: q [G][d], keys/vals [n][d] of which the first `coded` come from
    codes with value scales v_scale [coded]; positions below `low` hidden.  Returns o, lse and their
    bounds: fp32 scores and sums; for the product with v the weights (times v's scale) rounded to fp16
    for codes, relative down to 2^-28 of the largest, and to bf16 for the others; a bf16 result."""
    G, d = q.shape
    sv = np.concatenate([v_scale, np.ones(len(keys) - coded)])[low:]
    keys, vals, n_c = keys[low:], vals[low:], max(0, coded - low)
    n = len(keys)
    if n == 0:
        return np.zeros((G, d)), np.full(G, -np.inf), np.zeros((G, d)), np.zeros(G)
    s = q @ keys.T / math.sqrt(d)
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(1, keepdims=True)
    w = p / l
    o = w @ vals
    o_abs, o_code = w @ np.abs(vals), w[:, :n_c] @ np.abs(vals[:n_c])
    top = np.abs(s).max(1, keepdims=True)
    # a score: d products and their sum, a query's element below 2^-28 of the largest, three factors
    mag = (np.abs(q) @ np.abs(keys).T / math.sqrt(d)).max(1, keepdims=True)
    small = 2.0 ** -39 * np.abs(q).max(1, keepdims=True) * np.abs(keys).sum(1).max() / math.sqrt(d)
    ds = (d + 4) * U32 * mag + 8 * U32 * top + small
    rel = 2 * ds + (2 * n + 64) * U32
    # the exponent of a weight times its value scale: the logarithm (2^-21), sums of it, score and maxima
    pos = sv > 0
    span = np.abs(np.log2(sv[pos])).max(initial=0.0)
    ev = 2.0 ** -21 + 8 * U32 * (2 * span + 2 * 1.4427 * top + 16)
    # weights too small for fp16's full precision
    lost = 2.0 ** -39 * (w * sv).max(1, keepdims=True) * np.where(pos, np.abs(vals).max(1) / np.where(pos, sv, 1), 0)[:n_c].sum()
    err = U16 * o_code + UBF * (o_abs - o_code) + (rel + ev) * o_abs + lost
    err = err * (1 + UBF) + UBF * np.abs(o) + rel * np.abs(o)
    lse = (m + np.log(l))[:, 0]
    e_lse = (ds + (n + 64) * U32)[:, 0] + 4 * U32 * (np.abs(lse) + np.abs(m[:, 0]))
    return o, lse, err, e_lse
