"""64-bit definitions of the serving operators (attention over shared prefixes, accumulated
attention weights, cache eviction, low-rank adapters) and the error bounds that the tests hold
the kernels to.  numpy on float64 arrays; test infrastructure only.

Every bound counts roundings: a rounding to a type is off by at most half a step, eps / 2 of the
type relative to the value (bf16 2^-8, fp32 2^-24), and a sum of n fp32 terms by at most
n 2^-24 times the sum of their magnitudes.
"""
from __future__ import annotations

import math

import numpy as np

U32, UBF = 2.0 ** -24, 2.0 ** -8


def attention(q, keys, vals, low: int):
    """One query group on one KV head: q [G][d], keys/vals [n][d], positions below `low` hidden.
    Returns o [G][d], lse [G] and their error bounds for bf16 inputs, fp32 scores and sums,
    weights rounded to bf16 for the second product and a bf16 result."""
    G, d = q.shape
    keys, vals = keys[low:], vals[low:]
    n = len(keys)
    if n == 0:
        return (np.zeros((G, d)), np.full(G, -np.inf), np.zeros((G, d)), np.zeros(G))
    s = q @ keys.T / math.sqrt(d)
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(1, keepdims=True)
    w = p / l
    o, o_abs = w @ vals, w @ np.abs(vals)
    # a score: d products, the scale and its rounding; its error is the weight's relative error
    mag = (np.abs(q) @ np.abs(keys).T / math.sqrt(d)).max(1, keepdims=True)
    ds = (d + 4) * U32 * mag + 4 * U32 * np.abs(m)
    # twice (numerator and sum), the exponential's own error, the sums, rescalings on the way
    rel = 2 * ds + (2 * n + 64) * U32
    err = (UBF + rel) * o_abs + UBF * np.abs(o) * (1 + UBF) + rel * np.abs(o)
    lse = (m + np.log(l))[:, 0]
    e_lse = (ds + (n + 64) * U32)[:, 0] + 4 * U32 * (np.abs(lse) + np.abs(m[:, 0]))
    return o, lse, err, e_lse


def prefix_attention(q, kc, vc, kv_len, pk, pv, p_len, prefix_of, window: int):
    """q [T][nq][d]; own caches [T][nkv][cap][d]; prefixes [n][nkv][cap][d] (or None)."""
    T, nq, d = q.shape
    nkv = kc.shape[1]
    G = nq // nkv
    out = [np.zeros((T, nq, d)), np.zeros((T, nq)), np.zeros((T, nq, d)), np.zeros((T, nq))]
    for t in range(T):
        g = prefix_of[t] if pk is not None else -1
        P, L = (p_len[g] if g >= 0 else 0), kv_len[t]
        low = max(0, P + L - window) if window else 0
        for j in range(nkv):
            ks, vs = kc[t, j, :L], vc[t, j, :L]
            if P:
                ks, vs = np.concatenate([pk[g, j, :P], ks]), np.concatenate([pv[g, j, :P], vs])
            for dst, x in zip(out, attention(q[t, j * G:(j + 1) * G], ks, vs, low)):
                dst[t, j * G:(j + 1) * G] = x
    return out


def attention_weights(q, kc, kv_len, lse):
    """What one step adds to acc [T][nkv][cap], and the error bound of the addition."""
    T, nq, d = q.shape
    nkv, cap = kc.shape[1:3]
    G = nq // nkv
    add, err = np.zeros((T, nkv, cap)), np.zeros((T, nkv, cap))
    for t in range(T):
        L = kv_len[t]
        for j in range(nkv):
            x, z = q[t, j * G:(j + 1) * G], lse[t, j * G:(j + 1) * G]
            live = np.isfinite(z)
            x, z = x[live], z[live]
            s = x @ kc[t, j, :L].T / math.sqrt(d)
            p = np.exp(s - z[:, None])
            mag = np.abs(x) @ np.abs(kc[t, j, :L]).T / math.sqrt(d)
            rel = (d + 4) * U32 * mag + 4 * U32 * (np.abs(z[:, None]) + np.abs(s)) + 32 * U32
            add[t, j, :L] = p.sum(0)
            err[t, j, :L] = (p * rel).sum(0) + G * U32 * p.sum(0)
    return add, err


def evict(acc, length: int, budget: int, n_sink: int, n_recent: int):
    """Kept positions, in order, of one (sequence, KV head)."""
    if length <= budget:
        return np.arange(length)
    mid = list(range(n_sink, length - n_recent))
    weight = [(-math.inf, 0) if math.isnan(acc[p]) else (float(acc[p]), 1) for p in mid]
    order = sorted(range(len(mid)), key=lambda i: (-weight[i][0], -weight[i][1], i))
    keep = sorted(mid[i] for i in order[:budget - n_sink - n_recent])
    return np.array(list(range(n_sink)) + keep + list(range(length - n_recent, length)), dtype=int)


def lora(x, y, a, b, scale, rank, adapter_of):
    """y + scale B (A x) and its error bound: fp32 sums, A x kept as two bf16, a bf16 result."""
    out, err = y.copy(), UBF * np.abs(y)
    for t, i in enumerate(adapter_of):
        if i < 0 or rank[i] == 0:
            err[t] = 0.0
            continue
        A, B = a[i, :rank[i]], b[i, :, :rank[i]]
        v, v_abs = A @ x[t], np.abs(A) @ np.abs(x[t])
        out[t] = y[t] + scale[i] * (B @ v)
        n_in, r = len(x[t]), rank[i]
        ev = (n_in + 2) * U32 * v_abs + 2.0 ** -16 * np.abs(v)
        ed = np.abs(B) @ ev + (2 * r + 2) * U32 * (np.abs(B) @ np.abs(v))
        err[t] = UBF * (np.abs(out[t]) + scale[i] * ed) + (1 + UBF) * scale[i] * ed + 2 * U32 * np.abs(y[t])
    return out, err
