"""CPU oracle for the 4-bit key/value cache, attention over it, and the fused norms.

TEST INFRASTRUCTURE ONLY (see oracle/moe.py for who may import the oracle). Plain numpy in 64 bits, written
from the definitions in include/coli_moe.h; it shares no code with the library and knows nothing of the
cache's layout in memory: a cached token is the pair of its stored value rows.

The format's own roundings (binary32 steps, bfloat16 scale and offset) are part of its definition, so they
are carried out here as such; everything after them is in 64 bits.

Parity status: pinned by tests/test_kv4_oracle.py (worked groups, brute force, invariances).
"""
from __future__ import annotations

import numpy as np


def bf16(x):
    """Round to bfloat16 (nearest, ties to even), as binary32."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    nan = np.isnan(np.asarray(x, np.float32))
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)
    return np.where(nan, np.float32(np.nan), r)


def quantise(x, gs):
    """(scale, offset, codes) of rows x [..., hd]: scale and offset [..., hd / gs] binary32 holding bfloat16."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], -1, gs)
    lo, hi = g.min(-1), g.max(-1)
    with np.errstate(all="ignore"):
        span = np.float32(hi - lo)
        bad = ~np.isfinite(span) | ~np.isfinite(g).all(-1)
        s = bf16(span * np.float32(1 / 15))
        s = np.where(s < np.float32(2.0 ** -126), np.float32(0), s)
        o = bf16(np.float32(lo + np.float32(8) * s))
        inv = np.where(s > 0, np.float32(1) / np.where(s > 0, s, np.float32(1)), np.float32(0))
        n = np.rint(np.float32(g - o[..., None]) * inv[..., None]) + 8
    n = np.clip(np.where(bad[..., None], 8, n), 0, 15).astype(np.int64)
    return np.where(bad, np.float32(0), s), np.where(bad, np.float32(np.nan), o), n.reshape(x.shape)


def stored(x, gs):
    """What rows of x [..., hd] stand for once in the cache (64 bits)."""
    s, o, n = quantise(x, gs)
    g = n.reshape(*n.shape[:-1], -1, gs).astype(np.float64)
    return (o[..., None].astype(np.float64) + s[..., None].astype(np.float64) * (g - 8)).reshape(n.shape)


def attention(q, K, V, positions, scale, window=0):
    """q [m x q_heads x hd] at `positions` [m] of one sequence with stored K, V [len x heads x hd].

    Returns (out [m x q_heads x hd], slack): slack bounds, per output element, sum_t a_t |V_t - V_mean|-like
    magnitudes and the scores' size, for the tests' error bounds: (weighted mean of |V|, largest sum |q||K| scale).
    """
    m, hq, hd = q.shape
    heads = K.shape[1]
    out = np.zeros((m, hq, hd))
    mag = np.zeros((m, hq, hd))
    size = np.zeros((m, hq, 1))
    for i in range(m):
        p = int(positions[i])
        first = max(0, p - window + 1) if window else 0
        if p < 0 or first > p:
            continue
        for h in range(hq):
            k, v = K[first:p + 1, h // (hq // heads)], V[first:p + 1, h // (hq // heads)]
            x = scale * (k @ q[i, h].astype(np.float64))
            a = np.exp(x - x.max())
            a /= a.sum()
            out[i, h] = a @ v
            mag[i, h] = a @ np.abs(v)
            size[i, h] = abs(scale) * (np.abs(k) @ np.abs(q[i, h].astype(np.float64))).max()
    return out, mag, size


def norm_residual(block, resid, gate, alpha, w_post, w_pre, eps, gate_sigmoid=False):
    """(h, x) in 64 bits; x is None without w_pre."""
    f = lambda t: None if t is None else np.asarray(t, np.float64)  # noqa: E731
    block, resid, gate, w_post, w_pre = map(f, (block, resid, gate, w_post, w_pre))
    h = np.zeros_like(block if block is not None else resid)
    if block is not None:
        b = block
        if w_post is not None:
            b = b / np.sqrt((b * b).mean(-1, keepdims=True) + eps) * w_post
        if gate is not None:
            b = b * (1 / (1 + np.exp(-gate)) if gate_sigmoid else gate)
        h = alpha * b
    if resid is not None:
        h = resid + h
    return h, None if w_pre is None else h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w_pre
