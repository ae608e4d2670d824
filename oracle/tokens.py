"""CPU oracle for rotary positions, products with weights that are not quantised, and log probabilities.

TEST INFRASTRUCTURE ONLY (see oracle/moe.py for who may import the oracle). Plain numpy in 64 bits, written from the
definitions in include/coli_moe.h; it shares no code with the library.

Parity status: pinned by tests/test_tokens_oracle.py (worked cases, invariances).
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot, base, scaling="none", factor=1.0, original_len=0, low=1.0, high=32.0):
    """Radians per position of each pair."""
    out = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "base" and rot > 2 else base
        f = b ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            g = min(1.0, max(0.0, (original_len * f / (2 * math.pi) - low) / (high - low)))
            f = g * f + (1 - g) * f / factor
        out.append(f)
    return np.array(out)


def plan_positions(T, lens, q_start=None):
    """Position of each of T rows: None outside every sequence, negative before a sequence's first position."""
    pos = [None] * T
    for b, n in enumerate(lens):
        r0, r1 = (b, b + 1) if q_start is None else (q_start[b], q_start[b + 1])
        for r in range(r0, r1):
            pos[r] = n - r1 + r
    return pos


def rotary(x, turns, positions, interleaved=False, scale=1.0):
    """x [T x heads x hd] turned; turns [rot / 2] in 64-bit fractions of a turn per position (whole numbers)."""
    y = np.array(x, np.float64)
    half = len(turns)
    for r, p in enumerate(positions):
        for i, turn in enumerate(turns):
            part = int(turn) * int(p) % 2 ** 64  # exact
            angle = 2 * math.pi * (part / 2 ** 64)
            at = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
            a, b = np.array(x[r, :, at[0]], np.float64), np.array(x[r, :, at[1]], np.float64)
            y[r, :, at[0]] = scale * (a * math.cos(angle) - b * math.sin(angle))
            y[r, :, at[1]] = scale * (b * math.cos(angle) + a * math.sin(angle))
    return y


def act(z, kind):
    if kind == "silu":
        return z / (1 + np.exp(-z))
    if kind == "gelu":
        return z / 2 * np.vectorize(math.erfc)(-z / math.sqrt(2))
    if kind == "gelu_tanh":
        return z / 2 * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if kind == "relu":
        return np.maximum(z, 0)
    if kind == "relu2":
        return np.maximum(z, 0) ** 2
    return z


def linear(x, W, bias=None, kind="none", mul=None, resid=None):
    """(y, z, size): y [S x O]; z the argument of the activation; size = sum |W x| + |bias|, for error bounds."""
    x, W = np.asarray(x, np.float64), np.asarray(W, np.float64)
    z, size = x @ W.T, np.abs(x) @ np.abs(W).T
    if bias is not None:
        z, size = z + bias, size + np.abs(bias)
    y = act(z, kind)
    if mul is not None:
        y = y * np.asarray(mul, np.float64)
    return y if resid is None else y + np.asarray(resid, np.float64), z, size


def logprobs(x, scale=1.0):
    """(log p [S x V], entropy [S]) of rows of logits that may hold -infinity."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        top = x.max(-1, keepdims=True)
        z = np.where(x == -np.inf, -np.inf, scale * (x - np.where(top == -np.inf, 0, top)))
        e = np.exp(z)
        total = e.sum(-1, keepdims=True)
        lp = np.where(total > 0, z - np.log(np.where(total > 0, total, 1)), -np.inf)
        entropy = -np.where(e > 0, np.exp(lp) * np.where(e > 0, lp, 0), 0).sum(-1)
    return lp, entropy


def top(x, k):
    """Indices of the k largest entries of each row above -infinity, ties by index, -1 behind them."""
    out = []
    for row in np.asarray(x, np.float64):
        order = sorted((i for i in range(len(row)) if row[i] > -np.inf), key=lambda i: (-row[i], i))[:k]
        out.append(order + [-1] * (k - len(order)))
    return np.array(out, np.int64).reshape(len(out), k)
