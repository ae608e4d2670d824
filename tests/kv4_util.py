"""Helpers of the cache and attention tests: a batch of sequences on pages, and the oracle's answers."""
from __future__ import annotations

import numpy as np
import torch

import oracle.kv4 as O
from int4_grouped_expert_router_gb300 import binding as B

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rng(*key):
    return np.random.default_rng([20261206, *[abs(hash_of(k)) for k in key]])


def hash_of(k):
    return k if isinstance(k, int) else sum(ord(ch) * 131 ** i for i, ch in enumerate(str(k))) % (1 << 31)


def as_dtype(a, dtype):
    """A numpy array as the dtype holds it: (values in binary32, the tensor on the GPU)."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DT[dtype])
    return t.float().numpy(), t.cuda()


class Batch:
    """Sequences of the given lengths on shuffled pages of a cache filled with bytes of all ones (NaN scales and
    offsets in every place that no token was written to)."""

    def __init__(self, ctx, lens, heads, hd, gs, page, dtype, seed=0, k_scale=1.0, v_scale=1.0, spare=2, write=True):
        self.ctx, self.lens, self.heads, self.hd, self.gs, self.page, self.dtype = ctx, lens, heads, hd, gs, page, dtype
        r = rng("batch", seed, heads, hd, gs, page, *lens)
        used = [-(-n // page) for n in lens]
        pages = sum(used) + spare
        self.width = max(1, max(used))
        order = r.permutation(pages)
        self.table_np = np.zeros((len(lens), self.width), np.int32)
        at = 0
        for b, n in enumerate(used):
            self.table_np[b, :n] = order[at:at + n]
            at += n
        total = max(1, sum(lens))
        self.k, self.k_t = as_dtype(k_scale * (r.normal(size=(total, heads, hd)) + r.normal(size=(heads, hd))), dtype)
        self.v, self.v_t = as_dtype(v_scale * r.normal(size=(total, heads, hd)), dtype)
        self.start = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
        self.lens_t = torch.tensor(lens, dtype=torch.int32).cuda()
        self.table = torch.from_numpy(self.table_np).cuda()
        self.start_t = torch.from_numpy(self.start).cuda()
        self.cache = B.coli_kv4_cache(pages, page, heads, hd, gs)
        self.cache.data.fill_(255)
        if write and sum(lens):
            B.coli_kv4_append(ctx, self.cache, self.k_t, self.v_t, self.lens_t, self.table, self.start_t)
        self.K, self.V = O.stored(self.k, gs), O.stored(self.v, gs)

    def queries(self, rows, q_heads, seed=0, scale=1.0):
        r = rng("queries", seed, q_heads, *rows)
        self.q_start = np.concatenate(([0], np.cumsum(rows))).astype(np.int32)
        return as_dtype(scale * r.normal(size=(int(self.q_start[-1]), q_heads, self.hd)), self.dtype)

    def expect(self, q, rows, scale=None, window=0):
        scale = self.hd ** -0.5 if scale is None else scale
        parts = []
        for b, (n, m) in enumerate(zip(self.lens, rows)):
            s = slice(self.start[b], self.start[b] + n)
            qs = self.q_start[b]
            parts.append(O.attention(q[qs:qs + m], self.K[s], self.V[s], n - m + np.arange(m), scale, window))
        return tuple(np.concatenate(x) for x in zip(*parts))

    def attend(self, q_t, rows, scale=None, window=0, out=None):
        one = all(m == 1 for m in rows)
        out = torch.full_like(q_t, float("nan")) if out is None else out
        B.coli_kv4_attention(self.ctx, self.cache, q_t, self.lens_t, self.table, out,
                             q_start=None if one else torch.from_numpy(self.q_start).cuda(), scale=scale, window=window)
        return out


def bound(ref, mag, size, dtype, tokens, largest):
    """How far an output may be off, element by element. A score that is e off (in natural units) moves its weight by
    a factor exp(e), and the output by at most 2 e times the weighted mean of |V|. Scores: sum |q||K| scale times the
    relative error of a product sum in binary32 (256 terms: 2^-16 at the very worst, 2^-19 as sums of mixed sign go),
    queries held in 22 bits at least. Weights: 11 bits (bf16) or 22, and none smaller than 2^-38 of the largest (what a
    16-bit float can hold), so each token may be off by that much of the largest |V|. The output is rounded to the dtype
    once."""
    least = tokens * 2.0 ** -38 * largest
    if dtype == "bf16":
        return least + 2.0 ** -8 * np.abs(ref) + mag * (2.0 ** -10 + 2 * size * 2.0 ** -16)
    return least + 2.0 ** -22 * np.abs(ref) + mag * (2.0 ** -19 + 2 * size * 2.0 ** -19)


def assert_within(got, ref, tol, what=""):
    got = got.float().cpu().numpy().astype(np.float64)
    assert got.shape == ref.shape
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - ref) - tol
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.size} outside, worst by {over.max():.3g} at {np.unravel_index(over.argmax(), over.shape)}"
