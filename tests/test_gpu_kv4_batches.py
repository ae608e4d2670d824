"""Batches beyond a few sequences, and calls of which one CTA has a long stretch: paths that depend on how many sequences,
rows or stages there are."""
import numpy as np
import pytest
import torch

import oracle.kv4 as O
from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import Batch, as_dtype, assert_within, bound, rng
from test_gpu_kv4 import read_all, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = Ctx()
    yield c.ctx
    c.close()


def lengths(n, most):
    return [int(x) for x in rng("lengths", n).integers(0, most, n)]


def check(b, rows, q_heads, window=0):
    q, q_t = b.queries(rows, q_heads)
    out = b.attend(q_t, rows, window=window)
    ref, mag, size = b.expect(q, rows, window=window)
    assert B.coli_check_error(b.ctx) == 0
    assert_within(out, ref, bound(ref, mag, size, b.dtype, max(b.lens), np.abs(b.V).max()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [31, 32, 33, 200, 1500])
def test_rows_of_many_sequences_are_written_and_read_back(ctx, n, dtype):
    """From 32 sequences on a warp searches for its rows' sequence."""
    b = Batch(ctx, lengths(n, 12), 3, 64, 32, 16, dtype)
    k, v = read_all(b)
    assert B.coli_check_error(ctx) == 0
    assert np.array_equal(k[:sum(b.lens)], rounded(b.K, dtype)) and np.array_equal(v[:sum(b.lens)], rounded(b.V, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [160, 161, 400])
def test_one_token_of_many_sequences(ctx, n, dtype):
    """Above 160 sequences the streaming form deals its work out in rounds."""
    check(Batch(ctx, lengths(n, 150), 2, 64, 32, 16, dtype), [1] * n, 6)


@pytest.mark.parametrize("n", [512, 513, 1100])
def test_prompts_of_many_sequences(ctx, n):
    """Above 512 sequences the tensor-core form keeps its counts in pieces. Rows from none to more than there are tokens."""
    rows = [int(x) for x in rng("rows", n).integers(0, 9, n)]
    check(Batch(ctx, lengths(n, 40), 1, 64, 32, 16, "bf16"), rows, 8)


def test_a_prompt_among_many_decoding_sequences(ctx):
    """One chunk of a prompt among sequences of one row: together they take the tensor-core form."""
    n = 70
    lens = [40 + x for x in lengths(n, 200)]
    lens[33] = 700
    check(Batch(ctx, lens, 2, 128, 64, 64, "bf16"), [1] * 33 + [260] + [1] * (n - 34), 8)


@pytest.mark.parametrize("dtype,hd,gs,q_heads", [("bf16", 64, 64, 8), ("bf16", 128, 32, 8), ("bf16", 64, 64, 16), ("f32", 64, 64, 8)])
def test_more_than_64_stages_of_an_item_in_a_cta(ctx, dtype, hd, gs, q_heads):
    """160 requests over the same 30000 tokens (shared pages), less a few each: a CTA has about 150 stages, so that sums
    move to shared memory twice and, as the scores grow along the sequence, are rescaled there."""
    n, B_ = 30000, 160
    b = Batch(ctx, [n], 1, hd, gs, 64, dtype, write=False)
    b.k, b.k_t = as_dtype(b.k * np.linspace(0.2, 2.5, n)[:, None, None], dtype)
    B.coli_kv4_append(ctx, b.cache, b.k_t, b.v_t, b.lens_t, b.table, b.start_t)
    b.K = O.stored(b.k, gs)
    lens = [n - 37 * i for i in range(B_)]
    q, q_t = as_dtype(rng("shared", hd, q_heads).normal(size=(B_, q_heads, hd)), dtype)
    out = torch.empty_like(q_t)
    B.coli_kv4_attention(ctx, b.cache, q_t, torch.tensor(lens, dtype=torch.int32).cuda(), b.table.repeat(B_, 1), out)
    assert B.coli_check_error(ctx) == 0
    parts = [O.attention(q[i:i + 1], b.K[:m], b.V[:m], [m - 1], hd ** -0.5) for i, m in enumerate(lens)]
    ref, mag, size = (np.concatenate(x) for x in zip(*parts))
    assert_within(out, ref, bound(ref, mag, size, dtype, n, np.abs(b.V).max()))


@pytest.mark.parametrize("hd,gs", [(64, 64), (128, 32)])
@pytest.mark.parametrize("q_heads", [1, 8, 16])
def test_values_that_cancel_leave_what_32_bits_leave(ctx, hd, gs, q_heads):
    """Every second token has its neighbour's key and the negative of its value, all of them eighths, so that a bf16 call's
    rounded weights cancel too and the output is 0 (its own rounding then hides nothing). A sum of products whose terms are
    all of one sign, at most 8 s = 1 times the sum of the weights, loses less than 2^-23 of itself with each step that is
    cut off: 2^-19.9 over 16 steps as it grows, and once more as much below for the terms and the sums after."""
    n, B_, s = 30000, 160, 0.125
    r = rng("balanced", hd, gs)
    codes = r.integers(1, 16, (n // 2, 1, hd))
    codes = np.stack([codes, 16 - codes], 1).reshape(n, 1, hd)
    codes[..., ::gs], codes[..., 1::gs] = 0, 15  # of each group, so that its scale is s and its offset 0
    b = Batch(ctx, [n], 1, hd, gs, 64, "bf16", write=False)
    _, k_t = as_dtype(np.repeat(r.normal(size=(n // 2, 1, hd)), 2, 0), "bf16")
    v, v_t = as_dtype(s * (codes - 8), "bf16")
    assert np.array_equal(O.stored(v, gs), v)
    B.coli_kv4_append(ctx, b.cache, k_t, v_t, b.lens_t, b.table, b.start_t)
    _, q_t = as_dtype(1.2 * r.normal(size=(B_, q_heads, hd)), "bf16")
    out = torch.empty_like(q_t)
    B.coli_kv4_attention(ctx, b.cache, q_t, torch.tensor([n - 2 * i for i in range(B_)], dtype=torch.int32).cuda(),
                         b.table.repeat(B_, 1), out)
    assert B.coli_check_error(ctx) == 0
    out = out.float().cpu().numpy()
    fixed = np.arange(hd) % gs < 2
    assert np.abs(out[..., fixed] - v[0, 0, fixed]).max() <= 2.0 ** -9
    assert np.abs(out[..., ~fixed]).max() <= 2.0 ** -18.9
