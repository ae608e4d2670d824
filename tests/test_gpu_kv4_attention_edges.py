"""Attention over the 4-bit cache where numbers or places are at an end of their range: values of any size, what is not
finite and who sees it, windows of any size, pages that a window has left behind."""
import numpy as np
import pytest
import torch

import oracle.kv4 as O
from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import Batch, as_dtype, assert_within, bound, rng

pytestmark = pytest.mark.gpu

# (rows per sequence, query heads): one tile of up to 8 rows per key head, one of 9 to 16, and more rows
FORMS = [([1, 1], 8), ([1, 1], 24), ([70, 90], 8)]


@pytest.fixture(scope="module")
def ctx():
    c = Ctx()
    yield c.ctx
    c.close()


def within(b, out, ref, mag, size):
    assert_within(out, ref, bound(ref, mag, size, b.dtype, max(b.lens), np.abs(b.V).max()))


@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 2, (1 << 31) - 300, 1 << 30])
@pytest.mark.parametrize("dtype,hd", [("f32", 64), ("bf16", 64), ("bf16", 256)])
@pytest.mark.parametrize("rows", [[8, 60, 300], [8, 6, 3], [300, 9, 1]])
def test_a_window_as_large_as_an_int_is_none(ctx, rows, dtype, hd, window):
    """Sequences shorter than their rows among them: positions down to -297 less the window pass 32 bits."""
    b = Batch(ctx, [3, 40, 300], 1, hd, 64, 16, dtype)
    q, q_t = b.queries(rows, 2)
    out = b.attend(q_t, rows, window=window)
    assert B.coli_check_error(ctx) == 0
    assert torch.equal(out, b.attend(q_t, rows))
    within(b, out, *b.expect(q, rows))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_longest_sequence(ctx, dtype):
    """Two thousand million tokens, of which the last 600 are written and the windows see some; one more is an error."""
    n, page, heads, hd, gs = (1 << 31) - 256, 256, 2, 64, 32
    b = Batch(ctx, [600], heads, hd, gs, page, dtype, write=False)
    first = (n - 600) // page
    table = torch.full((1, (1 << 31) // page), -1, dtype=torch.int32, device="cuda")
    table[0, first:first + 4] = torch.tensor([2, 0, 3, 1], dtype=torch.int32)
    b.cache = B.coli_kv4_cache(4, page, heads, hd, gs)
    b.cache.data.fill_(255)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    B.coli_kv4_append(ctx, b.cache, b.k_t, b.v_t, lens, table, b.start_t)
    for rows, q_heads in (([1], 4), ([1], 24), ([70], 8)):
        q, q_t = b.queries(rows, q_heads)
        start = torch.from_numpy(b.q_start).cuda()
        out = torch.empty_like(q_t)
        B.coli_kv4_attention(ctx, b.cache, q_t, lens, table, out, q_start=start, window=300)
        assert B.coli_check_error(ctx) == 0
        within(b, out, *b.expect(q, rows, window=300))
        again = torch.empty_like(q_t)
        B.coli_kv4_attention(ctx, b.cache, q_t, lens + 1, table, again, q_start=start, window=300)
        assert B.coli_check_error(ctx) == B.COLI_E_RANGE
        assert torch.equal(out, again)  # of the clamped length
    k, v = torch.empty_like(b.k_t), torch.empty_like(b.v_t)
    B.coli_kv4_read(ctx, b.cache, k, v, lens, table, b.start_t)
    assert B.coli_check_error(ctx) == 0
    assert torch.equal(k.double().cpu(), torch.from_numpy(b.K).to(k.dtype).double())
    assert torch.equal(v.double().cpu(), torch.from_numpy(b.V).to(v.dtype).double())
    B.coli_kv4_read(ctx, b.cache, k, v, lens + 255, table, b.start_t)
    assert B.coli_check_error(ctx) == B.COLI_E_RANGE


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,q_heads", FORMS)
@pytest.mark.parametrize("v_scale", [1e-36, 2e-35])
def test_values_near_the_ends_of_binary32(ctx, v_scale, rows, q_heads, dtype):
    """Outputs of 1e-36 are normal numbers."""
    b = Batch(ctx, [77, 300], 2, 128, 64, 32, dtype, v_scale=v_scale)
    q, q_t = b.queries(rows, q_heads)
    out = b.attend(q_t, rows)
    assert B.coli_check_error(ctx) == 0
    within(b, out, *b.expect(q, rows))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,q_heads", FORMS)
def test_sums_of_values_near_the_upper_end(ctx, rows, q_heads, dtype):
    """Values of 1e35: a sum of 300 weights times them is finite, and so has to be every step on its way."""
    b = Batch(ctx, [77, 300], 2, 128, 64, 32, dtype, v_scale=1e35)
    q, q_t = b.queries(rows, q_heads)
    out = b.attend(q_t, rows)
    assert B.coli_check_error(ctx) == 0
    within(b, out, *b.expect(q, rows))


@pytest.mark.parametrize("v_scale", [1e-36, 1e35])
def test_sums_that_one_cta_finishes(ctx, v_scale):
    """More items than CTAs, so that many are finished where they are computed: 160 prompts of 140 rows over 900 tokens that
    weigh about the same, values around three times their spread."""
    b = Batch(ctx, [900] * 160, 1, 64, 64, 64, "bf16", k_scale=0.1, write=False)
    b.v = (v_scale * (3 + b.v)).astype(np.float32)
    B.coli_kv4_append(ctx, b.cache, b.k_t.float(), torch.from_numpy(b.v).cuda(), b.lens_t, b.table, b.start_t)
    b.V = O.stored(b.v, 64)
    rows = [140] * 160
    q, q_t = b.queries(rows, 1)
    out = b.attend(q_t, rows)
    assert B.coli_check_error(ctx) == 0
    within(b, out, *b.expect(q, rows))


def spoil(b, where, tokens, channels, value):
    """Write the batch's tokens again with `value` in some channels of the first head of one token of a sequence or more
    (through binary32, which holds every value); the oracle's keys or values follow."""
    k, v = torch.from_numpy(b.k.copy()), torch.from_numpy(b.v.copy())
    for t in tokens:
        (k if where == "keys" else v)[t, 0, channels] = value
    B.coli_kv4_append(b.ctx, b.cache, k.cuda(), v.cuda(), b.lens_t, b.table, b.start_t)
    b.K, b.V = O.stored(k.numpy(), b.gs), O.stored(v.numpy(), b.gs)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["keys", "values"])
@pytest.mark.parametrize("value", [3.4e38, -3.4e38])
@pytest.mark.parametrize("rows,q_heads,window", [([5], 2, 0), ([8], 4, 0), ([60], 4, 0), ([1], 4, 45), ([1], 24, 45), ([60], 4, 40)])
def test_what_is_infinite_in_masked_places_is_not_seen(ctx, rows, q_heads, window, value, where, dtype):
    """A whole group of 3.4e38 is finite, but its offset rounds to infinity. Rows before the token, and rows whose window has
    left it, are as without it."""
    b = Batch(ctx, [200], 2, 128, 32, 32, dtype)
    m = rows[0]
    token = 200 - m // 2 if m > 1 else 150
    spoil(b, where, [token], slice(32, 64), value)
    B.coli_check_error(ctx)
    q, q_t = b.queries(rows, q_heads)
    out = b.attend(q_t, rows, window=window)
    ref, mag, size = b.expect(q, rows, window=window)
    assert not np.isfinite(O.stored(np.full((1, 32), value, np.float32), 32)).any()
    p = 200 - m + np.arange(m)
    clear = (p < token) | ((p - window >= token) if window else False)
    assert clear.any()
    V = np.where(np.isfinite(b.V), b.V, 0)
    tol = bound(ref, mag, size, dtype, 200, np.abs(V).max())
    assert_within(out[torch.from_numpy(clear).cuda()], ref[clear], tol[clear])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,rows,q_heads", [([77, 300], [1, 1], 8), ([77, 300], [1, 1], 24), ([120, 300], [70, 90], 8),
                                               ([6000, 900], [1, 1], 8), ([6000, 900], [1, 1], 24), ([6000, 900], [20, 40], 8)])
def test_a_value_that_is_not_a_number_spoils_its_group_alone(ctx, lens, rows, q_heads, dtype):
    """The channels of the group, of the heads that share the key/value head, in the rows that see the token, however many
    rows there are and however the tokens are split."""
    b = Batch(ctx, lens, 2, 128, 32, 32, dtype)
    # before every row of sequence 0, and between the rows of sequence 1 (or before its only row)
    spoil(b, "values", [3], slice(40, 41), float("nan"))
    spoil(b, "values", [3, lens[0] + lens[1] - 1 - rows[1] // 2], slice(40, 41), float("nan"))
    assert B.coli_check_error(ctx) == B.COLI_E_NONFINITE
    q, q_t = b.queries(rows, q_heads)
    out = b.attend(q_t, rows).float().cpu().numpy().astype(np.float64)
    assert B.coli_check_error(ctx) == 0
    ref, mag, size = b.expect(q, rows)
    bad = np.isnan(ref)
    assert bad[:, :q_heads // 2, 32:64].any() and not bad[:, q_heads // 2:].any() and not bad[..., 64:].any()
    assert np.array_equal(np.isnan(out), bad)
    tol = bound(ref, mag, size, dtype, max(lens), np.nanmax(np.abs(b.V)))
    assert (np.abs(out - ref)[~bad] <= tol[~bad]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,rows,q_heads", [([77, 300], [1, 1], 8), ([77, 300], [1, 1], 24), ([120, 300], [70, 90], 8),
                                               ([6000, 900], [20, 40], 8)])
def test_a_key_that_is_not_a_number_spoils_its_heads_rows(ctx, lens, rows, q_heads, dtype):
    b = Batch(ctx, lens, 2, 128, 32, 32, dtype)
    spoil(b, "keys", [3, lens[0] + lens[1] - 1 - rows[1] // 2], slice(40, 41), float("nan"))
    assert B.coli_check_error(ctx) == B.COLI_E_NONFINITE
    q, q_t = b.queries(rows, q_heads)
    out = b.attend(q_t, rows).float().cpu().numpy().astype(np.float64)
    assert B.coli_check_error(ctx) == 0
    with np.errstate(invalid="ignore"):
        ref, mag, size = b.expect(q, rows)
    bad = np.isnan(ref)
    assert bad[:rows[0], :q_heads // 2].all() and not bad[:, q_heads // 2:].any()
    assert np.array_equal(np.isnan(out), bad)
    tol = bound(ref, mag, size, dtype, max(lens), np.abs(b.V).max())
    assert (np.abs(out - ref)[~bad] <= tol[~bad]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,q_heads", [([1, 1], 8), ([1, 1], 24), ([7, 3], 4), ([70, 90], 8), ([140, 20], 4)])
@pytest.mark.parametrize("page,window", [(16, 50), (64, 1), (16, 17), (32, 200)])
def test_pages_that_the_window_has_left_may_be_gone(ctx, page, window, rows, q_heads, dtype):
    """A server that gives back pages older than any row's window marks them as it likes."""
    b = Batch(ctx, [900, 333], 2, 128, 64, page, dtype)
    q, q_t = b.queries(rows, q_heads)
    with_all = b.attend(q_t, rows, window=window)
    gone = 0
    for i, (n, m) in enumerate(zip(b.lens, rows)):
        left = max(0, n - m - window + 1) // page  # whole pages before the first row's window
        b.table[i, :left] = torch.tensor([-1, b.cache.pages, -(1 << 31), (1 << 31) - 1], dtype=torch.int32).repeat(left)[:left].cuda()
        gone += left
    assert gone > 0
    out = b.attend(q_t, rows, window=window)
    assert B.coli_check_error(ctx) == 0
    assert torch.equal(out, with_all)
    within(b, out, *b.expect(q, rows, window=window))


@pytest.mark.parametrize("T", [1, 3])
def test_out_over_q_is_refused_and_slices_beside_it_are_not(ctx, T):
    b = Batch(ctx, [50, 90, 7][:T], 2, 128, 64, 16, "bf16")
    _, q = b.queries([1] * T, 4)
    row = 4 * 128
    want = b.attend(q, [1] * T)
    buf = torch.zeros(8 * T * row, dtype=q.dtype, device="cuda")

    def rows(at, stride):
        return buf.as_strided((T, 4, 128), (stride, 128, 1), at)

    base = 4 * row
    # places of out: on q, a little before and after it, on its last row, between its rows but too near
    for stride, at, out_stride in ((row, base, row), (row, base + 1, row), (row, base - 1, row), (row, base + T * row - 1, row),
                                   (row, base - T * row + 1, row), (2 * row + 1, base + row - 1, 2 * row + 1),
                                   (2 * row, base + row // 2, row + 3)):
        if T == 1 and abs(at - base) >= row:
            continue
        with pytest.raises(B.ColiError) as e:
            B.coli_kv4_attention(ctx, b.cache, rows(base, stride), b.lens_t, b.table, rows(at, out_stride))
        assert e.value.code == B.COLI_E_INVAL and "overlaps" in B.coli_last_error(ctx)
    for stride, at, out_stride in ((row, base + T * row, row), (row, base - T * row, row), (2 * row, base + row, 2 * row),
                                   (2 * row, base - row, 2 * row), (2 * row + 1, base + row, 2 * row + 1), (2 * row, 0, row)):
        buf.zero_()
        q2, out = rows(base, stride), rows(at, out_stride)
        q2.copy_(q)
        B.coli_kv4_attention(ctx, b.cache, q2, b.lens_t, b.table, out)
        assert torch.equal(out, want) and torch.equal(q2, q)
    assert B.coli_check_error(ctx) == 0


def test_queries_count_down_to_two_to_the_minus_27_of_their_largest(ctx):
    """bf16 queries are held in 16 bits at a common power of two per row. A channel of 1 beside channels of about 2^-27 that
    meet keys of 2^27, while the 1 meets keys of 0: every bit of the small ones is in the scores."""
    r = rng("spread")
    n, hd, gs = 60, 128, 32
    b = Batch(ctx, [n], 1, hd, gs, 16, "bf16", write=False)
    k = 2.0 ** 27 * r.normal(size=(n, 1, hd))
    k[..., :gs] = 0
    b.k, b.k_t = as_dtype(k, "bf16")
    B.coli_kv4_append(ctx, b.cache, b.k_t, b.v_t, b.lens_t, b.table, b.start_t)
    b.K = O.stored(b.k, gs)
    for m, heads in ((1, 8), (1, 16), (30, 8)):
        q = r.choice([-1.0, 1.0], size=(m, heads, hd)) * r.integers(128, 256, size=(m, heads, hd)) * 2.0 ** -34
        q[..., 0] = 1
        b.queries([m], heads)  # the rows' place
        q, q_t = as_dtype(q, "bf16")
        assert np.array_equal(q[..., 1:] * 2.0 ** 34, np.rint(q[..., 1:] * 2.0 ** 34))
        out = b.attend(q_t, [m], scale=0.25)
        assert B.coli_check_error(ctx) == 0
        within(b, out, *b.expect(q, [m], scale=0.25))
