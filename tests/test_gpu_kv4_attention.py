"""Attention over the 4-bit cache against the 64-bit oracle: head layouts, lengths, pages, windows, rows that see
nothing, strides, streams, refusals."""
import numpy as np
import pytest
import torch

from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import DT, Batch, assert_within, bound
from test_gpu_kv4 import SHAPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = Ctx()
    yield c.ctx
    c.close()


def check(b, rows, q_heads, window=0, scale=None, q_scale=1.0):
    q, q_t = b.queries(rows, q_heads, scale=q_scale)
    out = b.attend(q_t, rows, scale=scale, window=window)
    ref, mag, size = b.expect(q, rows, scale=scale, window=window)
    assert B.coli_check_error(b.ctx) == 0
    assert_within(out, ref, bound(ref, mag, size, b.dtype, max(b.lens), np.abs(b.V).max()), f"{b.lens} {rows} heads {q_heads}/{b.heads}")
    return q_t, out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,gs", SHAPES)
def test_every_head_shape(ctx, hd, gs, dtype):
    check(Batch(ctx, [1, 15, 16, 17, 64, 65, 200], 2, hd, gs, 16, dtype), [1] * 7, 8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,group", [(1, 1), (4, 1), (2, 3), (1, 8), (2, 9), (1, 16), (1, 40), (1, 64)])
def test_every_group_of_query_heads(ctx, heads, group, dtype):
    check(Batch(ctx, [130, 33], heads, 128, 64, 32, dtype), [1, 1], heads * group)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_every_page_size_and_lengths_around_its_end(ctx, page, dtype):
    check(Batch(ctx, [page - 1, page, page + 1, 3 * page + 5], 2, 64, 64, page, dtype), [1] * 4, 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,rows", [
    ([0], [1]), ([0, 5, 0], [1, 1, 1]), ([7, 3, 100], [7, 3, 100]), ([300], [300]), ([90, 40], [1, 40]),
    ([5, 200, 64], [0, 65, 64]), ([3, 1], [5, 4]), ([1000, 2], [17, 2]), ([129, 257, 1], [129, 129, 1]), ([600], [200]),
])
def test_prompts_drafts_and_rows_that_see_nothing(ctx, lens, rows, dtype):
    b = Batch(ctx, lens, 2, 128, 32, 16, dtype)
    q_t, out = check(b, rows, 6)
    for i, (n, m) in enumerate(zip(lens, rows)):
        for j in range(max(0, m - n)):
            assert bool((out[int(b.q_start[i]) + j] == 0).all())


@pytest.mark.parametrize("hd,gs", [(64, 64), (128, 32)])
@pytest.mark.parametrize("rows", [[31, 32, 33], [63, 64, 65, 1], [97, 127, 128, 129], [161, 255, 256, 257]])
def test_tiles_that_end_around_a_warp(ctx, hd, gs, rows):
    """Query rows per head one below, at and one above what fills a warp, a half and a tile of the tensor-core form."""
    check(Batch(ctx, [300 - 7 * i for i in range(len(rows))], 1, hd, gs, 16, "bf16"), rows, 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 5000])
@pytest.mark.parametrize("rows", [1, 6, 150])
def test_windows(ctx, window, rows, dtype):
    check(Batch(ctx, [400, 150, 151], 1, 64, 32, 64, dtype), [rows] * 3, 4, window=window)


@pytest.mark.parametrize("hd,gs", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_prompt_of_every_width(ctx, hd, gs, dtype):
    check(Batch(ctx, [700, 130], 2, hd, gs, 64, dtype), [260, 130], 8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_long_sequence_is_joined_from_many_parts(ctx, dtype):
    check(Batch(ctx, [9001], 1, 128, 64, 64, dtype), [1], 8)
    check(Batch(ctx, [5000, 1, 2500], 2, 64, 32, 16, dtype), [1, 1, 1], 2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k_scale,v_scale,scale", [(1.0, 1e-6, None), (1.0, 1e4, None), (30.0, 1.0, 1.0), (1e-3, 1.0, None),
                                                   (1.0, 1.0, 0.0), (1.0, 1.0, -0.1), (1e4, 1e-12, 1e-5), (1.0, 1e25, None)])
def test_sizes_of_keys_values_and_scale(ctx, k_scale, v_scale, scale, dtype):
    b = Batch(ctx, [77, 300], 2, 128, 64, 32, dtype, k_scale=k_scale, v_scale=v_scale)
    check(b, [1, 1], 8, scale=scale)
    check(b, [70, 90], 8, scale=scale)


def test_values_that_grow_along_the_sequence(ctx):
    """Each stretch of tokens is louder than everything before it, so that every running quantity is rescaled."""
    for dtype in ("f32", "bf16"):
        b = Batch(ctx, [512], 1, 64, 32, 16, dtype, write=False)
        grow = torch.logspace(-6, 6, 512, device="cuda").view(-1, 1, 1)
        for t, name in ((b.v_t, "v"), (b.k_t, "k")):
            t.copy_(t * (grow if name == "v" else torch.linspace(0.1, 3, 512, device="cuda").view(-1, 1, 1)))
        import oracle.kv4 as O
        b.K, b.V = (O.stored(t.float().cpu().numpy(), 32) for t in (b.k_t, b.v_t))
        B.coli_kv4_append(ctx, b.cache, b.k_t, b.v_t, b.lens_t, b.table, b.start_t)
        check(b, [1], 4)
        check(b, [130], 4)


def test_rows_apart_and_any_alignment(ctx):
    for dtype in ("f32", "bf16"):
        for rows in ([1, 1, 1], [4, 70, 1]):
            b = Batch(ctx, [50, 90, 7], 2, 128, 64, 16, dtype)
            q, q_t = b.queries(rows, 6)
            T, wide = q_t.shape[0], 6 * 128 + 11
            buf = torch.zeros(T * wide + 1, dtype=DT[dtype], device="cuda")[1:].view(T, wide)
            qs = buf[:, 3:3 + 768].unflatten(1, (6, 128))
            qs.copy_(q_t)
            res = torch.full((T * wide + 1,), 9.0, dtype=DT[dtype], device="cuda")[1:].view(T, wide)
            out = b.attend(qs, rows, out=res[:, 5:5 + 768].unflatten(1, (6, 128)))
            assert torch.equal(out, b.attend(q_t, rows))
            assert bool((res[:, :5] == 9).all()) and bool((res[:, 5 + 768:] == 9).all())
            ref, mag, size = b.expect(q, rows)
            assert_within(out, ref, bound(ref, mag, size, dtype, max(b.lens), np.abs(b.V).max()))


def test_results_repeat_and_follow_the_stream(ctx):
    b = Batch(ctx, [4000, 123, 0, 1], 2, 128, 64, 64, "bf16")
    for rows in ([1] * 4, [200, 100, 0, 1]):
        _, q_t = b.queries(rows, 8)
        first = b.attend(q_t, rows)
        for _ in range(5):
            assert torch.equal(first, b.attend(q_t, rows))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        B.coli_set_stream(ctx, side)
        try:
            with torch.cuda.stream(side):
                q2 = q_t * 1.0  # made on the side stream just before
                again = b.attend(q2, rows)
            side.synchronize()
        finally:
            B.coli_set_stream(ctx, torch.cuda.current_stream())
        assert torch.equal(first, again)


def test_a_step_replays_as_a_graph(ctx):
    b = Batch(ctx, [300, 77], 2, 128, 64, 32, "bf16")
    _, q_t = b.queries([1, 1], 8)
    out = b.attend(q_t, [1, 1])
    eager = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    rows = [int(b.start[i + 1]) - 1 for i in range(2)]
    k, v = b.k_t[rows].contiguous(), b.v_t[rows].contiguous()
    try:
        with torch.cuda.graph(graph, stream=side):
            B.coli_set_stream(ctx, torch.cuda.current_stream())
            B.coli_kv4_append(ctx, b.cache, k, v, b.lens_t, b.table)
            b.attend(q_t, [1, 1], out=out)
    finally:
        B.coli_set_stream(ctx, torch.cuda.current_stream())
    out.zero_()
    for _ in range(3):
        graph.replay()
    assert torch.equal(out, eager) and B.coli_check_error(ctx) == 0


def test_a_query_that_is_not_finite_spoils_its_row_alone(ctx):
    for dtype in ("f32", "bf16"):
        for rows in ([1, 1], [30, 80]):
            b = Batch(ctx, [300, 80], 1, 64, 32, 16, dtype)
            _, q_t = b.queries(rows, 4)
            good = b.attend(q_t, rows)
            q_t[0, 2, 5] = float("nan")
            out = b.attend(q_t, rows)
            assert bool(out[0, 2].isnan().all())
            out[0, 2], good[0, 2] = 0, 0
            assert torch.equal(out, good)
            assert B.coli_check_error(ctx) == B.COLI_E_NONFINITE


def test_a_masked_token_that_is_not_finite_is_not_seen(ctx):
    """NaN keys and values after a row's position, or before its window, leave it alone."""
    for dtype in ("f32", "bf16"):
        b = Batch(ctx, [200], 1, 64, 32, 16, dtype, write=False)
        for t in (b.k_t, b.v_t):
            t[190:] = float("nan")
            t[:20] = float("nan")
        B.coli_kv4_append(ctx, b.cache, b.k_t, b.v_t, b.lens_t, b.table, b.start_t)
        assert B.coli_check_error(ctx) == B.COLI_E_NONFINITE
        for m in (30, 100):
            q, q_t = b.queries([m], 4)
            out = b.attend(q_t, [m], window=60)
            fine = 190 - (200 - m)
            assert bool(out[:fine][max(0, 80 - (200 - m)):].isfinite().all())
            assert bool(out[fine:].isnan().all())


def test_a_page_outside_the_cache_is_reported(ctx):
    for rows in ([1, 1], [40, 100]):
        b = Batch(ctx, [300, 100], 1, 64, 32, 16, "bf16")
        _, q_t = b.queries(rows, 4)
        good = b.attend(q_t, rows)
        b.table[0, 3] = b.cache.pages + 5
        out = b.attend(q_t, rows)
        assert B.coli_check_error(ctx) == B.COLI_E_RANGE
        assert torch.equal(out[rows[0]:], good[rows[0]:])  # the other sequence is as it was
        b.lens_t[0] = 1 << 30
        out = b.attend(q_t, rows)
        assert B.coli_check_error(ctx) == B.COLI_E_RANGE
        assert torch.equal(out[rows[0]:], good[rows[0]:])


def test_refusals(ctx):
    b = Batch(ctx, [4, 4], 2, 64, 32, 16, "f32")
    _, q = b.queries([1, 1], 4)
    out = torch.empty_like(q)
    ok = lambda **k: B.coli_kv4_attention(ctx, b.cache, **{**dict(q=q, lens=b.lens_t, table=b.table, out=out), **k})  # noqa: E731
    ok()
    for wrong in (dict(q=q[:, :3], out=out[:, :3]), dict(out=out.bfloat16()), dict(out=out[:1]), dict(scale=float("nan")),
                  dict(scale=float("inf")), dict(window=-1), dict(q=q.half(), out=out.half()), dict(q=q.cpu()),
                  dict(q_start=b.start_t[:2]), dict(table=b.table.long())):
        with pytest.raises((ValueError, B.ColiError)):
            ok(**wrong)
    lib = B.library()
    call = lambda **k: lib.coli_kv4_attention(*{**dict(ctx=ctx, c=b.cache, q=q.data_ptr(), qs=256, dt=0, h=4, T=2, st=None,  # noqa: E731
                                                       lens=b.lens_t.data_ptr(), B=2, table=b.table.data_ptr(), w=b.width,
                                                       scale=0.1, win=0, out=out.data_ptr(), os=256), **k}.values())
    assert call() == 0
    for wrong in (dict(q=None), dict(out=None), dict(c=None), dict(qs=255), dict(os=10), dict(h=5), dict(h=0), dict(h=2 * 65),
                  dict(dt=7), dict(T=1), dict(T=0), dict(B=70000, T=70000), dict(out=out.data_ptr() + 1)):
        assert call(**wrong) == B.COLI_E_INVAL, wrong
        assert B.coli_last_error(ctx).startswith("kv4_attention")
    assert B.coli_check_error(ctx) == 0


@pytest.mark.parametrize("rows", [[1, 1], [40, 100]])
def test_a_wait_that_gives_up_is_reported_and_leaves_the_context_usable(rows):
    """The first copy of a call is withheld: the waits on it give up (limit 20 ms), the call ends with an error, and the next
    call on the same context is right again."""
    c = Ctx.with_env(COLI_TEST_WAIT_NS=20_000_000, COLI_TEST_WITHHOLD=1)
    try:
        b = Batch(c.ctx, [3000, 1500], 2, 128, 64, 64, "bf16")
        _, q_t = b.queries(rows, 8)
        b.attend(q_t, rows)
        assert B.coli_check_error(c.ctx) == B.COLI_E_TIMEOUT
        check(b, rows, 8)
    finally:
        B.coli_destroy(c.ctx)
