"""The 4-bit key/value cache on the GPU: what is written and read back is the format's, bit for bit."""
import numpy as np
import pytest
import torch

import oracle.kv4 as O
from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import DT, Batch, as_dtype, rng

pytestmark = pytest.mark.gpu

SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 64), (256, 128)]


@pytest.fixture(scope="module")
def ctx():
    c = Ctx()
    yield c.ctx
    c.close()


def rounded(x, dtype):
    """64-bit values that fit 20 bits, as the dtype holds them."""
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).float().numpy()


def read_all(b):
    k, v = (torch.full((max(1, sum(b.lens)), b.heads, b.hd), 7.0, dtype=DT[b.dtype], device="cuda") for _ in range(2))
    B.coli_kv4_read(b.ctx, b.cache, k, v, b.lens_t, b.table, b.start_t)
    return k.float().cpu().numpy(), v.float().cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,gs", SHAPES)
@pytest.mark.parametrize("page,heads,lens", [(16, 3, [1, 0, 16, 17, 33]), (64, 1, [63, 65, 130]), (256, 2, [300])])
def test_read_gives_back_what_the_codes_stand_for(ctx, hd, gs, page, heads, lens, dtype):
    b = Batch(ctx, lens, heads, hd, gs, page, dtype)
    k, v = read_all(b)
    assert B.coli_check_error(ctx) == 0
    assert np.array_equal(k, rounded(b.K, dtype)) and np.array_equal(v, rounded(b.V, dtype))


def test_tokens_written_one_by_one_equal_those_written_at_once(ctx):
    lens = [37, 5, 18]
    b = Batch(ctx, lens, 2, 128, 64, 16, "bf16")
    c = Batch(ctx, lens, 2, 128, 64, 16, "bf16", write=False)
    for step in range(max(lens)):
        now = [min(n, step + 1) for n in lens]
        rows = [c.start[i] + now[i] - 1 for i in range(3)]  # a sequence that has ended writes its last token again
        B.coli_kv4_append(ctx, c.cache, c.k_t[rows], c.v_t[rows], torch.tensor(now, dtype=torch.int32).cuda(), c.table)
    for x, y in zip(read_all(b), read_all(c)):
        assert np.array_equal(x, y)
    assert torch.equal(b.cache.data, c.cache.data)  # every other byte still as it was filled
    assert B.coli_check_error(ctx) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,hd,gs", [(8, 64, 32), (4, 128, 64), (2, 256, 128)])
def test_many_rows_at_once_equal_those_written_in_pieces(ctx, heads, hd, gs, dtype):
    """Thousands of rows, which a warp takes several at a time (tokens that share words among them), against pieces of a
    few hundred, most of them from an odd token on."""
    lens = [1501, 3, 700, 0, 513]
    b = Batch(ctx, lens, heads, hd, gs, 32, dtype)
    c = Batch(ctx, lens, heads, hd, gs, 32, dtype, write=False)
    for i, n in enumerate(lens):
        for at in range(0, n, 301):
            to = min(n, at + 301)
            rows = slice(int(c.start[i]) + at, int(c.start[i]) + to)
            B.coli_kv4_append(ctx, c.cache, c.k_t[rows], c.v_t[rows], torch.tensor([to], dtype=torch.int32).cuda(),
                              c.table[i:i + 1], torch.tensor([0, to - at], dtype=torch.int32).cuda())
    assert torch.equal(b.cache.data, c.cache.data)
    k, v = read_all(b)
    assert B.coli_check_error(ctx) == 0
    assert np.array_equal(k, rounded(b.K, dtype)) and np.array_equal(v, rounded(b.V, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slices_of_a_fused_projection_at_any_alignment(ctx, dtype):
    """k and v as slices of wider rows that start off any vector boundary; the read-back goes into such slices too."""
    heads, hd, T = 2, 128, 21
    wide = 3 * heads * hd + 13
    b = Batch(ctx, [T], heads, hd, 32, 16, dtype, write=False)
    buf = torch.zeros(T * wide + 1, dtype=DT[dtype], device="cuda")[1:].view(T, wide)
    ks, vs = (buf[:, o:o + heads * hd].unflatten(1, (heads, hd)) for o in (5, 5 + heads * hd))
    ks.copy_(b.k_t)
    vs.copy_(b.v_t)
    B.coli_kv4_append(ctx, b.cache, ks, vs, b.lens_t, b.table, b.start_t)
    out = torch.full((T * wide + 1,), 3.0, dtype=DT[dtype], device="cuda")[1:].view(T, wide)
    ko, vo = (out[:, o:o + heads * hd].unflatten(1, (heads, hd)) for o in (7, 7 + heads * hd))
    B.coli_kv4_read(ctx, b.cache, ko, vo, b.lens_t, b.table, b.start_t)
    assert np.array_equal(ko.float().cpu().numpy(), rounded(b.K, dtype))
    assert np.array_equal(vo.float().cpu().numpy(), rounded(b.V, dtype))
    assert bool((out[:, :7] == 3).all()) and bool((out[:, 7 + 2 * heads * hd:] == 3).all())
    assert B.coli_check_error(ctx) == 0


def test_rows_before_the_sequence_and_rows_of_no_sequence(ctx):
    """Sequence 0 has 3 rows but 1 token: two rows store nothing and read zeros. Rows past q_start[B] are left alone."""
    b = Batch(ctx, [1, 4], 1, 64, 32, 16, "f32", write=False)
    _, x = as_dtype(rng("rows").normal(size=(9, 1, 64)), "f32")
    qs = torch.tensor([0, 3, 7], dtype=torch.int32).cuda()
    B.coli_kv4_append(ctx, b.cache, x, x, b.lens_t, b.table, qs)
    k, v = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
    B.coli_kv4_read(ctx, b.cache, k, v, b.lens_t, b.table, qs)
    ref = rounded(O.stored(x.cpu().numpy(), 32), "f32")
    for y in (k.cpu().numpy(), v.cpu().numpy()):
        assert (y[:2] == 0).all() and np.array_equal(y[2:7], ref[2:7]) and (y[7:] == 5).all()
    assert B.coli_check_error(ctx) == 0


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3.3e38])
def test_a_group_that_is_not_finite_is_kept_as_nan_and_reported(ctx, value):
    b = Batch(ctx, [3], 1, 128, 32, 16, "f32", write=False)
    k = b.k_t.clone()
    k[1, 0, 40] = value
    if value == 3.3e38:
        k[1, 0, 41] = -value  # finite, but the span is not
    B.coli_kv4_append(ctx, b.cache, k, b.v_t, b.lens_t, b.table, b.start_t)
    kr, vr = read_all(b)
    ref = rounded(O.stored(k.cpu().numpy(), 32), "f32")
    assert np.isnan(ref[1, 0, 32:64]).all() and np.array_equal(kr, ref, equal_nan=True)
    assert np.array_equal(vr, rounded(b.V, "f32"))
    assert B.coli_check_error(ctx) == B.COLI_E_NONFINITE
    assert B.coli_check_error(ctx) == 0


@pytest.mark.parametrize("scale", [1e-37, 1e-20, 1e20, 1e37])
def test_the_whole_range_of_binary32(ctx, scale):
    b = Batch(ctx, [40], 1, 64, 64, 32, "f32", k_scale=scale, v_scale=scale)
    k, v = read_all(b)
    assert np.array_equal(k, rounded(b.K, "f32")) and np.array_equal(v, rounded(b.V, "f32"))
    assert B.coli_check_error(ctx) == 0


def test_bad_lengths_pages_and_row_ranges_are_reported_and_touch_nothing_else(ctx):
    b = Batch(ctx, [20, 20], 1, 64, 32, 16, "f32")
    before = b.cache.data.clone()
    x = b.k_t[:2].contiguous()
    bad = lambda **k: torch.tensor(k["v"], dtype=torch.int32).cuda()  # noqa: E731
    table = b.table.clone()
    table[0, 1], table[1, 1] = b.cache.pages, -1  # both tokens fall on pages outside the cache
    B.coli_kv4_append(ctx, b.cache, x, x, b.lens_t, table)
    assert B.coli_check_error(ctx) == B.COLI_E_RANGE and torch.equal(before, b.cache.data)
    k, v = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
    B.coli_kv4_read(ctx, b.cache, k, v, b.lens_t, table)
    assert B.coli_check_error(ctx) == B.COLI_E_RANGE and bool((k == 0).all()) and bool((v == 0).all())
    B.coli_kv4_append(ctx, b.cache, x, x, bad(v=[-3, 0]), b.table)  # no such positions
    assert B.coli_check_error(ctx) == B.COLI_E_RANGE and torch.equal(before, b.cache.data)
    B.coli_kv4_read(ctx, b.cache, k, v, bad(v=[1000, 20]), b.table)  # clamped to the table's 32 positions
    assert B.coli_check_error(ctx) == B.COLI_E_RANGE
    for qs in ([0, 2, 3], [-1, 1, 2], [2, 1, 2]):
        B.coli_kv4_append(ctx, b.cache, x, x, bad(v=[0, 0]), b.table, bad(v=qs))
        assert B.coli_check_error(ctx) == B.COLI_E_RANGE and torch.equal(before, b.cache.data)


def test_refusals(ctx):
    assert B.coli_kv4_bytes(4, 64, 2, 128, 64) == 4 * 64 * 2 * (128 + 16)
    for shape in ((0, 64, 1, 128, 64), (1, 48, 1, 128, 64), (1, 64, 0, 128, 64), (1, 64, 257, 128, 64),
                  (1, 64, 1, 96, 32), (1, 64, 1, 128, 16), (1, 64, 1, 64, 128), (1, 64, 1, 256, 32),
                  (1 << 25, 64, 1, 64, 32)):
        assert B.coli_kv4_bytes(*shape) == 0
        with pytest.raises(ValueError):
            B.coli_kv4_cache(*shape)
    b = Batch(ctx, [4, 4], 2, 64, 32, 16, "f32")
    one = b.k_t[:2].contiguous()
    ok = lambda **k: B.coli_kv4_append(ctx, b.cache, **{**dict(k=one, v=one, lens=b.lens_t, table=b.table), **k})  # noqa: E731
    ok()
    for wrong in (dict(k=one.half(), v=one.half()), dict(k=one.double(), v=one.double()), dict(v=one.bfloat16()),
                  dict(k=one[:1]), dict(k=one.cpu()), dict(k=one.transpose(0, 1)), dict(k=one[..., ::2]),
                  dict(lens=b.lens_t.long()), dict(table=b.table[:1]), dict(table=b.table.flatten()),
                  dict(q_start=b.lens_t), dict(k=b.k_t, v=b.v_t)):
        with pytest.raises((ValueError, B.ColiError)):
            ok(**wrong)
    lib, st = B.library(), b.cache
    call = lambda **k: lib.coli_kv4_append(*{**dict(ctx=ctx, c=st, k=one.data_ptr(), ks=128, v=one.data_ptr(), vs=128, dt=0,  # noqa: E731
                                                    T=2, qs=None, lens=b.lens_t.data_ptr(), B=2, table=b.table.data_ptr(),
                                                    w=b.width), **k}.values())
    assert call() == 0
    for wrong in (dict(c=None), dict(k=None), dict(lens=None), dict(table=None), dict(ks=127), dict(vs=0), dict(dt=2),
                  dict(T=0), dict(T=3), dict(B=0), dict(w=0), dict(k=one.data_ptr() + 2), dict(T=1 << 25, B=1 << 25)):
        assert call(**wrong) == B.COLI_E_INVAL, wrong
        assert B.coli_last_error(ctx).startswith("kv4_append")
    assert lib.coli_kv4_append(None, st, one.data_ptr(), 128, one.data_ptr(), 128, 0, 2, None, b.lens_t.data_ptr(), 2,
                               b.table.data_ptr(), b.width) == B.COLI_E_INVAL
    assert B.coli_check_error(ctx) == 0
