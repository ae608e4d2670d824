"""Rotary positions against the 64-bit oracle: layouts, sizes, strides, where rows are, refusals."""
import numpy as np
import pytest
import torch

import oracle.tokens as O
from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import DT, as_dtype, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = Ctx()
    yield c.ctx
    c.close()


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def check(got, x, turns, positions, interleaved, scale, dtype):
    """The turn is found to 2^-32 and read to 2^-25 of a half turn (1e-7 of an angle), sine and cosine are good to 2^-22, and
    two products and a sum of them round to 2^-24 each: below 2^-20 of |scale| (|a| + |b|) together. Then one rounding."""
    want = O.rotary(x, turns, [0 if p is None or p < 0 else p for p in positions] if not isinstance(positions, np.ndarray) else positions,
                    interleaved, scale)
    half, T = len(turns), x.shape[0]
    size = np.zeros(x.shape)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        size[:, :, a] = size[:, :, b] = abs(scale) * (np.abs(x[:, :, a]) + np.abs(x[:, :, b]))
    last = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for r in range(T):
        p = positions[r]
        g = got[r].float().cpu().numpy()
        if p is None:
            assert (g == 7.0).all(), r  # left alone
        elif p < 0 and not isinstance(positions, np.ndarray):
            assert np.array_equal(g, x[r]), r  # copied
        else:
            off = np.abs(g - want[r]) - (size[r] * 2.0 ** -20 + last * np.abs(want[r]))
            assert (off <= 0).all(), (r, float(off.max()))
            assert np.array_equal(g[:, 2 * half:], x[r][:, 2 * half:])


def make(T, heads, hd, dtype, seed=0):
    return as_dtype(rng("rotary", T, heads, hd, seed).normal(size=(T, heads, hd)), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hd,rot", [(128, 128), (64, 32), (80, 36), (96, 38), (256, 256), (10, 6), (2, 2), (33, 8), (1024, 1024), (40, 24)])
def test_heads(ctx, hd, rot, interleaved, dtype):
    T, hq, hk = 5, 3, 2
    freqs = B.coli_rotary_freqs(rot, 10000.0)
    q, qt = make(T, hq, hd, dtype)
    k, kt = make(T, hk, hd, dtype, 1)
    pos = np.array([0, 1, 4097, 2 ** 31 - 1, -2 ** 31], np.int64)
    qo, ko = torch.full_like(qt, 7.0), torch.full_like(kt, 7.0)
    B.coli_rotary(ctx, qt, kt, freqs, qo, ko, positions=i32(pos.tolist()), interleaved=interleaved, scale=1.25)
    assert B.coli_check_error(ctx) == 0
    turns = freqs.cpu().numpy()
    check(qo, q, turns, pos, interleaved, 1.25, dtype)
    check(ko, k, turns, pos, interleaved, 1.25, dtype)


@pytest.mark.parametrize("hq,hk,hd,rot,interleaved", [(8400, 8100, 1022, 4, False), (16384, 16384, 8, 8, False), (16384, 1, 66, 64, True)])
def test_many_heads(ctx, hq, hk, hd, rot, interleaved):
    freqs = B.coli_rotary_freqs(rot, 10000.0)
    q, qt = make(2, hq, hd, "f32")
    k, kt = make(2, hk, hd, "f32", 1)
    pos = np.array([77, -5], np.int64)
    qo, ko = torch.full_like(qt, 7.0), torch.full_like(kt, 7.0)
    B.coli_rotary(ctx, qt, kt, freqs, qo, ko, positions=i32(pos.tolist()), interleaved=interleaved)
    assert B.coli_check_error(ctx) == 0
    check(qo, q, freqs.cpu().numpy(), pos, interleaved, 1.0, "f32")
    check(ko, k, freqs.cpu().numpy(), pos, interleaved, 1.0, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hk,hd,rot", [(70, 9, 4, 80, 38), (33, 100, 3, 130, 130), (3, 0, 2, 1022, 1022), (40, 1, 0, 6, 2), (5, 7, 7, 1023, 1022)])
def test_heads_that_are_no_whole_vectors(ctx, T, hq, hk, hd, rot, interleaved, dtype):
    """Runs of heads that start anywhere in a vector, outputs that start elsewhere, few and many heads, in place and apart."""
    freqs = B.coli_rotary_freqs(rot, 1000.0)
    pos = rng("runs", T).integers(-9000, 9000, size=T)
    sides = []
    for heads, out_shift in ((hq, 0), (hk, 3)):
        if not heads:
            sides.append((None, None, None))
            continue
        x, xt = make(T, heads, hd, dtype, heads)
        buf = torch.full((T * (heads * hd + 5) + 8,), 7.0, dtype=xt.dtype, device="cuda")
        out = buf[out_shift:out_shift + T * (heads * hd + 5)].view(T, -1)[:, :heads * hd].unflatten(1, (heads, hd))
        sides.append((x, xt, (buf, out)))
    q, k = sides
    B.coli_rotary(ctx, q[1], k[1], freqs, None if q[0] is None else q[2][1], None if k[0] is None else k[2][1],
                  positions=i32(pos.tolist()), interleaved=interleaved, scale=0.5)
    assert B.coli_check_error(ctx) == 0
    for x, xt, rest in (q, k):
        if x is None:
            continue
        buf, out = rest
        check(out, x, freqs.cpu().numpy(), pos, interleaved, 0.5, dtype)
        B.coli_rotary(ctx, xt, None, freqs, xt, None, positions=i32(pos.tolist()), interleaved=interleaved, scale=0.5)
        assert torch.equal(xt, out)
        out.fill_(7.0)
        assert (buf == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,hq,hk", [(1, 64, 8), (1, 1, 1), (300, 1, 1), (700, 5, 1), (65, 40, 3)])
def test_rows_and_heads(ctx, T, hq, hk, dtype):
    freqs = B.coli_rotary_freqs(16, 500.0)
    q, qt = make(T, hq, 16, dtype)
    k, kt = make(T, hk, 16, dtype, 1)
    pos = rng("positions", T).integers(-10 ** 6, 10 ** 6, size=T)
    qo, ko = torch.full_like(qt, 7.0), torch.full_like(kt, 7.0)
    B.coli_rotary(ctx, qt, kt, freqs, qo, ko, positions=i32(pos.tolist()))
    assert B.coli_check_error(ctx) == 0
    check(qo, q, freqs.cpu().numpy(), pos, False, 1.0, dtype)
    check(ko, k, freqs.cpu().numpy(), pos, False, 1.0, dtype)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("offset", [0, 1, 4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_of_a_fused_projection_in_place_and_apart(ctx, dtype, offset, interleaved):
    """q and k as slices of [q | k | v] rows with a gap of `offset` elements; what lies around them stays as it was."""
    T, hq, hk, hd = 9, 4, 2, 64
    freqs = B.coli_rotary_freqs(48, 10000.0)
    width = (hq + 2 * hk) * hd + offset
    x, xt = as_dtype(rng("fused", offset).normal(size=(T, width)), dtype)
    flat = torch.cat([xt.flatten(), xt.new_zeros(8)])
    lens, start = [4, 0, 1000], [0, 3, 3, 9]
    pos = O.plan_positions(T, lens, start)

    def parts(t):
        rows = t[offset:offset + T * width].as_strided((T, width), (width, 1))
        return rows[:, :hq * hd].unflatten(1, (hq, hd)), rows[:, hq * hd:(hq + hk) * hd].unflatten(1, (hk, hd))

    q, k = parts(flat)
    want = [t.float().cpu().numpy().astype(np.float64) for t in (q, k)]
    for apart in (True, False):
        out = torch.full_like(flat, 7.0) if apart else flat.clone()
        src = flat if apart else out
        B.coli_rotary(ctx, *parts(src), freqs, *parts(out), lens=i32(lens), q_start=i32(start), interleaved=interleaved)
        assert B.coli_check_error(ctx) == 0
        for g, w in zip(parts(out), want):
            check(g, w, freqs.cpu().numpy(), pos, interleaved, 1.0, dtype)
        rest = out.clone()
        for t in parts(rest):
            t.fill_(0)
        left = torch.full_like(flat, 7.0) if apart else flat.clone()
        for t in parts(left):
            t.fill_(0)
        assert torch.equal(rest, left)


def test_plans(ctx):
    """Empty sequences, rows before a sequence's first position, rows of no sequence, more sequences than a warp."""
    freqs = B.coli_rotary_freqs(32)
    for T, lens, start in ((7, [5, 2, 1], [0, 2, 2, 5]), (6, [0, 0, 3], [0, 0, 3, 6]), (4, [9], [1, 3]),
                           (200, list(range(100)), [2 * b for b in range(101)]), (40, [3] * 2000, [min(b, 40) for b in range(2001)])):
        x, xt = make(T, 2, 32, "f32")
        out = torch.full_like(xt, 7.0)
        B.coli_rotary(ctx, xt, None, freqs, out, None, lens=i32(lens), q_start=i32(start))
        assert B.coli_check_error(ctx) == 0
        check(out, x, freqs.cpu().numpy(), O.plan_positions(T, lens, start), False, 1.0, "f32")
    lens = [0, 7, 2 ** 31 - 1]
    x, xt = make(3, 2, 32, "bf16")
    out = torch.full_like(xt, 7.0)
    B.coli_rotary(ctx, None, xt, freqs, None, out, lens=i32(lens))
    assert B.coli_check_error(ctx) == 0
    check(out, x, freqs.cpu().numpy(), O.plan_positions(3, lens), False, 1.0, "bf16")


@pytest.mark.parametrize("lens,start,T", [([-1, 4], None, 2), ([4, 4], [0, 3, 5], 4), ([4, 4], [0, 3, 2], 4), ([4, 4], [-1, 2, 4], 4),
                                          ([4, -5], [0, 2, 4], 4)])
def test_plans_that_do_not_fit_are_reported(ctx, lens, start, T):
    """Nothing outside the arrays is touched: guard rows around the output stay."""
    freqs = B.coli_rotary_freqs(32)
    _, xt = make(T, 2, 32, "f32")
    out = torch.full((T + 4, 2, 32), 7.0, device="cuda")
    B.coli_rotary(ctx, xt, None, freqs, out[2:-2], None, lens=i32(lens), q_start=None if start is None else i32(start))
    assert B.coli_check_error(ctx) == B.COLI_E_RANGE
    assert (out[:2] == 7).all() and (out[-2:] == 7).all()
    assert B.coli_check_error(ctx) == 0


def test_turning_back_and_the_gradient(ctx):
    """Negated positions undo a turn, and <g, turn(x)> = <turn back(g), x>: the gradient; a difference quotient agrees."""
    freqs = B.coli_rotary_freqs(64)
    x, xt = make(6, 3, 64, "f32")
    g, gt = make(6, 3, 64, "f32", 5)
    pos = i32([0, 3, 100, 5000, 77777, 123456789])
    y, back, dx = (torch.empty_like(xt) for _ in range(3))
    B.coli_rotary(ctx, xt, None, freqs, y, None, positions=pos, scale=1.5)
    B.coli_rotary(ctx, gt, None, freqs, dx, None, positions=-pos, scale=1.5)
    B.coli_rotary(ctx, y, None, freqs, back, None, positions=-pos, scale=1 / 1.5)
    assert (back - xt).abs().max() < 2.0 ** -19 * 6  # two turns of values below 6
    d = torch.randn(xt.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    y2 = torch.empty_like(y)
    B.coli_rotary(ctx, xt + 0.5 * d, None, freqs, y2, None, positions=pos, scale=1.5)
    slope = (gt.double() * (y2.double() - y.double())).sum() / 0.5
    assert abs(float(slope - (dx.double() * d.double()).sum())) < 1e-3
    assert B.coli_check_error(ctx) == 0


def test_captured_with_new_positions_each_replay(ctx):
    freqs = B.coli_rotary_freqs(128)
    x, xt = make(3, 8, 128, "bf16")
    k, kt = make(3, 2, 128, "bf16", 1)
    out, ko, lens = torch.empty_like(xt), torch.empty_like(kt), i32([5, 9, 2])
    stream = torch.cuda.Stream()
    B.coli_rotary(ctx, xt, kt, freqs, out, ko, lens=lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    before = torch.cuda.current_stream()
    with torch.cuda.graph(graph, stream=stream):
        B.coli_set_stream(ctx, stream)
        B.coli_rotary(ctx, xt, kt, freqs, out, ko, lens=lens)
        lens += 1
    B.coli_set_stream(ctx, before)
    lens.copy_(i32([5, 9, 2]))
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        check(out, x, freqs.cpu().numpy(), [4 + step, 8 + step, 1 + step], False, 1.0, "bf16")
        check(ko, k, freqs.cpu().numpy(), [4 + step, 8 + step, 1 + step], False, 1.0, "bf16")
    assert B.coli_check_error(ctx) == 0


def test_refusals(ctx):
    freqs = B.coli_rotary_freqs(32)
    x = torch.zeros(4, 2, 32, device="cuda")
    o, pos = torch.zeros_like(x), i32([0, 1, 2, 3])

    def refused(*args, error=(B.ColiError, ValueError), **kw):
        with pytest.raises(error):
            B.coli_rotary(ctx, *args, **kw)

    refused(None, None, freqs, None, None, positions=pos)
    refused(x, None, freqs, None, None, positions=pos)
    refused(x, x, freqs, o, None, positions=pos)
    refused(x, None, freqs, o.bfloat16(), None, positions=pos)
    refused(x.half(), None, freqs, o.half(), None, positions=pos)
    refused(x.cpu(), None, freqs, o, None, positions=pos)
    refused(x, None, freqs.int(), o, None, positions=pos)
    refused(x, None, freqs, o, None, positions=pos[:3])
    refused(x, None, freqs, o, None, positions=pos.long())
    refused(x, None, freqs, o, None)
    refused(x, None, freqs, o, None, positions=pos, lens=pos)
    refused(x, None, freqs, o, None, lens=pos[:3])
    refused(x, None, freqs, o, None, lens=pos[:2], q_start=pos)
    refused(x, None, freqs, o, None, positions=pos, scale=float("nan"))
    refused(x, None, freqs, o, None, positions=pos, scale=float("inf"))
    refused(x, None, torch.zeros(17, dtype=torch.int64, device="cuda"), o, None, positions=pos)  # 34 of 32 channels
    refused(x, None, torch.zeros(0, dtype=torch.int64, device="cuda"), o, None, positions=pos)
    refused(x.transpose(1, 2), None, freqs, o.transpose(1, 2), None, positions=pos)
    refused(x[:1].expand(4, 2, 32), None, freqs, o, None, positions=pos)
    both = torch.zeros(5, 2, 32, device="cuda")
    refused(both[:4], None, freqs, both[1:], None, positions=pos)
    refused(x, x, freqs, o, o, positions=pos)
    refused(x, o, freqs, o, torch.zeros_like(x), positions=pos)
    refused(x, o, freqs, torch.zeros_like(x), x, positions=pos)
    assert B.coli_check_error(ctx) == 0
