"""Products with 16-bit weights and their epilogue against the 64-bit oracle."""
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


def weight(ctx, O_, I, scale=0.05):
    W, Wt = as_dtype(scale * rng("weight", O_, I).normal(size=(O_, I)), "bf16")
    return W, B.coli_dense_upload(ctx, Wt)


def close(got, x, W, bias, kind, mul, resid, y, x_dtype="bf16"):
    """Products are exact (binary32 activations: three parts of 8 bits). A sum of I of them in binary32, in steps of 16 and
    joined at most 64 times, each step cut off to 2^-23 of what it has reached: (I / 16 + 64) 2^-23 of sum |W x|, three
    times the steps for three parts. The activations' slopes stay below 1.2 (relu2: 2 |z|), their own error below 2^-20;
    in norm a chunk of at most 32 steps may lose 32 * 2^-24, its sum with the others as much again."""
    want, z, size = O.linear(x, W, bias, kind, mul, resid)
    I = x.shape[1]
    dz = size * (I / 16 * (3 if x_dtype == "f32" else 1) + 64) * 2.0 ** -23
    slope = 2 * (np.abs(z) + dz) if kind == "relu2" else 1.2
    a = np.abs(O.act(z, kind))
    m = 1.0 if mul is None else np.abs(mul)
    last = 2.0 ** -8 if y == "bf16" else 2.0 ** -23
    tol = m * (slope * dz + 2.0 ** -20 * a + 1e-37) + last * np.abs(want)
    g = got.float().cpu().numpy()
    off = np.abs(g - want) - tol
    assert (off <= 0).all(), (float(off.max()), np.unravel_index(off.argmax(), off.shape))
    if y == "f32" and kind == "none" and mul is None and g.size > 500 and I >= 16:
        assert np.linalg.norm(g - want) <= 4e-6 * np.linalg.norm(want)


def run(ctx, S, I, O_, x_dtype="bf16", y="f32", kind="none", bias=False, mul=False, resid=False, seed=0):
    r = rng("dense", S, I, O_, seed)
    W, h = weight(ctx, O_, I)
    x, xt = as_dtype(r.normal(size=(S, I)), x_dtype)
    b, bt = as_dtype(r.normal(size=O_), "f32") if bias else (None, None)
    m, mt = as_dtype(r.normal(size=(S, O_)), y) if mul else (None, None)
    q, qt = as_dtype(r.normal(size=(S, O_)), y) if resid else (None, None)
    guard = torch.full((S + 2, O_), 7.0, dtype=DT[y], device="cuda")
    yt = guard[1:-1]
    B.coli_dense_linear(ctx, h, xt, yt, bias=bt, act=kind, mul=mt, resid=qt)
    assert B.coli_check_error(ctx) == 0
    B.coli_dense_free(ctx, h)
    assert (guard[0] == 7).all() and (guard[-1] == 7).all()
    close(yt, x, W, b, kind, m, q, y, x_dtype)
    return yt


@pytest.mark.parametrize("x_dtype,y", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("S,I,O_", [(1, 1, 1), (1, 64, 128), (1, 1000, 300), (2, 63, 127), (5, 65, 129), (16, 256, 256), (17, 640, 200),
                                    (33, 127, 1000), (64, 512, 130), (65, 192, 384), (100, 2048, 96), (129, 320, 257),
                                    (257, 100, 140), (300, 1024, 260), (600, 72, 515), (1, 6144, 257), (8, 4104, 129)])
def test_sizes(ctx, S, I, O_, x_dtype, y):
    run(ctx, S, I, O_, x_dtype, y)


@pytest.mark.parametrize("S,I,O_,x_dtype,y", [(2700, 100, 4700, "bf16", "bf16"), (2500, 130, 3100, "f32", "f32"), (1100, 70, 20001, "bf16", "f32"),
                                              (4100, 64, 2049, "f32", "bf16"), (1, 300, 60001, "bf16", "bf16"), (40, 700, 19457, "bf16", "f32"),
                                              (256, 256, 38912, "bf16", "bf16")])
def test_many_tiles(ctx, S, I, O_, x_dtype, y):
    """Several tiles for every share, whole and split ones, token tiles of more than one group, and none left to split."""
    run(ctx, S, I, O_, x_dtype, y, "relu", bias=True, resid=True)


@pytest.mark.parametrize("y", ["bf16", "f32"])
@pytest.mark.parametrize("kind", list(B.ACTIVATIONS))
@pytest.mark.parametrize("S", [1, 20, 150])
def test_epilogues(ctx, S, kind, y):
    for bias, mul, resid in ((True, False, False), (False, True, False), (False, False, True), (True, True, True)):
        run(ctx, S, 192, 200, "bf16", y, kind, bias, mul, resid)


@pytest.mark.parametrize("kind", list(B.ACTIVATIONS))
def test_activations_over_their_whole_range(ctx, kind):
    """W = 1 x 1: the product is exact, so the activation's own error shows: 2^-20 relative, or 1e-37."""
    h = B.coli_dense_upload(ctx, torch.ones(1, 1, dtype=torch.bfloat16))
    z = np.concatenate((np.linspace(-30, 30, 4001), [0, -0.0, 1e-30, -1e-30, 88.5, -88.5, 200, -200, 1e18, -1e18])).astype(np.float32)
    if kind == "gelu":
        z = z[np.abs(z) > 0]
    zt, y = torch.from_numpy(z[:, None]).cuda(), torch.empty(len(z), 1, device="cuda")
    B.coli_dense_linear(ctx, h, zt, y, act=kind)
    assert B.coli_check_error(ctx) == 0
    with np.errstate(all="ignore"):
        want = O.act(z.astype(np.float64), kind)
    if kind == "gelu_tanh":  # 1 + tanh(u) as 2 / (1 + exp(-2u)): no cancellation for u below 0
        u = np.sqrt(2 / np.pi) * (z.astype(np.float64) + 0.044715 * z.astype(np.float64) ** 3)
        with np.errstate(all="ignore"):
            want = z / (1 + np.exp(-2 * u))
        rel = 2.0 ** -20 * (1 + np.abs(np.minimum(2 * u, 0)))  # the exponential's argument rounds
    else:
        # erfc and exp of an argument that rounds: relative errors grow with its square, its size
        rel = 2.0 ** -20 + {"gelu": 2.0 ** -22 * np.square(np.minimum(z, 0)), "silu": 2.0 ** -23 * np.abs(np.minimum(z, 0))}.get(kind, 0)
    off = np.abs(y.cpu().numpy()[:, 0] - want) - (rel * np.abs(want) + 1e-37)
    assert (off <= 0).all(), (kind, z[off.argmax()], float(off.max()))
    B.coli_dense_free(ctx, h)


@pytest.mark.parametrize("x_dtype,y", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("S", [1, 3, 40, 280])
def test_strides_offsets_and_in_place(ctx, S, x_dtype, y):
    I, O_ = 200, 136
    r = rng("strides", S)
    W, h = weight(ctx, O_, I)
    for gap, offset in ((0, 1), (5, 0), (8, 8), (3, 3)):
        x, xt = as_dtype(r.normal(size=(S, I)), x_dtype)
        m, mt = as_dtype(r.normal(size=(S, O_)), y)
        q, qt = as_dtype(r.normal(size=(S, O_)), y)

        def spread(t):
            buf = torch.full((S * (t.shape[1] + gap) + 16,), 7.0, dtype=t.dtype, device="cuda")
            view = buf[offset:offset + S * (t.shape[1] + gap)].view(S, -1)[:, :t.shape[1]]
            view.copy_(t)
            return buf, view

        for place in ("apart", "resid", "mul"):
            bx, vx = spread(xt)
            bm, vm = spread(mt)
            bq, vq = spread(qt)
            by, vy = {"apart": spread(torch.zeros_like(qt)), "resid": (bq, vq), "mul": (bm, vm)}[place]
            B.coli_dense_linear(ctx, h, vx, vy, mul=vm, resid=vq, act="silu")
            assert B.coli_check_error(ctx) == 0
            close(vy, x, W, None, "silu", m, q, y, x_dtype)
            vy.fill_(7.0)
            assert (by == 7).all(), place
    B.coli_dense_free(ctx, h)


def test_a_fused_projection_and_slices_of_one_buffer(ctx):
    """x and y as column slices of the same rows."""
    S, I, O_ = 30, 128, 192
    W, h = weight(ctx, O_, I)
    x, xt = as_dtype(rng("one buffer").normal(size=(S, I)), "bf16")
    buf = torch.zeros(S, I + O_, dtype=torch.bfloat16, device="cuda")
    buf[:, :I] = xt
    B.coli_dense_linear(ctx, h, buf[:, :I], buf[:, I:])
    assert B.coli_check_error(ctx) == 0
    close(buf[:, I:], x, W, None, "none", None, None, "bf16")
    assert torch.equal(buf[:, :I], xt)
    B.coli_dense_free(ctx, h)


@pytest.mark.parametrize("x_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", [1, 20, 300])
def test_what_is_not_finite_stays_in_its_row(ctx, S, x_dtype):
    I, O_ = 300, 260
    W, h = weight(ctx, O_, I)
    x, xt = as_dtype(rng("broken", S).normal(size=(S, I)), x_dtype)
    clean = torch.empty(S, O_, device="cuda")
    B.coli_dense_linear(ctx, h, xt, clean)
    assert B.coli_check_error(ctx) == 0
    for bad in (float("nan"), float("inf"), float("-inf")):
        xb, row = xt.clone(), S // 2
        xb[row, 77] = bad
        y = torch.empty(S, O_, device="cuda")
        B.coli_dense_linear(ctx, h, xb, y)
        assert B.coli_check_error(ctx) == B.COLI_E_NONFINITE
        rest = [t for t in range(S) if t != row]
        assert torch.equal(y[rest], clean[rest])
        assert not torch.isfinite(y[row]).any()
        if bad != bad or x_dtype == "f32":
            continue
        sign = torch.from_numpy(np.sign(W[:, 77])).cuda() * (1 if bad > 0 else -1)
        assert torch.equal(torch.sign(y[row]), sign.float())
    B.coli_dense_free(ctx, h)
    W[5, 7] = np.inf
    h = B.coli_dense_upload(ctx, torch.from_numpy(W).bfloat16())
    y = torch.empty(S, O_, device="cuda")
    B.coli_dense_linear(ctx, h, xt, y)
    assert B.coli_check_error(ctx) == B.COLI_E_NONFINITE
    keep = [o for o in range(O_) if o != 5]
    assert torch.equal(y[:, keep], clean[:, keep]) and not torch.isfinite(y[:, 5]).any()
    B.coli_dense_free(ctx, h)


def test_binary32_activations_keep_their_24_bits(ctx):
    """x = 1 + 2^-23 against W = 1: the last bit of x arrives; and the largest values do not overflow."""
    h = B.coli_dense_upload(ctx, torch.eye(64, dtype=torch.bfloat16))
    for S in (1, 64):
        x = torch.full((S, 64), 1.0, device="cuda") + 2.0 ** -23
        x[0, :4] = torch.tensor([3.4e38, -3.4028234e38, 1e-30, -1.2345678e-20])
        y = torch.empty_like(x)
        B.coli_dense_linear(ctx, h, x, y)
        assert B.coli_check_error(ctx) == 0
        assert torch.equal(x, y)
    B.coli_dense_free(ctx, h)


def test_uploads_from_host_and_device_in_pieces(ctx):
    """A weight of more than one piece of the upload's buffer, and one that is not a whole number of tiles."""
    for O_, I in ((2300, 32768), (1, 9), (130, 7)):
        g = torch.Generator().manual_seed(O_)
        W = (0.02 * torch.randn(O_, I, generator=g)).bfloat16()
        x = torch.randn(3, I, generator=g).bfloat16().cuda()
        ys = []
        for src in (W, W.cuda()):
            h = B.coli_dense_upload(ctx, src)
            assert B.coli_dense_shape(ctx, h) == (O_, I)
            del src
            y = torch.empty(3, O_, device="cuda")
            B.coli_dense_linear(ctx, h, x, y)
            assert B.coli_check_error(ctx) == 0
            B.coli_dense_free(ctx, h)
            ys.append(y)
        assert torch.equal(*ys)
        want = x.double() @ W.cuda().double().t()
        assert (ys[0] - want).norm() <= 8e-6 * want.norm()


@pytest.mark.parametrize("S,I,O_", [(1, 2048, 384), (24, 1024, 1000), (300, 512, 700)])
def test_runs_give_the_same_bits_and_captures_replay(ctx, S, I, O_):
    _, h = weight(ctx, O_, I)
    xt = torch.randn(S, I, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    xb = xt.bfloat16()
    y, z = torch.empty(S, O_, device="cuda"), torch.empty(S, O_, device="cuda")
    B.coli_dense_linear(ctx, h, xt, y)
    B.coli_dense_linear(ctx, h, xb, z)
    first = y.clone(), z.clone()
    for _ in range(10):
        B.coli_dense_linear(ctx, h, xt, y)
        B.coli_dense_linear(ctx, h, xb, z)
        assert torch.equal(y, first[0]) and torch.equal(z, first[1])
    stream, before, graph = torch.cuda.Stream(), torch.cuda.current_stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        B.coli_set_stream(ctx, stream)
        B.coli_dense_linear(ctx, h, xt, y)
        B.coli_dense_linear(ctx, h, xb, z)
    B.coli_set_stream(ctx, before)
    for _ in range(3):
        y.zero_(), z.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first[0]) and torch.equal(z, first[1])
    assert B.coli_check_error(ctx) == 0
    B.coli_dense_free(ctx, h)


def test_refusals(ctx):
    with pytest.raises(ValueError):
        B.coli_dense_upload(ctx, torch.zeros(4, 4))
    with pytest.raises(ValueError):
        B.coli_dense_upload(ctx, torch.zeros(4, 4, dtype=torch.bfloat16).t()[:3])
    with pytest.raises(B.ColiError):
        B.coli_dense_upload(ctx, torch.zeros(1, 40000, dtype=torch.bfloat16))
    h = B.coli_dense_upload(ctx, torch.zeros(8, 16, dtype=torch.bfloat16))
    x, y = torch.zeros(4, 16, device="cuda"), torch.zeros(4, 8, device="cuda")
    b = torch.zeros(8, device="cuda")

    def refused(x, y, handle=h, **kw):
        with pytest.raises((B.ColiError, ValueError)):
            B.coli_dense_linear(ctx, handle, x, y, **kw)

    refused(x, y, 0)
    refused(x, y, h + 1)
    refused(x[:, :8], y)
    refused(x, y[:3])
    refused(x.cpu(), y)
    refused(x.half(), y)
    refused(x, y.half())
    refused(x, y, act="swish")
    refused(x, y, bias=b[:7])
    refused(x, y, bias=b.bfloat16())
    refused(x, y, mul=y.bfloat16())
    refused(x, y, resid=torch.zeros(4, 9, device="cuda"))
    refused(torch.zeros(16, 4, device="cuda").t(), y)
    refused(x[:1].expand(4, 16), y)
    refused(x, y[:1].expand(4, 8))
    refused(x, x[:, :8])
    both = torch.zeros(5, 8, device="cuda")
    refused(x, both[1:], resid=both[:4])
    refused(x, both[1:], mul=both[:4])
    refused(torch.zeros(0, 16, device="cuda"), torch.zeros(0, 8, device="cuda"))
    B.coli_dense_free(ctx, h)
    refused(x, y)
    with pytest.raises(B.ColiError):
        B.coli_dense_free(ctx, h)
    assert B.coli_check_error(ctx) == 0


@pytest.mark.parametrize("x_dtype,y", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("S,I,O_", [(60, 1030, 4001), (300, 320, 6100), (600, 700, 4000), (2100, 1030, 5001), (700, 2050, 12001),
                                    (260, 6144, 9001), (100, 2048, 6144), (512, 2048, 6144), (225, 76, 53865), (396, 66, 61170),
                                    (134, 73, 82442)])
def test_every_tile_of_tokens(ctx, S, I, O_, x_dtype, y):
    """Sizes at which tiles of 32, 64, 128 tokens and pairs of CTAs with 64, 128 and more are chosen, shared by CTAs or not, and a weight larger than
    L2 that two tiles of tokens read in step. In norm: see close(); a bf16 result rounds to 2^-9 on average."""
    g = torch.Generator(device="cuda").manual_seed(S)
    W = (0.05 * torch.randn(O_, I, device="cuda", generator=g)).bfloat16()
    x = torch.randn(S, I, device="cuda", generator=g).to(DT[x_dtype])
    bias, resid = torch.randn(O_, device="cuda", generator=g), torch.randn(S, O_, device="cuda", generator=g).to(DT[y])
    guard = torch.full((S + 2, O_), 7.0, dtype=DT[y], device="cuda")
    h = B.coli_dense_upload(ctx, W)
    B.coli_dense_linear(ctx, h, x, guard[1:-1], bias=bias, act="relu", resid=resid)
    assert B.coli_check_error(ctx) == 0
    want = torch.relu(x.double() @ W.double().t() + bias.double()) + resid.double()
    off = guard[1:-1].double() - want
    assert off.norm() <= (4e-6 if y == "f32" else 2.0 ** -8) * want.norm()
    size = x.double().abs() @ W.double().abs().t() + bias.abs().double()
    steps = I / 16 * (3 if x_dtype == "f32" else 1) + 64
    assert ((off.abs() - size * steps * 2.0 ** -23 - want.abs() * (2.0 ** -8 if y == "bf16" else 2.0 ** -23)) <= 0).all()
    assert (guard[0] == 7).all() and (guard[-1] == 7).all()
    again = torch.empty_like(guard[1:-1])
    B.coli_dense_linear(ctx, h, x, again, bias=bias, act="relu", resid=resid)
    assert torch.equal(again, guard[1:-1])
    B.coli_dense_free(ctx, h)


@pytest.mark.parametrize("S,I,O_,x_dtype", [(1, 2048, 3000, "bf16"), (1, 64, 100, "bf16"), (3, 2048, 3000, "f32"), (60, 1030, 4001, "f32"),
                                            (2100, 1030, 5001, "bf16")])
def test_a_copy_that_never_comes_ends_the_waits(S, I, O_, x_dtype):
    """A copy is withheld once: the waits on it give up, the call reports it, and the next one is healthy."""
    c = Ctx.with_env(COLI_TEST_WAIT_NS=20_000_000, COLI_TEST_WITHHOLD=1)
    try:
        g = torch.Generator(device="cuda").manual_seed(S)
        W = (0.05 * torch.randn(O_, I, device="cuda", generator=g)).bfloat16()
        x = torch.randn(S, I, device="cuda", generator=g).to(DT[x_dtype])
        y = torch.empty(S, O_, device="cuda")
        h = B.coli_dense_upload(c.ctx, W)
        B.coli_dense_linear(c.ctx, h, x, y)
        assert B.coli_check_error(c.ctx) == B.COLI_E_TIMEOUT
        for _ in range(2):
            B.coli_dense_linear(c.ctx, h, x, y)
            assert B.coli_check_error(c.ctx) == 0
            want = x.double() @ W.double().t()
            assert (y - want).norm() <= 4e-6 * want.norm()
    finally:
        c.close()


def test_reserve_is_enough_and_moves_nothing():
    """After coli_reserve a captured product outlives larger ones: nothing is allocated, nothing moves."""
    c = Ctx()
    try:
        B.coli_reserve(c.ctx, 300, 16, 4, 2048, 512)
        x = torch.randn(40, 1000, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
        _, h = weight(c.ctx, 700, 1000)
        _, big = weight(c.ctx, 600, 2048)
        y, z, xb = torch.empty(40, 700, device="cuda"), torch.empty(300, 600, device="cuda"), torch.randn(300, 2048, device="cuda")
        B.coli_dense_linear(c.ctx, h, x, y)
        first = y.clone()
        stream, before, graph = torch.cuda.Stream(), torch.cuda.current_stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            B.coli_set_stream(c.ctx, stream)
            B.coli_dense_linear(c.ctx, h, x, y)
        B.coli_set_stream(c.ctx, before)
        B.coli_dense_linear(c.ctx, big, xb, z)
        torch.cuda.synchronize()
        free = torch.cuda.mem_get_info()[0]
        B.coli_dense_linear(c.ctx, big, xb, z)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first) and torch.cuda.mem_get_info()[0] == free
        assert B.coli_check_error(c.ctx) == 0
    finally:
        c.close()
