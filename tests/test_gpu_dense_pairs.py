"""Products with 16-bit weights by pairs of CTAs: any number of stage refills, calls one behind another, strides and outputs in place where
tiles are whole, split and in groups, and copies that never come. The sizes are such that pairs are chosen on 152 SMs; whatever is chosen,
the answers are the same."""
import pytest
import torch

from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import DT

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")]


@pytest.fixture(scope="module")
def ctx():
    c = Ctx()
    yield c.ctx
    c.close()


def make(ctx, S, I, O_, x_dtype):
    g = torch.Generator(device="cuda").manual_seed(1000 * S + I)
    W = (0.05 * torch.randn(O_, I, device="cuda", generator=g)).bfloat16()
    x = torch.randn(S, I, device="cuda", generator=g).to(DT[x_dtype])
    return B.coli_dense_upload(ctx, W), x, x.double() @ W.double().t()


def close(y, want, I, x_dtype):
    """In norm. A bf16 result rounds by at most 2^-8; a sum of I products is cut off at each of at most I / 16 + 64 steps (three times as
    many for three parts) by at most 2^-23 of what it has reached, which in norm is no larger than the whole."""
    steps = I / 16 * (3 if x_dtype == "f32" else 1) + 64
    assert (y.double() - want).norm() <= ((2.0 ** -8 if y.dtype == torch.bfloat16 else 0) + steps * 2.0 ** -23) * want.norm()


@pytest.mark.parametrize("x_dtype,y", TYPES)
@pytest.mark.parametrize("I", [64, 192, 512, 576, 1280, 1920, 2496])
def test_stages_filled_any_number_of_times_and_calls_behind_one_another(ctx, I, x_dtype, y):
    """Stages of both CTAs are filled once to ten times, odd and even numbers. What follows at once, on the same SMs, takes their memory."""
    h, x, want = make(ctx, 512, I, 6144, x_dtype)
    one, x1, want1 = make(ctx, 1, 640, 2000, "bf16")
    ys, zs = ([torch.empty(*w.shape, dtype=dt, device="cuda") for _ in range(12)] for w, dt in ((want, DT[y]), (want1, torch.float32)))
    for a, b in zip(ys, zs):
        B.coli_dense_linear(ctx, h, x, a)
        B.coli_dense_linear(ctx, one, x1, b)
    assert B.coli_check_error(ctx) == 0
    close(ys[0], want, I, x_dtype)
    close(zs[0], want1, 640, "bf16")
    assert all(torch.equal(a, ys[0]) for a in ys) and all(torch.equal(b, zs[0]) for b in zs)
    for handle in (h, one):
        B.coli_dense_free(ctx, handle)


@pytest.mark.parametrize("x_dtype,y", TYPES)
@pytest.mark.parametrize("S,I,O_", [(300, 6144, 2100), (2100, 1030, 5001), (700, 2050, 12001), (2048, 520, 2500)])
def test_strides_and_outputs_in_place(ctx, S, I, O_, x_dtype, y):
    """Rows with gaps, at any alignment, outputs in place of the factor and of the residual: the bits of contiguous rows."""
    h, x, z = make(ctx, S, I, O_, x_dtype)
    g = torch.Generator(device="cuda").manual_seed(5)
    mul, resid = (torch.randn(S, O_, device="cuda", generator=g).to(DT[y]) for _ in range(2))
    plain = torch.empty(S, O_, dtype=DT[y], device="cuda")
    B.coli_dense_linear(ctx, h, x, plain, act="relu", mul=mul, resid=resid)
    assert B.coli_check_error(ctx) == 0
    # the factor and the residual add a rounding each, within the steps that are counted
    close(plain, torch.relu(z) * mul.double() + resid.double(), I, x_dtype)

    def spread(t, gap, offset):
        width = t.shape[1] + gap
        buf = torch.full((S * width + 16,), 7.0, dtype=t.dtype, device="cuda")
        view = buf[offset:offset + S * width].view(S, width)[:, :t.shape[1]]
        view.copy_(t)
        return buf, view

    for gap, offset in ((0, 1), (5, 3), (8, 8)):
        for place in ("apart", "resid", "mul"):
            bx, vx = spread(x, gap, offset)
            bm, vm = spread(mul, gap, offset)
            bq, vq = spread(resid, gap, offset)
            by, vy = {"apart": spread(torch.zeros_like(plain), gap, offset), "resid": (bq, vq), "mul": (bm, vm)}[place]
            B.coli_dense_linear(ctx, h, vx, vy, act="relu", mul=vm, resid=vq)
            assert torch.equal(vy, plain), (gap, offset, place)
            vy.fill_(7.0)
            assert (by == 7).all()
    assert B.coli_check_error(ctx) == 0
    B.coli_dense_free(ctx, h)


@pytest.mark.parametrize("x_dtype,y", TYPES)
@pytest.mark.parametrize("S,I,O_", [(512, 64, 6144), (512, 2496, 6144), (300, 6144, 2100)])
def test_a_copy_that_never_comes_to_a_pair(S, I, O_, x_dtype, y):
    """Both CTAs give up by themselves, with few products and with many still to come, and the calls after that are healthy."""
    c = Ctx.with_env(COLI_TEST_WAIT_NS=20_000_000, COLI_TEST_WITHHOLD=1)
    try:
        h, x, want = make(c.ctx, S, I, O_, x_dtype)
        out = torch.empty(S, O_, dtype=DT[y], device="cuda")
        B.coli_dense_linear(c.ctx, h, x, out)
        assert B.coli_check_error(c.ctx) == B.COLI_E_TIMEOUT
        for _ in range(2):
            B.coli_dense_linear(c.ctx, h, x, out)
            assert B.coli_check_error(c.ctx) == 0
            close(out, want, I, x_dtype)
    finally:
        c.close()


@pytest.mark.parametrize("x_dtype,y", TYPES)
@pytest.mark.parametrize("S,I,O_", [(512, 1280, 6144), (300, 6144, 2100)])
def test_captures_replay(ctx, S, I, O_, x_dtype, y):
    """Pairs of CTAs, whole and split tiles, in a graph: new activations each replay, the bits of calls outside it."""
    h, x, want = make(ctx, S, I, O_, x_dtype)
    out, stream, before = torch.empty(S, O_, dtype=DT[y], device="cuda"), torch.cuda.Stream(), torch.cuda.current_stream()
    xs = [x.clone(), -x, x.flip(0), x * 2]
    outside = []
    for v in xs:
        B.coli_dense_linear(ctx, h, v, out)
        outside.append(out.clone())
    close(outside[0], want, I, x_dtype)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        B.coli_set_stream(ctx, stream)
        for _ in range(3):
            B.coli_dense_linear(ctx, h, x, out)
    B.coli_set_stream(ctx, before)
    for v, one in zip(xs, outside):
        x.copy_(v)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, one)
    assert B.coli_check_error(ctx) == 0
    B.coli_dense_free(ctx, h)
