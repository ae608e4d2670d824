"""Rotary positions, 16-bit products and log probabilities at the sizes that the header allows, and where offsets pass 32 bits. What is
compared with 64-bit arithmetic is a sample of the rows, the first and the last among them."""
import numpy as np
import pytest
import torch

import oracle.tokens as O
from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import DT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = Ctx()
    yield c.ctx
    c.close()
    torch.cuda.empty_cache()


def turned(ctx, x, freqs, positions, rows):
    """The sampled rows turned by 64-bit arithmetic, and the tolerance: sines and products below 2^-20 of |a| + |b|, one rounding."""
    xs = x[rows].double().cpu().numpy()
    want = O.rotary(xs, freqs.cpu().numpy(), positions[rows].cpu().numpy())
    half = freqs.numel()
    size = np.zeros_like(xs)
    size[:, :, :half] = size[:, :, half:2 * half] = np.abs(xs[:, :, :half]) + np.abs(xs[:, :, half:2 * half])
    return want, size * 2.0 ** -20 + (2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24) * np.abs(want)


@pytest.mark.parametrize("T,heads,hd,rot,dtype", [(16777216, 1, 2, 2, "bf16"), (16777216, 1, 16, 16, "bf16"), (16777213, 1, 6, 4, "f32"),
                                                  (300001, 72, 128, 128, "bf16"), (500003, 40, 80, 38, "bf16"), (300001, 40, 96, 36, "f32")])
def test_rotary(ctx, T, heads, hd, rot, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, heads, hd, dtype=DT[dtype], device="cuda", generator=g)
    positions = torch.randint(-2 ** 31, 2 ** 31, (T,), device="cuda", generator=g).to(torch.int32)
    freqs = B.coli_rotary_freqs(rot, 10000.0)
    rows = torch.tensor([0, 1, 15, 16, T // 3, T // 2, T - 17, T - 2, T - 1], device="cuda")
    want, tol = turned(ctx, x, freqs, positions, rows)
    few = torch.empty(4099, heads, hd, dtype=x.dtype, device="cuda")  # the last rows by themselves
    B.coli_rotary(ctx, x[T - 4099:], None, freqs, few, None, positions=positions[T - 4099:].contiguous())
    B.coli_rotary(ctx, x, None, freqs, x, None, positions=positions)
    assert B.coli_check_error(ctx) == 0
    assert (np.abs(x[rows].double().cpu().numpy() - want) <= tol).all()
    assert torch.equal(x[T - 4099:], few)


def test_rotary_of_the_most_sequences(ctx):
    """65536 sequences of no, one, two or three rows."""
    r = np.random.default_rng(3)
    new = r.integers(0, 4, size=65536)
    start = np.concatenate(([0], np.cumsum(new)))
    lens = new + r.integers(0, 10 ** 6, size=65536)
    T = int(start[-1])
    positions = torch.from_numpy((np.repeat(lens - start[1:], new) + np.arange(T)).astype(np.int32)).cuda()
    x = torch.randn(T, 2, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    freqs, a, b = B.coli_rotary_freqs(64), torch.empty_like(x), torch.empty_like(x)
    B.coli_rotary(ctx, x, None, freqs, a, None, lens=torch.from_numpy(lens.astype(np.int32)).cuda(),
                  q_start=torch.from_numpy(start.astype(np.int32)).cuda())
    B.coli_rotary(ctx, x, None, freqs, b, None, positions=positions)
    assert B.coli_check_error(ctx) == 0
    assert torch.equal(a, b)


@pytest.mark.parametrize("x_dtype,y", [("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("S,I,O_", [(1, 64, 1048576), (1, 520, 1048575), (40, 70, 1048576), (1100, 200, 1048573), (65536, 72, 130), (65535, 1000, 1),
                                    (65536, 136, 9000)])
def test_products(ctx, S, I, O_, x_dtype, y):
    g = torch.Generator(device="cuda").manual_seed(S + O_)
    W = torch.randn(O_, I, dtype=torch.bfloat16, device="cuda", generator=g)
    x = torch.randn(S, I, device="cuda", generator=g).to(DT[x_dtype])
    out = torch.full((S + 1, O_), 7.0, dtype=DT[y], device="cuda")
    h = B.coli_dense_upload(ctx, W)
    B.coli_dense_linear(ctx, h, x, out[:S], act="relu")
    assert B.coli_check_error(ctx) == 0
    B.coli_dense_free(ctx, h)
    assert (out[S] == 7).all()
    pick = lambda n: torch.unique(torch.linspace(0, n - 1, 997, device="cuda").long())
    for rows, cols in ((pick(S), slice(None)) if O_ < 1000 else (pick(S), pick(O_)), (slice(max(0, S - 3), S), slice(None)), (slice(0, 2), slice(None))):
        ws, xs = W[cols].double(), x[rows].double()
        want, size = torch.relu(xs @ ws.t()), xs.abs() @ ws.abs().t()
        got = out[:S][rows][:, cols].double()
        # I / 16 + 64 steps, three times as many for three parts, each cut off to 2^-23 of what it has reached; two parts hold 16 bits
        steps = I / 16 * (3 if x_dtype == "f32" else 1) + 64
        tol = size * (steps * 2.0 ** -23 + (2.0 ** -15 if (x_dtype, y) == ("f32", "bf16") else 0))
        assert ((got - want).abs() <= tol + want * (2.0 ** -8 if y == "bf16" else 2.0 ** -23)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,V,gap", [(1, 16777216, 0), (3, 16777215, 3), (60001, 50001, 0), (65536, 7, 1)])
def test_log_probabilities(ctx, S, V, gap, dtype):
    if dtype == "f32" and S * V > 2 ** 31:
        S //= 2  # offsets pass 32 bits all the same
    g = torch.Generator(device="cuda").manual_seed(V)
    buf = torch.empty(S, V + gap, dtype=DT[dtype], device="cuda").normal_(generator=g).mul_(3)
    x = buf[:, :V]
    k = 32
    tokens = torch.randint(0, V, (S, 2), device="cuda", generator=g, dtype=torch.int32)
    tokens[:, 1] = V - 1
    out = dict(logp=torch.empty(S, 2, device="cuda"), entropy=torch.empty(S, device="cuda"),
               top_id=torch.empty(S, k, dtype=torch.int32, device="cuda"), top_logp=torch.empty(S, k, device="cuda"))
    B.coli_logprobs(ctx, x, tokens=tokens, **out)
    assert B.coli_check_error(ctx) == 0
    for r in sorted({0, S // 2, max(0, S - 2), S - 1}):
        row = x[r].double()
        lp = torch.log_softmax(row, 0)
        near = torch.nonzero(row >= torch.topk(row, min(k, V)).values[-1]).flatten()
        order = sorted(near.tolist(), key=lambda i: (-float(row[i]), i))[:k]
        assert out["top_id"][r].tolist() == order + [-1] * (k - len(order))
        # differences, products and logarithms to 2^-18 in all, and at most V / 512 + 64 roundings of the sum
        tol = 2.0 ** -18 + (V / 512 + 64) * 2.0 ** -24
        assert ((out["logp"][r].double() - lp[tokens[r].long()]).abs() <= tol + 2.0 ** -22 * 50).all()
        assert ((out["top_logp"][r][:len(order)].double() - lp[order]).abs() <= tol).all()
        h = float(torch.special.entr(lp.exp()).sum())
        assert abs(float(out["entropy"][r]) - h) <= 2.0 ** -18 + (h + 17) * (2.0 ** -20 + (V / 512 + 64) * 2.0 ** -24)


def test_as_many_given_tokens_as_entries(ctx):
    V = n = 1 << 20
    x = torch.randn(2, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    tokens = torch.arange(n, dtype=torch.int32, device="cuda").repeat(2, 1)
    logp = torch.empty(2, n, device="cuda")
    B.coli_logprobs(ctx, x, tokens=tokens, logp=logp)
    assert B.coli_check_error(ctx) == 0
    assert ((logp.double() - torch.log_softmax(x.double(), 1)).abs() <= 2.0 ** -18 + (V / 512 + 64) * 2.0 ** -24).all()
