"""Log probabilities, entropies and alternatives against the 64-bit oracle."""
import numpy as np
import pytest
import torch

import oracle.tokens as O
from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import DT, as_dtype, rng

pytestmark = pytest.mark.gpu

NEG = -np.inf


@pytest.fixture(scope="module")
def ctx():
    c = Ctx()
    yield c.ctx
    c.close()


def call(ctx, xt, tokens=None, k=0, scale=1.0, entropy=True, code=0):
    S = xt.shape[0]
    out = dict(logp=None if tokens is None else torch.full(tokens.shape, 7.0, device="cuda"),
               entropy=torch.full((S,), 7.0, device="cuda") if entropy else None,
               top_id=torch.full((S, k), 77, dtype=torch.int32, device="cuda") if k else None,
               top_logp=torch.full((S, k), 7.0, device="cuda") if k else None)
    B.coli_logprobs(ctx, xt, scale=scale, tokens=tokens, **out)
    assert B.coli_check_error(ctx) == code
    return {n: None if t is None else t.cpu().numpy() for n, t in out.items()}


def close(got, want, size, V):
    """log p = scale (x - m) - log s: a difference and a product of 2^-24 relative to |scale (x - m)|, the logarithm to 2^-23 of
    at most 17, s itself to 2^-21 (exponentials) and (V / 512 + 64) 2^-24 (sums)."""
    tol = 2.0 ** -22 * size + 2.0 ** -18 + (V / 512 + 64) * 2.0 ** -24
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True)
    off = np.abs(got[fine] - want[fine]) - np.broadcast_to(tol, got.shape)[fine]
    assert off.size == 0 or off.max() <= 0, float(off.max())


def check(ctx, x, xt, k=5, n=2, scale=1.0):
    S, V = x.shape
    tokens = rng("tokens", S, V).integers(0, V, size=(S, n)).astype(np.int32)
    got = call(ctx, xt, torch.from_numpy(tokens).cuda(), k, scale)
    lp, h = O.logprobs(x, scale)
    with np.errstate(all="ignore"):
        size = np.where(np.isfinite(x), scale * (x.max(-1, keepdims=True) - x), 0)
    close(got["logp"], np.take_along_axis(lp, tokens, 1), np.take_along_axis(size, tokens, 1), V)
    # entropy = log s - t / s: t's terms, y 2^y, add up to at most the entropy (in sum with log s), each to 2^-21
    assert (np.abs(got["entropy"] - h) <= 2.0 ** -18 + (h + 17) * (2.0 ** -20 + (V / 512 + 64) * 2.0 ** -24)).all()
    if k:
        ids = O.top(x, k)
        assert np.array_equal(got["top_id"], ids)
        at = np.maximum(ids, 0)
        close(got["top_logp"], np.where(ids < 0, NEG, np.take_along_axis(lp, at, 1)), np.take_along_axis(size, at, 1), V)
    return got


def logits(S, V, dtype, spread=3.0, seed=0):
    return as_dtype(spread * rng("logits", S, V, seed).normal(size=(S, V)), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,V", [(1, 1), (3, 2), (1, 31), (2, 32), (5, 511), (1, 4096), (3, 4097), (2, 20011), (1, 70001), (160, 5003),
                                 (310, 1003), (700, 100)])
def test_sizes(ctx, S, V, dtype):
    x, xt = logits(S, V, dtype)
    check(ctx, x, xt, k=min(V, 20) if S < 100 else 3, scale=0.8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", [0, 1, 2, 16, 17, 31, 32])
@pytest.mark.parametrize("S", [2, 40])
def test_numbers_of_alternatives(ctx, S, k, dtype):
    x, xt = logits(S, 12345, dtype)
    check(ctx, x, xt, k=k, n=3)


def test_fewer_entries_than_alternatives(ctx):
    x, xt = logits(4, 9, "f32")
    x[1, 3:] = NEG
    x[2] = NEG
    x[3, 1:] = NEG
    check(ctx, x, torch.from_numpy(x).cuda(), k=32)


@pytest.mark.parametrize("V", [700, 50000, 300000])
@pytest.mark.parametrize("kind", ["all alike", "few values", "ascending", "descending", "peak last", "lowest", "zeros", "many tops"])
@pytest.mark.parametrize("S", [1, 400])
def test_ties_and_orders(ctx, S, kind, V):
    """Rows whose largest entries tie, by the thousand, or stand where one thread or one CTA finds them all."""
    if S * V > 30_000_000:
        S = 30_000_000 // V
    if kind == "all alike":
        row = np.full(V, -3.25)
    elif kind == "few values":
        row = rng("few", V).integers(0, 3, size=V).astype(float)
    elif kind == "ascending":
        row = np.arange(V) / 256
    elif kind == "descending":
        row = -np.arange(V) / 256
    elif kind == "peak last":
        row = np.zeros(V)
        row[-1] = 50
    elif kind == "lowest":
        row = np.full(V, float(np.finfo(np.float32).min))
        row[V // 2] = NEG
    elif kind == "zeros":
        row = np.where(rng("zeros", V).random(V) < 0.5, 0.0, -0.0)
        row[:5] = -1
    else:  # thousands that reach any bound
        row = np.where(rng("tops", V).random(V) < 0.2, 9.0, rng("tops", V, 1).normal(size=V))
    row = row.astype(np.float32)
    xt = torch.from_numpy(row).cuda().expand(S, V).contiguous()
    one = check(ctx, row[None], xt[:1], k=32)
    got = call(ctx, xt, torch.zeros(S, 1, dtype=torch.int32, device="cuda"), 32)
    assert (got["top_id"] == one["top_id"]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset,gap", [(0, 0), (1, 0), (3, 5), (0, 8), (7, 1)])
def test_strides_and_alignments(ctx, dtype, offset, gap):
    for S, V in ((3, 3001), (200, 515)):
        x, xt = logits(S, V, dtype)
        buf = torch.full((S * (V + gap) + 16,), float("nan"), dtype=DT[dtype], device="cuda")
        view = buf[offset:offset + S * (V + gap)].view(S, V + gap)[:, :V]
        view.copy_(xt)
        check(ctx, x, view, k=7)


def test_what_is_not_a_number_stays_in_its_row(ctx):
    for S, V in ((3, 40000), (200, 300)):
        for bad in (np.nan, np.inf):
            x, _ = logits(S, V, "f32")
            x[1, V // 3] = bad
            tokens = torch.zeros(S, 2, dtype=torch.int32, device="cuda")
            got = call(ctx, torch.from_numpy(x).cuda(), tokens, 4, code=B.COLI_E_NONFINITE)
            assert np.isnan(got["logp"][1]).all() and np.isnan(got["entropy"][1]) and np.isnan(got["top_logp"][1]).all()
            assert (got["top_id"][1] == -1).all()
            x[1] = 0
            lp, _ = O.logprobs(x)
            rest = [r for r in range(S) if r != 1]
            assert np.allclose(got["logp"][rest, 0], lp[rest, 0], atol=2e-5)
            assert np.array_equal(got["top_id"][rest], O.top(x, 4)[rest])


def test_tokens_that_are_none_or_too_large(ctx):
    x, xt = logits(3, 100, "f32")
    tokens = torch.tensor([[0, -1, 99], [-100, 5, 5], [-2 ** 31, 1, 2]], dtype=torch.int32, device="cuda")
    got = call(ctx, xt, tokens)
    lp, _ = O.logprobs(x)
    assert (got["logp"][[0, 1, 2], [1, 0, 0]] == 0).all()
    assert np.allclose(got["logp"][1, 1:], lp[1, 5], atol=1e-5)
    tokens[1, 1] = 100
    got = call(ctx, xt, tokens, code=B.COLI_E_RANGE)
    assert np.isnan(got["logp"][1, 1]) and np.isclose(got["logp"][1, 2], lp[1, 5], atol=1e-5)


def test_forbidden_tokens_and_huge_entries(ctx):
    x, _ = logits(5, 5000, "f32")
    x[0, ::2] = NEG
    x[1] = NEG
    x[1, 4321] = -2.5
    x[2] *= 1e30
    x[3] = np.finfo(np.float32).min
    x[3, 17] = np.finfo(np.float32).max / 4
    x[4] = NEG
    got = check(ctx, x[:2], torch.from_numpy(x[:2]).cuda(), k=6)
    assert got["top_id"][1].tolist() == [4321] + [-1] * 5
    got = call(ctx, torch.from_numpy(x).cuda(), torch.full((5, 1), 17, dtype=torch.int32, device="cuda"), 3)
    assert got["top_logp"][2, 0] == 0 and got["entropy"][2] == 0
    assert got["logp"][3, 0] == 0 and got["top_id"][3, 0] == 17
    assert got["logp"][4, 0] == NEG and got["entropy"][4] == 0 and (got["top_id"][4] == -1).all()


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 50.0, 1e30])
@pytest.mark.parametrize("S", [2, 200])
def test_scales(ctx, S, scale):
    """Inverse temperatures from almost even to almost certain: log p of the largest entry keeps an absolute error of 2^-20."""
    x, xt = logits(S, 3000, "f32")
    lp, h = O.logprobs(x, scale)
    got = call(ctx, xt, torch.zeros(S, 1, dtype=torch.int32, device="cuda"), 3, scale=scale)
    ids = O.top(x, 3)
    want = np.take_along_axis(lp, ids, 1)
    assert np.array_equal(got["top_id"], ids)
    assert (np.abs(got["top_logp"] - want) <= 2.0 ** -18 + 2.0 ** -21 * np.abs(want)).all()
    assert (np.abs(got["entropy"] - h) <= 1e-4).all()


def test_entries_far_above_those_before_them(ctx):
    """Steps up of many powers of two between one vector and the next, in every thread and CTA."""
    for S in (1, 300):
        x = np.zeros((S, 40000), np.float32)
        x += (np.arange(40000) // 2500 * 25).astype(np.float32)
        x += rng("steps", S).normal(size=x.shape).astype(np.float32)
        check(ctx, x, torch.from_numpy(x).cuda(), k=9)
        check(ctx, x[:, ::-1].copy(), torch.from_numpy(x[:, ::-1].copy()).cuda(), k=9)


def test_each_output_alone(ctx):
    x, xt = logits(2, 3000, "f32")
    tokens = torch.tensor([[5], [6]], dtype=torch.int32, device="cuda")
    every = call(ctx, xt, tokens, 4)
    assert np.array_equal(call(ctx, xt, tokens, 0, entropy=False)["logp"], every["logp"])
    assert np.array_equal(call(ctx, xt, None, 0)["entropy"], every["entropy"])
    alone = call(ctx, xt, None, 4, entropy=False)
    assert np.array_equal(alone["top_id"], every["top_id"]) and np.array_equal(alone["top_logp"], every["top_logp"])
    flat = torch.empty(2, device="cuda")
    B.coli_logprobs(ctx, xt, tokens=tokens[:, 0].contiguous(), logp=flat)
    assert np.array_equal(flat.cpu().numpy(), every["logp"][:, 0])


def test_runs_give_the_same_bits_and_captures_replay(ctx):
    x, xt = logits(3, 60001, "bf16")
    tokens = torch.tensor([[5], [6], [7]], dtype=torch.int32, device="cuda")
    first = call(ctx, xt, tokens, 20)
    for _ in range(5):
        again = call(ctx, xt, tokens, 20)
        for n in first:
            assert np.array_equal(first[n], again[n])
    out = dict(logp=torch.empty(3, 1, device="cuda"), entropy=torch.empty(3, device="cuda"),
               top_id=torch.empty(3, 20, dtype=torch.int32, device="cuda"), top_logp=torch.empty(3, 20, device="cuda"))
    stream, before, graph = torch.cuda.Stream(), torch.cuda.current_stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        B.coli_set_stream(ctx, stream)
        B.coli_logprobs(ctx, xt, tokens=tokens, **out)
        B.coli_logprobs(ctx, xt, tokens=tokens, **out)
    B.coli_set_stream(ctx, before)
    for _ in range(3):
        for t in out.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n, t in out.items():
            assert np.array_equal(first[n], t.cpu().numpy())
    assert B.coli_check_error(ctx) == 0


def test_refusals(ctx):
    x = torch.zeros(2, 100, device="cuda")
    t, lp, h = torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.zeros(2, 1, device="cuda"), torch.zeros(2, device="cuda")
    ids, tl = torch.zeros(2, 33, dtype=torch.int32, device="cuda"), torch.zeros(2, 33, device="cuda")
    for args, kw in (((x,), {}), ((x,), dict(tokens=t)), ((x,), dict(logp=lp)), ((x,), dict(top_id=ids[:, :3].contiguous())),
                     ((x,), dict(top_id=ids, top_logp=tl)), ((x.half(),), dict(entropy=h)), ((x.cpu(),), dict(entropy=h)),
                     ((x,), dict(entropy=h, scale=0.0)), ((x,), dict(entropy=h, scale=-1.0)), ((x,), dict(entropy=h, scale=float("nan"))),
                     ((x,), dict(entropy=h, scale=float("inf"))), ((x,), dict(tokens=t.long(), logp=lp)),
                     ((x,), dict(tokens=t, logp=lp.double())), ((x,), dict(entropy=h[:1])), ((x[0],), dict(entropy=h)),
                     ((x.t(),), dict(entropy=torch.zeros(100, device="cuda"))), ((x[:1].expand(2, 100),), dict(entropy=h)),
                     ((x[:0],), dict(entropy=h[:0]))):
        with pytest.raises((B.ColiError, ValueError)):
            B.coli_logprobs(ctx, *args, **kw)
    assert B.coli_check_error(ctx) == 0
