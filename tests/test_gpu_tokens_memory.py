"""Arrays that share memory: rotary positions, 16-bit products and log probabilities refuse an output in another array, whatever
the strides, and nothing else."""
import numpy as np
import pytest
import torch

from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = Ctx()
    yield c.ctx
    c.close()


def runs(ctx, call):
    try:
        call()
        return True
    except B.ColiError as e:
        assert e.code == B.COLI_E_INVAL and "overlap" in B.coli_last_error(ctx)
        return False


def elements(base, at, stride, row, n):
    """The places in `base` of n rows of `row` elements, `stride` apart, from `at` on, and the view."""
    places = (at + stride * np.arange(n)[:, None] + np.arange(row)[None, :]).ravel()
    return set(places.tolist()), torch.as_strided(base, (n, row), (stride, 1), at)


@pytest.mark.parametrize("seed", range(4))
def test_rows_of_one_buffer(ctx, seed):
    """Residual, bias, logits and outputs anywhere in one buffer, with strides of their own."""
    r = rng("rows", seed)
    base = torch.zeros(4000, device="cuda")
    O, I = 10, 8
    h = B.coli_dense_upload(ctx, torch.zeros(O, I, dtype=torch.bfloat16))
    x = {S: torch.zeros(S, I, device="cuda") for S in (1, 2, 3, 7)}
    both = set()
    for _ in range(300):
        base.zero_()
        S = int(r.choice([1, 2, 3, 7]))
        sy, sr = (int(r.choice([10, 11, 20, 30, 57])) for _ in range(2))
        py, y = elements(base, int(r.integers(0, 300)), sy, O, S)
        pr, resid = elements(base, int(r.integers(0, 300)), sr, O, S)
        pb, bias = elements(base, int(r.integers(0, 300)), O, O, 1)
        same = resid.data_ptr() == y.data_ptr() and (sy == sr or S == 1)
        fine = (same or not py & pr) and not py & pb
        assert runs(ctx, lambda: B.coli_dense_linear(ctx, h, x[S], y, resid=resid, bias=bias[0])) == fine
        both.add(fine)
        # rows of logits, and outputs between them
        pe, entropy = elements(base, int(r.integers(0, 300)), S, S, 1)
        fine = not pe & pr
        assert runs(ctx, lambda: B.coli_logprobs(ctx, resid, entropy=entropy[0])) == fine
    assert both == {True, False}
    B.coli_dense_free(ctx, h)
    assert B.coli_check_error(ctx) == 0


def test_small_arrays(ctx):
    words = torch.zeros(400, dtype=torch.int32, device="cuda")
    floats = words.view(torch.float32)
    freqs = words[200:208].view(torch.int64)
    pos = words[300:304]
    k_in, k_out = torch.zeros(4, 1, 8, device="cuda"), torch.zeros(4, 1, 8, device="cuda")
    start = torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda")

    def rotary(at, **where):
        out = floats[at:at + 32].view(4, 1, 8)
        return runs(ctx, lambda: B.coli_rotary(ctx, k_in, None, freqs, out, None, **where))

    assert rotary(0, positions=pos) and rotary(168, positions=pos) and rotary(208, positions=pos) and rotary(268, positions=pos)
    assert not rotary(169, positions=pos) and not rotary(207, positions=pos)
    assert not rotary(269, positions=pos) and not rotary(303, positions=pos)
    assert rotary(0, lens=pos) and not rotary(303, lens=pos)
    assert rotary(302, lens=pos[:2], q_start=start) and not rotary(301, lens=pos[:2], q_start=start)
    words[320:323] = start
    assert rotary(323, lens=pos[:2], q_start=words[320:323]) and not rotary(322, lens=pos[:2], q_start=words[320:323])
    words.zero_()

    x = torch.zeros(2, 50, device="cuda")

    def logprobs(*at):
        logp, entropy, top_id, top_logp, tokens = (t[i:i + n].view(s) for t, i, n, s in zip(
            (floats, floats, words, floats, words), at, (6, 2, 4, 4, 6), ((2, 3), (2,), (2, 2), (2, 2), (2, 3))))
        return runs(ctx, lambda: B.coli_logprobs(ctx, x, tokens=tokens, logp=logp, entropy=entropy, top_id=top_id, top_logp=top_logp))

    apart = [0, 6, 8, 12, 16]
    assert logprobs(*apart)
    words.zero_()
    for i in range(4):
        for j in range(5):
            if i != j:
                at = [50 * n for n in range(5)]
                at[i] = at[j] + 1
                words.zero_()
                assert not logprobs(*at), (i, j)
    assert B.coli_check_error(ctx) == 0
