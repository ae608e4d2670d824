"""How close the sums of products with 16-bit weights come for binary32 outputs: in norm, close enough to tell sums in chunks of 256
columns from sums that run over all columns in the tensor core."""
import pytest
import torch

from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import DT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = Ctx()
    yield c.ctx
    c.close()


def lost(steps):
    """In norm, what cutting off takes from a sum of `steps` random terms. A step drops half a unit in the last place on average, 0.36
    2^-23 of what the sum has reached (0.72 the mean of 1 / m over the significands m), always towards zero; what it has reached, summed over
    the steps of a random walk, is sqrt((n + 1)(2 n + 1) / 6) of the end."""
    return 0.36 * 2.0 ** -23 * ((steps + 1) * (2 * steps + 1) / 6) ** 0.5


@pytest.mark.parametrize("x_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("I", [2048, 6144])
@pytest.mark.parametrize("S,O_", [(1, 20000), (5, 4000), (24, 2500), (64, 2000), (301, 2100), (1500, 1100), (4096, 1000)])
def test_sums_are_held_in_chunks(ctx, S, I, O_, x_dtype):
    """A chunk of 256 columns is 16 steps, chunks are added with rounding: at most I / 256 roundings of 2^-24 / sqrt 3 each of what the sum has
    reached, half of it in the mean square. Parts of binary32 activations that share a sum make three steps of one, unless a tile
    has 64 tokens at most and they are summed side by side."""
    g = torch.Generator(device="cuda").manual_seed(S + I)
    W = (0.05 * torch.randn(O_, I, device="cuda", generator=g)).bfloat16()
    x = torch.randn(S, I, device="cuda", generator=g).to(DT[x_dtype])
    y = torch.empty(S, O_, device="cuda")
    h = B.coli_dense_upload(ctx, W)
    B.coli_dense_linear(ctx, h, x, y)
    assert B.coli_check_error(ctx) == 0
    B.coli_dense_free(ctx, h)
    want = x.double() @ W.double().t()
    off = ((y.double() - want).norm() / want.norm()).item()
    times = 3 if x_dtype == "f32" and S > 64 else 1
    added = (I / 256 / 2 / 3) ** 0.5 * 2.0 ** -24
    bound = ((times * lost(16)) ** 2 + added ** 2) ** 0.5
    assert bound < 0.5 * times * lost(I // 16)  # what it would be without chunks
    assert off <= 1.1 * bound, (off, bound)  # a tenth for the sample


@pytest.mark.parametrize("S", [1, 64, 600])
def test_tiny_binary32_activations(ctx, S):
    """W = 1: values from 2^-110 on arrive whole, smaller ones to a multiple of 2^-133, the smallest bfloat16."""
    h = B.coli_dense_upload(ctx, torch.eye(64, dtype=torch.bfloat16))
    g = torch.Generator(device="cuda").manual_seed(S)
    for e in (100, 110, 111, 118, 126, 127, 133, 134, 149):
        x = ((1 + torch.rand(S, 64, dtype=torch.float64, device="cuda", generator=g)) * 2.0 ** -e).float()
        y = torch.empty(S, 64, device="cuda")
        B.coli_dense_linear(ctx, h, x, y)
        off = (y.double() - x.double()).abs()
        assert (off == 0).all() if e <= 110 else (off < 2.0 ** -133).all()
    assert B.coli_check_error(ctx) == 0
    B.coli_dense_free(ctx, h)
