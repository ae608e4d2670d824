"""Attention over the 4-bit cache where numbers or places are at an end of their range: values of any size, what is not
finite and who sees it, windows of any size, pages that a window has left behind."""
import numpy as np
import pytest
import torch

import oracle.kv4 as O
from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import Batch, assert_within, bound

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
