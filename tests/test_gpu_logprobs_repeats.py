"""Alternatives of thousands of calls: every one has the same ids and bits, with all SMs busy and rows split or whole."""
import numpy as np
import pytest
import torch

import oracle.tokens as O
from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import as_dtype, rng

pytestmark = pytest.mark.gpu


# One row in many parts, a few rows in some, a row for each CTA with four CTAs on an SM, and rows of few keys beside rows of many.
@pytest.mark.parametrize("S,V,dtype", [(1, 50021, "f32"), (15, 32003, "f32"), (64, 20011, "bf16"), (608, 1500, "f32"), (1300, 700, "bf16")])
@pytest.mark.parametrize("k", [2, 5, 32])
def test_every_call_gives_the_same_alternatives(S, V, dtype, k):
    c = Ctx()
    try:
        x, xt = as_dtype(3 * rng("repeats", S, V).normal(size=(S, V)), dtype)
        if S > 1:
            x[1, k + 9:] = -np.inf  # not many entries more than are asked for
            xt[1, k + 9:] = -np.inf
        ids, logp = torch.empty(S, k, dtype=torch.int32, device="cuda"), torch.empty(S, k, device="cuda")
        B.coli_logprobs(c.ctx, xt, top_id=ids, top_logp=logp)
        want = torch.from_numpy(O.top(x, k).astype(np.int32)).cuda()
        first, off = logp.clone(), torch.zeros((), dtype=torch.int64, device="cuda")
        for _ in range(2000):
            ids.fill_(-7)
            B.coli_logprobs(c.ctx, xt, top_id=ids, top_logp=logp)
            off += (ids != want).sum() + (logp != first).sum()
        assert off.item() == 0
        assert B.coli_check_error(c.ctx) == 0
    finally:
        c.close()
