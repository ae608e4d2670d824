"""Log probabilities of logits at both ends of binary32, whose difference is beyond it."""
import numpy as np
import pytest
import torch

import oracle.tokens as O
from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import as_dtype

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-30, 1e-3, 0.25, 0.49])
@pytest.mark.parametrize("S,V", [(1, 40), (1, 50021), (700, 300)])
def test_differences_beyond_binary32(S, V, scale, dtype):
    """log p = scale (x - m) - log s: a difference, a product and a sum that round, the scale to binary32: 2^-22 relative."""
    c = Ctx()
    try:
        x, xt = as_dtype(np.linspace(-3.3e38, 3.3e38, V) * np.ones((S, 1)), dtype)
        x[:, V // 2], xt[:, V // 2] = -np.inf, -np.inf
        tokens = torch.tensor([0, 1, V // 3, V // 2, V - 2, V - 1], dtype=torch.int32, device="cuda").expand(S, 6).contiguous()
        out = dict(logp=torch.empty(S, 6, device="cuda"), entropy=torch.empty(S, device="cuda"),
                   top_id=torch.empty(S, 32, dtype=torch.int32, device="cuda"), top_logp=torch.empty(S, 32, device="cuda"))
        B.coli_logprobs(c.ctx, xt, scale=scale, tokens=tokens, **out)
        assert B.coli_check_error(c.ctx) == 0
        lp, entropy = O.logprobs(x[:1], scale)
        for got, at in ((out["logp"], tokens[0].cpu().numpy()), (out["top_logp"], O.top(x[:1], 32)[0])):
            want = lp[0, at]
            got = got.double().cpu().numpy()
            assert np.array_equal(got == -np.inf, np.broadcast_to(want == -np.inf, got.shape))
            fine = want > -np.inf
            assert (np.abs(got[:, fine] - want[fine]) <= 2.0 ** -22 * np.abs(want[fine]) + 2.0 ** -18).all()
        assert (out["top_id"].cpu().numpy() == O.top(x[:1], 32)).all()
        assert (np.abs(out["entropy"].cpu().numpy() - entropy) <= 2.0 ** -18).all()
    finally:
        c.close()
