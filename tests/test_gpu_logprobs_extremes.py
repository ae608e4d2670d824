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


@pytest.mark.parametrize("S,V", [(1, 5000), (700, 5000), (2, 70001)])
def test_close_to_certain(S, V):
    """One entry takes all but 1e-3 to 1e-12 of a row. Its log p is never above 0; its error and the entropy's are those of at most V / 512 +
    64 roundings of s = 1 + ... and of the logarithm: absolute ones."""
    c = Ctx()
    try:
        for tail in (1e-3, 1e-5, 1e-7, 1e-9, 1e-12):
            x = np.full((S, V), np.log(tail / (V - 1)), np.float32)
            x += 0.1 * np.random.default_rng(7).normal(size=V).astype(np.float32)
            at = np.arange(S) * 7919 % V
            x[np.arange(S), at] = 3.0
            xt = torch.from_numpy(x).cuda()
            tokens = torch.from_numpy(at.astype(np.int32)).cuda()[:, None].contiguous()
            logp, entropy = torch.empty(S, 1, device="cuda"), torch.empty(S, device="cuda")
            B.coli_logprobs(c.ctx, xt, tokens=tokens, logp=logp, entropy=entropy)
            assert B.coli_check_error(c.ctx) == 0
            lp, h = O.logprobs(x)
            got = logp.double().cpu().numpy()[:, 0]
            tol = (V / 512 + 64) * 2.0 ** -24 + 2.0 ** -22
            assert (got <= 0).all() and (np.abs(got - lp[np.arange(S), at]) <= tol).all()
            got = entropy.double().cpu().numpy()
            assert (got >= 0).all() and (np.abs(got - h) <= tol + 2.0 ** -20 * h).all()
    finally:
        c.close()


@pytest.mark.parametrize("S", [1, 700])
def test_log_p_is_never_above_0(S):
    """Logits so large that the next one above is 8 to 32 further: what precedes the largest entry carries almost nothing, and what is left is 1."""
    c = Ctx()
    try:
        for first in (1e8, 1.5e8, 2.5e8, 5e8, 3e9):
            for step in (8, 16, 24, 32, 64):
                x = np.zeros((S, 5000), np.float32)
                x[:, 0], x[:, 1024] = first, np.float32(first) + np.float32(step)
                xt = torch.from_numpy(x).cuda()
                logp, entropy = torch.empty(S, 1, device="cuda"), torch.empty(S, device="cuda")
                B.coli_logprobs(c.ctx, xt, tokens=torch.full((S, 1), 1024, dtype=torch.int32, device="cuda"), logp=logp, entropy=entropy)
                assert B.coli_check_error(c.ctx) == 0
                lp, h = O.logprobs(x[:1])
                assert (logp <= 0).all() and (np.abs(logp.double().cpu().numpy() - lp[0, 1024]) <= 2.0 ** -20).all()
                # t adds up terms of up to 2^5 powers of two that round to 2^-24 each
                assert (entropy >= 0).all() and (np.abs(entropy.double().cpu().numpy() - h) <= 2.0 ** -17).all()
    finally:
        c.close()
