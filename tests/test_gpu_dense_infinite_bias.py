"""An infinite bias is no error of the sums: what the activations make of it, as 64-bit arithmetic has it."""
import numpy as np
import pytest
import torch

import oracle.tokens as O
from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import DT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x_dtype,y", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("kind", list(B.ACTIVATIONS))
@pytest.mark.parametrize("S", [1, 20, 600])
def test_infinite_bias(S, kind, x_dtype, y):
    c = Ctx()
    try:
        O_ = 700
        bias = np.zeros(O_, np.float32)
        bias[0::7], bias[1::7], bias[2::7], bias[3::7], bias[4::7] = np.inf, 1e30, -np.inf, -1e30, np.nan
        h = B.coli_dense_upload(c.ctx, torch.ones(O_, 64, dtype=torch.bfloat16))
        x = torch.full((S, 64), 1 / 64, dtype=DT[x_dtype], device="cuda")  # every sum is 1 exactly
        out = torch.empty(S, O_, dtype=DT[y], device="cuda")
        B.coli_dense_linear(c.ctx, h, x, out, bias=torch.from_numpy(bias).cuda(), act=kind)
        assert B.coli_check_error(c.ctx) == 0
        with np.errstate(all="ignore"):
            want = O.act((bias + np.float32(1)).astype(np.float64), kind)
        got = out.double().cpu().numpy()
        assert (got == got[:1]).all() or np.array_equal(got, np.broadcast_to(got[:1], got.shape), equal_nan=True)
        # up to one rounding, and the activations' 2^-20; the squares of 1e30 are beyond either type
        inside = np.abs(want) < 3e38
        assert np.array_equal(got[0][~inside & ~np.isnan(want)] > 0, want[~inside & ~np.isnan(want)] > 0)
        assert np.isinf(got[0][~inside & ~np.isnan(want)]).all() and np.array_equal(np.isnan(got[0]), np.isnan(want))
        last = 2.0 ** -8 if y == "bf16" else 2.0 ** -24
        assert (np.abs(got[0][inside] - want[inside]) <= (last + 2.0 ** -20) * np.abs(want[inside]) + 1e-37).all()
    finally:
        c.close()
