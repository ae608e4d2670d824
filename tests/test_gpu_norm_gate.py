"""The norm's sigmoid gate over the whole range of its argument."""
import numpy as np
import pytest
import torch

import oracle.kv4 as O
from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import as_dtype, rng

pytestmark = pytest.mark.gpu


def test_an_f32_gate_is_exact_to_a_few_units_in_the_last_place():
    """h = alpha * sigmoid(gate) * block alone: an exponential (2 units), a sum, a quotient and three products (half a unit
    each) stay within 5 units of 2^-24 relative to the result twice over; below the normal numbers, two of 2^-149."""
    S, D = 5, 1003
    r = rng("gate", S, D)
    gate, gate_t = as_dtype(r.uniform(-105, 30, size=(S, D)), "f32")
    gate[0, :6] = [0, -0.0, 88.8, -88.8, 104, -104]
    gate_t.copy_(torch.from_numpy(gate))
    block, block_t = as_dtype(np.sign(r.normal(size=(S, D))) * r.uniform(0.5, 1, size=(S, D)), "f32")
    c = Ctx()
    try:
        h = torch.empty(S, D, device="cuda")
        B.coli_norm_residual(c.ctx, block_t, None, gate_t, 0.75, None, None, 0.0, h, None, gate_sigmoid=True)
        assert B.coli_check_error(c.ctx) == 0
        ref, _ = O.norm_residual(block, None, gate, 0.75, None, None, 0.0, gate_sigmoid=True)
        off = np.abs(h.cpu().numpy().astype(np.float64) - ref) - (10 * 2.0 ** -24 * np.abs(ref) + 2 * 2.0 ** -149)
        assert (off <= 0).all(), (int((off > 0).sum()), float((off / np.abs(ref)).max()))
    finally:
        c.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_at_the_ends(dtype):
    """sigmoid(+-infinity) is 1 and 0; a gate that is not a number shows and is reported."""
    c = Ctx()
    try:
        _, block = as_dtype(np.linspace(1, 2, 64)[None].repeat(3, 0), dtype)
        _, gate = as_dtype(np.array([[np.inf], [-np.inf], [1.0]]).repeat(64, 1), dtype)
        h = torch.empty_like(block)
        B.coli_norm_residual(c.ctx, block, None, gate, 1.0, None, None, 0.0, h, None, gate_sigmoid=True)
        assert B.coli_check_error(c.ctx) == 0
        assert torch.equal(h[0], block[0]) and bool((h[1] == 0).all())
        gate[2, 5] = float("nan")
        B.coli_norm_residual(c.ctx, block, None, gate, 1.0, None, None, 0.0, h, None, gate_sigmoid=True)
        assert B.coli_check_error(c.ctx) == B.COLI_E_NONFINITE
        assert h.isnan().nonzero().tolist() == [[2, 5]]
    finally:
        c.close()
