"""Rotary positions: tables, positions and plans that do not lie on a boundary of their elements are refused before anything is launched."""
import pytest
import torch

from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx

pytestmark = pytest.mark.gpu


def test_arrays_off_their_alignment_are_refused():
    c = Ctx()
    try:
        T, heads, hd = 4, 2, 32
        x = torch.zeros(T, heads, hd, device="cuda")
        freqs = torch.zeros(hd // 2 + 1, dtype=torch.int64, device="cuda")
        words = {n: torch.zeros(T + 2, dtype=torch.int32, device="cuda") for n in ("positions", "q_start", "lens")}

        def call(freqs_off=0, positions=None, q_start=None, lens=None, B_=0):
            at = {n: None if off is None else words[n].data_ptr() + off for n, off in
                  (("positions", positions), ("q_start", q_start), ("lens", lens))}
            row = heads * hd
            return B.library().coli_rotary(c.ctx, x.data_ptr(), row, x.data_ptr(), row, heads, None, 0, None, 0, 0, B.COLI_DTYPE_F32,
                                           hd, hd, 0, freqs.data_ptr() + freqs_off, 1.0, T, at["positions"], at["q_start"], at["lens"], B_)

        assert call(positions=0) == call(lens=0, B_=T) == call(lens=0, q_start=0, B_=T) == B.COLI_OK
        assert call(freqs_off=8, positions=4) == call(lens=4, q_start=4, B_=T) == B.COLI_OK
        for bad in (dict(freqs_off=1, positions=0), dict(freqs_off=4, positions=0), dict(positions=1), dict(positions=2),
                    dict(lens=1, B_=T), dict(lens=2, B_=T), dict(lens=0, q_start=1, B_=T), dict(lens=0, q_start=3, B_=T),
                    dict(freqs_off=4, lens=0, B_=T)):
            assert call(**bad) == B.COLI_E_INVAL, bad
            assert "aligned" in B.coli_last_error(c.ctx)
        assert B.coli_check_error(c.ctx) == 0
    finally:
        c.close()
