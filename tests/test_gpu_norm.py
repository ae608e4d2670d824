"""The fused norms against the 64-bit oracle: every combination of parts, sizes, alignments, refusals."""
import itertools

import numpy as np
import pytest
import torch

import oracle.kv4 as O
from int4_grouped_expert_router_gb300 import binding as B
from gpu_util import Ctx
from kv4_util import DT, as_dtype, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = Ctx()
    yield c.ctx
    c.close()


def make(S, D, dtype, gate="row", post=True, pre=True, resid=True, block=True, size=1.0, offset=0):
    r = rng("norm", S, D)
    a = {}
    for name, on, shape in (("block", block, (S, D)), ("resid", resid, (S, D)),
                            ("gate", gate, (D,) if gate == "channel" else (S, D))):
        a[name], t = as_dtype(size * r.normal(size=shape) if name != "gate" else r.normal(size=shape), dtype) if on else (None, None)
        if t is not None and offset:
            t = torch.cat([torch.zeros(offset, dtype=t.dtype, device="cuda"), t.flatten()])[offset:].view(t.shape)
        a[name + "_t"] = t
    for name, on in (("w_post", post), ("w_pre", pre)):
        a[name], a[name + "_t"] = as_dtype(1 + 0.2 * r.normal(size=D), "f32") if on else (None, None)
    return a


def run(ctx, a, S, D, dtype, alpha=0.7, eps=1e-5, sigmoid=False, store_h=True):
    h = torch.full((S, D), 3.0, dtype=DT[dtype], device="cuda") if store_h else None
    x = torch.full((S, D), 3.0, dtype=DT[dtype], device="cuda") if a["w_pre"] is not None else None
    B.coli_norm_residual(ctx, a["block_t"], a["resid_t"], a["gate_t"], alpha, a["w_post_t"], a["w_pre_t"], eps, h, x,
                         gate_sigmoid=sigmoid)
    assert B.coli_check_error(ctx) == 0
    ref = O.norm_residual(a["block"], a["resid"], a["gate"], alpha, a["w_post"], a["w_pre"], eps, sigmoid)
    # h: a handful of binary32 roundings (2^-24 each) of terms no larger than |resid| + |alpha g b|; x: those, carried
    # through the norm's factor, and its own. Mean squares of D terms are good to 2^-20. Then one rounding to the dtype.
    h_ref, x_ref = ref
    base = np.abs(h_ref) if a["resid"] is None else np.abs(a["resid"]) + np.abs(h_ref - a["resid"])
    last = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -22
    for got, want, tol in ((h, h_ref, base * 2.0 ** -19 + last * np.abs(h_ref)),
                           (x, x_ref, None if x_ref is None else
                            base * 2.0 ** -18 * np.abs(a["w_pre"]) / np.sqrt((h_ref ** 2).mean(-1, keepdims=True) + eps)
                            + last * np.abs(x_ref))):
        if got is not None:
            off = np.abs(got.float().cpu().numpy() - want) - tol
            assert (off <= 0).all(), (S, D, dtype, float(off.max()))
    return h, x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,D", [(1, 1), (1, 6144), (3, 7), (2, 64), (5, 1000), (17, 1111), (4, 8192), (1, 32768), (2, 32767),
                                 (3, 16384), (300, 160), (2, 12345), (700, 2048)])
def test_sizes(ctx, S, D, dtype):
    run(ctx, make(S, D, dtype), S, D, dtype, sigmoid=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate,post,pre,resid", list(itertools.product((None, "row", "channel"), (True, False), (True, False),
                                                                       (True, False))))
def test_parts(ctx, gate, post, pre, resid, dtype):
    a = make(6, 520, dtype, gate=gate, post=post, pre=pre, resid=resid)
    run(ctx, a, 6, 520, dtype)
    run(ctx, a, 6, 520, dtype, sigmoid=True, alpha=-1.5)
    if pre:
        run(ctx, a, 6, 520, dtype, store_h=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_norm_before_a_first_block(ctx, dtype):
    a = make(5, 6144, dtype, gate=None, post=False, block=False)
    h, _ = run(ctx, a, 5, 6144, dtype)
    assert torch.equal(h, a["resid_t"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [1, 2, 4])
def test_rows_off_a_vector_boundary(ctx, offset, dtype):
    run(ctx, make(9, 512, dtype, offset=offset), 9, 512, dtype)


@pytest.mark.parametrize("size", [0.0, 1e-12, 1e-3, 1e4, 1e15])
def test_sizes_of_the_values(ctx, size):
    run(ctx, make(3, 768, "f32", size=size), 3, 768, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,D", [(1, 6144), (40, 1111), (600, 640)])
def test_in_place(ctx, S, D, dtype):
    a = make(S, D, dtype)
    h, x = run(ctx, a, S, D, dtype)
    r, b = a["resid_t"].clone(), a["block_t"].clone()
    B.coli_norm_residual(ctx, b, r, a["gate_t"], 0.7, a["w_post_t"], a["w_pre_t"], 1e-5, r, b)
    assert torch.equal(r, h) and torch.equal(b, x) and B.coli_check_error(ctx) == 0


def test_values_that_are_not_finite(ctx):
    for where in ("block_t", "resid_t"):
        a = make(4, 300, "f32", gate=None)
        a[where][2, 17] = float("inf")
        h, x = torch.empty(4, 300, device="cuda"), torch.empty(4, 300, device="cuda")
        B.coli_norm_residual(ctx, a["block_t"], a["resid_t"], None, 1.0, a["w_post_t"], a["w_pre_t"], 1e-5, h, x)
        assert B.coli_check_error(ctx) == B.COLI_E_NONFINITE
        assert bool(x[[0, 1, 3]].isfinite().all()) and not bool(x[2].isfinite().all())


def test_refusals(ctx):
    a = make(4, 64, "f32")
    h, x = torch.empty(4, 64, device="cuda"), torch.empty(4, 64, device="cuda")
    base = dict(block=a["block_t"], resid=a["resid_t"], gate=a["gate_t"], alpha=1.0, w_post=a["w_post_t"],
                w_pre=a["w_pre_t"], eps=1e-5, h=h, x=x)
    ok = lambda **k: B.coli_norm_residual(ctx, **{**base, **k})  # noqa: E731
    ok()
    for wrong in (dict(block=None), dict(block=None, resid=None), dict(block=None, gate=None), dict(h=None, x=None, w_pre=None),
                  dict(x=None), dict(w_pre=None), dict(x=h), dict(eps=-1.0), dict(eps=float("nan")), dict(alpha=float("inf")),
                  dict(resid=a["resid_t"].bfloat16()), dict(gate=a["gate_t"][:2].contiguous()), dict(h=h[:2]),
                  dict(w_post=a["w_post_t"][:5].contiguous()), dict(resid=a["resid_t"].t()), dict(w_pre=a["w_pre_t"].bfloat16())):
        with pytest.raises((ValueError, B.ColiError)):
            ok(**wrong)
    lib = B.library()
    call = lambda **k: lib.coli_norm_residual(*{**dict(ctx=ctx, b=a["block_t"].data_ptr(), r=None, g=None, gr=0, gsig=0, al=1.0,  # noqa: E731
                                                       wp=None, wq=None, eps=0.0, dt=0, S=4, D=64, h=h.data_ptr(), x=None),
                                                  **k}.values())
    assert call() == 0
    for wrong in (dict(S=0), dict(S=65537), dict(D=0), dict(D=32769), dict(dt=3), dict(g=h.data_ptr(), gr=2),
                  dict(b=a["block_t"].data_ptr() + 2), dict(h=None)):
        assert call(**wrong) == B.COLI_E_INVAL, wrong
        assert B.coli_last_error(ctx).startswith("norm_residual")
