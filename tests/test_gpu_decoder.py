"""A decoder layer run as it would be used (norms, int4 projections, 4-bit cache, attention, router and experts),
against the oracles put together the same way."""
import numpy as np
import pytest
import torch

import oracle.kv4 as K
import oracle.moe as O
from int4_grouped_expert_router_gb300 import binding as B
from int4_grouped_expert_router_gb300.run_decoder import DecoderLayer
from int4_grouped_expert_router_gb300.workload import LayerConfig
from gpu_util import Ctx, oracle_experts
from kv4_util import rng

pytestmark = pytest.mark.gpu

# 64 channels of a head in a group, f32 activations: an output is off by what one code of the cache that rounds the
# other way (its input a binary32 rounding away from the middle) moves it, at most a few such codes of thousands.
# A step is about a seventh of a group's range; the rows are compared in norm, with one in ten thousand allowed.
NORMWISE = 1e-4


def forward_oracle(layer, cfg, h, new, cached):
    """The same layer with the oracles; `cached` holds the plain k, v rows of each sequence so far."""
    w = {k: v.cpu().numpy().astype(np.float64) for k, v in layer.norms.items()}
    hq, hk, hd = layer.q_heads, layer.kv_heads, layer.head_dim
    tensor = {k: O.Tensor(*layer.packed[k], *layer.shapes[k], 0) for k in layer.packed}
    _, n = K.norm_residual(None, h, None, 1.0, None, w["w_in"], layer.eps)
    qkv = O.w4_linear(n, tensor["qkv"], None)
    att, at = [], 0
    for b, m in enumerate(new):
        rows = qkv[at:at + m]
        at += m
        k, v = (rows[:, o:o + hk * hd].reshape(m, hk, hd).astype(np.float32) for o in (hq * hd, (hq + hk) * hd))
        cached[b] = [np.concatenate(p) if p[0] is not None else p[1] for p in zip(cached[b], (k, v))]
        ks, vs = (K.stored(t, layer.cache.gs) for t in cached[b])
        total = ks.shape[0]
        att.append(K.attention(rows[:, :hq * hd].reshape(m, hq, hd), ks, vs, total - m + np.arange(m), hd ** -0.5)[0])
    o = O.w4_linear(np.concatenate(att).reshape(-1, hq * hd), tensor["o"], None)
    h1, n = K.norm_residual(o, h, None, 1.0, w["w_post"], w["w_pre"], layer.eps)
    n = n.astype(np.float32)
    idx, wt, kept, _ = O.router_select(n, layer.moe.Wr.cpu().numpy(), layer.moe.bias.cpu().numpy(), cfg.K, cfg.topp,
                                       cfg.norm_topk, cfg.routed_scale)
    y = O.expert_group(n, oracle_experts(cfg, idx), idx, wt, kept, None)
    return K.norm_residual(y, h1, None, 1.0, w["w_post2"], w["w_next"], layer.eps)


def test_prompt_and_decode_steps_match_the_oracles():
    cfg = LayerConfig("decoder", D=256, I=128, E=8, K=2, routed_scale=2.5)
    c = Ctx()
    layer = DecoderLayer(c.ctx, cfg, 8, 2, 64, 64, batch=2, max_len=80)
    try:
        cached = [[None, None], [None, None]]
        for step, new in enumerate(([37, 20], [1, 1], [1, 1], [3, 2])):
            h = rng("decoder", step).normal(size=(sum(new), cfg.D)).astype(np.float32)
            got = layer.forward(torch.from_numpy(h).cuda(), new)
            assert B.coli_check_error(c.ctx) == 0
            want = forward_oracle(layer, cfg, h, new, cached)
            for g, r in zip(got, want):
                off = np.linalg.norm(g.cpu().numpy() - r) / np.linalg.norm(r)
                assert off < NORMWISE, (step, off)
    finally:
        layer.free()
        c.close()


def test_the_example_runs(capsys):
    from int4_grouped_expert_router_gb300 import run_decoder
    assert run_decoder.main(["--prompt", "70", "--steps", "3", "--batch", "3"]) == 0
    assert "decode step" in capsys.readouterr().out
