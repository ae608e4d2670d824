"""A decoder layer with positions and an output head, run as it would be used, against the oracles put together the same way."""
import numpy as np
import pytest
import torch

import oracle.kv4 as K
import oracle.moe as O
import oracle.tokens as T
from int4_grouped_expert_router_gb300 import binding as B
from int4_grouped_expert_router_gb300.run_decoder import DecoderLayer, Head
from int4_grouped_expert_router_gb300.workload import LayerConfig
from gpu_util import Ctx, oracle_experts
from kv4_util import rng

pytestmark = pytest.mark.gpu

# An output is off by what one code of the cache that rounds the other way moves it (see the test of the layer alone), in norm.
NORMWISE = 1e-4


def forward_oracle(layer, cfg, h, new, cached, turns):
    """The layer with the oracles; `cached` holds the turned k and the v rows of each sequence so far."""
    w = {k: v.cpu().numpy().astype(np.float64) for k, v in layer.norms.items()}
    hq, hk, hd = layer.q_heads, layer.kv_heads, layer.head_dim
    tensor = {k: O.Tensor(*layer.packed[k], *layer.shapes[k], 0) for k in layer.packed}
    _, n = K.norm_residual(None, h, None, 1.0, None, w["w_in"], layer.eps)
    qkv = O.w4_linear(n, tensor["qkv"], None)
    att, at = [], 0
    for b, m in enumerate(new):
        rows = qkv[at:at + m]
        at += m
        have = 0 if cached[b][0] is None else cached[b][0].shape[0]
        pos = have + np.arange(m)
        q, k, v = (rows[:, o:o + n_ * hd].reshape(m, n_, hd) for o, n_ in ((0, hq), (hq * hd, hk), ((hq + hk) * hd, hk)))
        q, k = T.rotary(q, turns, pos), T.rotary(k, turns, pos)
        new_kv = (k.astype(np.float32), v.astype(np.float32))
        cached[b] = [np.concatenate(p) if p[0] is not None else p[1] for p in zip(cached[b], new_kv)]
        ks, vs = (K.stored(t, layer.cache.gs) for t in cached[b])
        att.append(K.attention(q, ks, vs, pos, hd ** -0.5)[0])
    o = O.w4_linear(np.concatenate(att).reshape(-1, hq * hd), tensor["o"], None)
    h1, n = K.norm_residual(o, h, None, 1.0, w["w_post"], w["w_pre"], layer.eps)
    n = n.astype(np.float32)
    idx, wt, kept, _ = O.router_select(n, layer.moe.Wr.cpu().numpy(), layer.moe.bias.cpu().numpy(), cfg.K, cfg.topp,
                                       cfg.norm_topk, cfg.routed_scale)
    y = O.expert_group(n, oracle_experts(cfg, idx), idx, wt, kept, None)
    return K.norm_residual(y, h1, None, 1.0, w["w_post2"], w["w_next"], layer.eps)


def test_prompt_and_decode_steps_with_positions_and_a_head():
    cfg = LayerConfig("decoder tokens", D=256, I=128, E=8, K=2, routed_scale=2.5)
    c = Ctx()
    freqs = B.coli_rotary_freqs(64, 500.0, scaling="parts", factor=4.0, original_len=32, low=1.0, high=4.0)
    layer = DecoderLayer(c.ctx, cfg, 8, 2, 64, 64, batch=2, max_len=80, rotary=freqs)
    head = Head(c.ctx, cfg, 1003)
    W = head.weight.float().numpy().astype(np.float64)
    try:
        cached = [[None, None], [None, None]]
        for step, new in enumerate(([37, 20], [1, 1], [1, 1], [3, 2])):
            h = rng("decoder tokens", step).normal(size=(sum(new), cfg.D)).astype(np.float32)
            got = layer.forward(torch.from_numpy(h).cuda(), new)
            last = torch.tensor(np.cumsum(new) - 1, device="cuda")
            answer = head.forward(got[1][last], top=5)
            assert B.coli_check_error(c.ctx) == 0
            want = forward_oracle(layer, cfg, h, new, cached, [int(t) % 2 ** 64 for t in freqs.cpu()])
            for g, r in zip(got, want):
                off = np.linalg.norm(g.cpu().numpy() - r) / np.linalg.norm(r)
                assert off < NORMWISE, (step, off)
            logits = want[1][np.cumsum(new) - 1] @ W.T
            have = answer["logits"].cpu().numpy()
            assert np.linalg.norm(have - logits) < 2 * NORMWISE * np.linalg.norm(logits)
            lp, entropy = T.logprobs(have)
            ids = T.top(have, 5)
            assert np.array_equal(answer["top_id"].cpu().numpy(), ids)
            assert np.allclose(answer["top_logp"].cpu().numpy(), np.take_along_axis(lp, ids, 1), atol=1e-5)
            assert np.allclose(answer["entropy"].cpu().numpy(), entropy, atol=1e-4)
    finally:
        head.free()
        layer.free()
        c.close()


def test_the_layer_without_positions_is_as_it_was():
    """A table whose frequencies are 0 turns nothing: the same bits as without a rotary step."""
    cfg = LayerConfig("decoder tokens", D=256, I=128, E=8, K=2, routed_scale=2.5)
    c = Ctx()
    outs = []
    try:
        for rotary in (None, torch.zeros(32, dtype=torch.int64, device="cuda")):
            layer = DecoderLayer(c.ctx, cfg, 8, 2, 64, 64, batch=2, max_len=80, rotary=rotary)
            for step, new in enumerate(([9, 4], [1, 1])):
                h = rng("still", step).normal(size=(sum(new), cfg.D)).astype(np.float32)
                outs.append(layer.forward(torch.from_numpy(h).cuda(), new)[0])
            layer.free()
        assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
        assert B.coli_check_error(c.ctx) == 0
    finally:
        c.close()


def test_the_example_runs(capsys):
    from int4_grouped_expert_router_gb300 import run_decoder
    assert run_decoder.main(["--prompt", "70", "--steps", "3", "--batch", "3", "--rotary", "--vocab", "1000"]) == 0
    out = capsys.readouterr().out
    assert "decode step" in out and "mean entropy" in out


def test_calls_one_after_another_read_what_the_one_before_wrote():
    """Projection, rotary in its rows, append, head and log probabilities with no wait between them, many times over: each kernel
    starts while the one before it ends, and gives what it gives with a wait between."""
    c = Ctx()
    g = torch.Generator(device="cuda").manual_seed(5)
    try:
        W = B.coli_dense_upload(c.ctx, (0.1 * torch.randn(640, 256, device="cuda", generator=g)).bfloat16())
        H = B.coli_dense_upload(c.ctx, (0.1 * torch.randn(5000, 256, device="cuda", generator=g)).bfloat16())
        freqs = B.coli_rotary_freqs(64)
        for S in (1, 40, 300):
            xs = [torch.randn(S, 256, device="cuda", generator=g) for _ in range(6)]
            runs = []
            for wait in (True, False):
                res = []
                qkv, logits = torch.empty(S, 10, 64, device="cuda"), torch.empty(S, 5000, device="cuda")
                x2 = torch.empty(S, 256, device="cuda")
                for i in range(30):
                    e, ids, lp = torch.empty(S, device="cuda"), torch.empty(S, 4, dtype=torch.int32, device="cuda"), torch.empty(S, 4, device="cuda")
                    pos = torch.full((S,), i, dtype=torch.int32, device="cuda")
                    for call in (lambda: B.coli_dense_linear(c.ctx, W, xs[i % 6], qkv.view(S, 640)),
                                 lambda: B.coli_rotary(c.ctx, qkv[:, :8], qkv[:, 8:], freqs, qkv[:, :8], qkv[:, 8:], positions=pos),
                                 lambda: B.coli_norm_residual(c.ctx, None, qkv.view(S, 640)[:, :256].contiguous(), None, 1.0, None,
                                                              torch.ones(256, device="cuda"), 1e-5, None, x2),
                                 lambda: B.coli_dense_linear(c.ctx, H, x2, logits),
                                 lambda: B.coli_logprobs(c.ctx, logits, entropy=e, top_id=ids, top_logp=lp)):
                        call()
                        if wait:
                            torch.cuda.synchronize()
                    res += [e, ids, lp]
                assert B.coli_check_error(c.ctx) == 0
                runs.append(res)
            for a, b in zip(*runs):
                assert torch.equal(a, b)
    finally:
        c.close()
