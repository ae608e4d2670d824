"""Run a synthetic decoder layer through the C ABI: a prompt, then one token at a time.

    python -m int4_grouped_expert_router_gb300.run_decoder [--workload tiny] [--batch B] [--prompt N] [--steps N]

The layer on the device, with nothing but library calls between the residual stream going in and coming out. It has no
positions: the library has no rotary step, which a model's q and k get between the projection and the append.

    n      = rmsnorm(h, w_in)                                    coli_norm_residual (no block)
    q,k,v  = Wqkv n                                              coli_w4_linear
    the new k, v quantised into the paged 4-bit cache            coli_kv4_append
    a      = attention of q over the cache                       coli_kv4_attention
    o      = Wo a                                                coli_w4_linear
    h, n   = h + rmsnorm(o, w_post), rmsnorm(h, w_pre)           coli_norm_residual
    y      = routed int4 experts of n                            coli_router_select, coli_expert_group
    h, n   = h + rmsnorm(y, w_post2), rmsnorm(h, w_next)         coli_norm_residual

Prints the event-timed microseconds of the prompt pass and of a decode step (the median), after the device error word has
come back clean.
"""
from __future__ import annotations

import argparse
import sys

import numpy as np
import torch

from . import binding as B
from . import synth
from .build import build
from .workload import CONFIGS, DeviceLayer


class DecoderLayer:
    """The weights of one layer and its cache: `batch` sequences of up to `max_len` tokens on pages of 64."""

    PAGE = 64

    def __init__(self, ctx, cfg, q_heads, kv_heads, head_dim, gs, batch, max_len, device="cuda"):
        self.ctx, self.cfg, self.q_heads, self.kv_heads, self.head_dim = ctx, cfg, q_heads, kv_heads, head_dim
        self.eps = 1e-5
        self.moe = DeviceLayer(ctx, cfg)
        self.shapes = {"qkv": ((q_heads + 2 * kv_heads) * head_dim, cfg.D), "o": (cfg.D, q_heads * head_dim)}
        self.packed, self.linear = {}, {}
        for name, (rows, cols) in self.shapes.items():
            p, s = synth.expert_tensor(synth.stream_seed(cfg.seed, "attention", name), rows, cols, 0)
            self.packed[name] = (p, s)
            self.linear[name] = B.coli_expert_upload(ctx, torch.from_numpy(p), torch.from_numpy(s), rows, cols, 0)
        # one weight per channel and norm: before attention, after it, before the experts, after them, next layer's
        self.norms = {name: torch.from_numpy((0.25 + 0.05 * synth.normal(synth.stream_seed(cfg.seed, "norm", name), cfg.D))
                                             .astype(np.float32)).to(device)
                      for name in ("w_in", "w_post", "w_pre", "w_post2", "w_next")}
        per = -(-max_len // self.PAGE)
        self.cache = B.coli_kv4_cache(batch * per, self.PAGE, kv_heads, head_dim, gs, device)
        self.table = torch.arange(batch * per, dtype=torch.int32, device=device).view(batch, per)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)

    def forward(self, h, new):
        """One pass over `h` [T x D], the rows of sequence b being its next `new[b]` tokens; returns (h, the next
        layer's normed input)."""
        B_, ctx, w = B, self.ctx, self.norms
        T, dt, dev = h.shape[0], h.dtype, h.device
        self.lens += torch.tensor(new, dtype=torch.int32, device=dev)
        one = all(m == 1 for m in new)
        start = None if one else torch.tensor(np.concatenate(([0], np.cumsum(new))), dtype=torch.int32, device=dev)
        plan = dict(lens=self.lens, table=self.table, q_start=start)
        n = torch.empty_like(h)
        B_.coli_norm_residual(ctx, None, h, None, 1.0, None, w["w_in"], self.eps, None, n)
        qkv = torch.empty(T, self.shapes["qkv"][0], dtype=dt, device=dev)
        B_.coli_w4_linear(ctx, self.linear["qkv"], n, None, qkv)
        q, k, v = (t.unflatten(1, (-1, self.head_dim)) for t in
                   qkv.split([self.q_heads * self.head_dim, self.kv_heads * self.head_dim, self.kv_heads * self.head_dim], 1))
        B_.coli_kv4_append(ctx, self.cache, k, v, **plan)
        a = torch.empty(T, self.q_heads, self.head_dim, dtype=dt, device=dev)
        B_.coli_kv4_attention(ctx, self.cache, q, out=a, **plan)
        o = torch.empty_like(h)
        B_.coli_w4_linear(ctx, self.linear["o"], a.view(T, -1), None, o)
        h1 = torch.empty_like(h)
        B_.coli_norm_residual(ctx, o, h, None, 1.0, w["w_post"], w["w_pre"], self.eps, h1, n)
        out = self.moe.outputs(T)
        self.moe.step(n, None, out)
        h2 = torch.empty_like(h)
        B_.coli_norm_residual(ctx, out["y"], h1, None, 1.0, w["w_post2"], w["w_next"], self.eps, h2, n)
        return h2, n

    def free(self):
        self.moe.free()
        for t in self.linear.values():
            B.coli_expert_free(self.ctx, t)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--workload", default="tiny", choices=sorted(CONFIGS))
    ap.add_argument("--experts", type=int, default=0, help="use only the first E experts")
    ap.add_argument("--heads", type=int, default=8, help="query heads")
    ap.add_argument("--kv-heads", type=int, default=2)
    ap.add_argument("--head-dim", type=int, default=64)
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--prompt", type=int, default=100, help="tokens of each prompt")
    ap.add_argument("--steps", type=int, default=20, help="tokens decoded after it")
    args = ap.parse_args(argv)
    import dataclasses
    build()
    cfg = CONFIGS[args.workload]
    if args.experts:
        cfg = dataclasses.replace(cfg, E=args.experts, K=min(cfg.K, args.experts))
    ctx = B.coli_init(0)
    layer = DecoderLayer(ctx, cfg, args.heads, args.kv_heads, args.head_dim, 64, args.batch, args.prompt + args.steps)
    times = []
    for step in range(args.steps + 1):
        new = [args.prompt if step == 0 else 1] * args.batch
        h = layer.moe.act_tensor(synth.normal(synth.stream_seed(cfg.seed, "hidden", step), sum(new) * cfg.D)
                                 .reshape(-1, cfg.D))
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        layer.forward(h, new)
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 1000.0)
    rc = B.coli_check_error(ctx)
    layer.free()
    B.coli_destroy(ctx)
    if rc != 0:
        print(f"device error {rc}", file=sys.stderr)
        return 1
    decode = sorted(times[1:])
    print(f"{cfg.name} batch {args.batch}: prompt of {args.prompt} {times[0]:.1f} us, decode step "
          f"{decode[len(decode) // 2] if decode else float('nan'):.1f} us (median of {len(decode)})")
    return 0


if __name__ == "__main__":
    sys.exit(main())
