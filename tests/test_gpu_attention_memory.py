"""Where the cache attention keeps its partial results: memory of the context's own that is there after coli_reserve or the
first call, and that no later call moves."""
import pytest
import torch

from int4_grouped_expert_router_gb300 import binding as B
from int4_grouped_expert_router_gb300.workload import CONFIGS, DeviceLayer
from gpu_util import Ctx
from kv4_util import Batch

pytestmark = pytest.mark.gpu

FORMS = [("bf16", 64, 32, [1, 1], 8), ("bf16", 128, 64, [1, 1], 24), ("f32", 256, 128, [1, 1], 32), ("bf16", 128, 64, [200, 300], 8)]


def test_a_reserve_is_enough_for_every_form():
    """After coli_reserve no compute call allocates: free memory stays as it is through the first attention of each form."""
    def attend_all(ctx):
        for b, q, rows in work:
            b.ctx = ctx
            b.attend(q, rows, out=outs[id(b)])
        assert B.coli_check_error(ctx) == 0

    a, c = Ctx(), Ctx()
    try:
        work, outs = [], {}
        for dtype, hd, gs, rows, q_heads in FORMS:
            b = Batch(a.ctx, [2000, 700], 2, hd, gs, 32, dtype)
            _, q = b.queries(rows, q_heads)
            work.append((b, q, rows))
            outs[id(b)] = torch.empty_like(q)
        attend_all(a.ctx)  # loads the kernels, and fills torch's own pool
        B.coli_reserve(c.ctx, 1, 16, 4, 256, 128)
        torch.cuda.synchronize()
        free, _ = torch.cuda.mem_get_info()
        attend_all(c.ctx)
        assert torch.cuda.mem_get_info()[0] == free
    finally:
        a.close()
        c.close()


@pytest.mark.parametrize("reserve", [True, False])
def test_a_captured_step_outlives_larger_calls(reserve):
    """A decode step (experts and attention) is captured; prompts of other forms then run in the same context; the step
    replays as it was."""
    c = Ctx()
    layer = None
    try:
        if reserve:
            B.coli_reserve(c.ctx, 1, 16, 4, 256, 128)
        cfg = CONFIGS["tiny"]
        layer = DeviceLayer(c.ctx, cfg)
        out = layer.outputs()
        x = torch.randn(1, cfg.D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
        b = Batch(c.ctx, [3000, 700], 2, 64, 32, 32, "bf16")
        _, q = b.queries([1, 1], 8)
        att = torch.empty_like(q)

        def step():
            layer.step(x, None, out)
            b.attend(q, [1, 1], out=att)

        step()
        torch.cuda.synchronize()
        want = out["y"].clone(), att.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        try:
            with torch.cuda.graph(graph, stream=side):
                B.coli_set_stream(c.ctx, torch.cuda.current_stream())
                step()
        finally:
            B.coli_set_stream(c.ctx, torch.cuda.current_stream())
        held = []
        for dtype, hd, gs, rows, q_heads in FORMS:
            p = Batch(c.ctx, [2000, 700], 2, hd, gs, 32, dtype)
            _, pq = p.queries(rows, q_heads)
            p.attend(pq, rows)
            # whatever was freed would be handed out again here, and a replay would write into it
            held.append([torch.zeros(1 << 20, device="cuda") for _ in range(8)])
        torch.cuda.synchronize()
        out["y"].zero_()
        att.zero_()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["y"], want[0]) and torch.equal(att, want[1])
        assert not any(bool(t.any()) for ts in held for t in ts)
        assert B.coli_check_error(c.ctx) == 0
    finally:
        if layer is not None:
            layer.free()
        c.close()
